// Tiles of the gated recurrence, one fp32 channel a lane.
#include "recurrence_tile.h"

namespace prism {
PRISM_RECURRENCE_TILES(float, 1)
}  // namespace prism
