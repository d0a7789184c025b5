// Tiles of the gated recurrence, one bf16 channel a lane.
#include "recurrence_tile.h"

namespace prism {
PRISM_RECURRENCE_TILES(bf16, 1)
}  // namespace prism
