// Tiles of the gated recurrence, two bf16 channels a lane.
#include "recurrence_tile.h"

namespace prism {
PRISM_RECURRENCE_TILES(bf16, 2)
}  // namespace prism
