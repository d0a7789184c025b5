// Which tile a workgroup of the gated recurrence takes.  Plain C++, without HIP's
// headers: its range is checked on the host too.
#pragma once

#ifdef __HIPCC__
#define PRISM_HOST_DEVICE __host__ __device__
#else
#define PRISM_HOST_DEVICE
#endif

namespace prism {

struct TilePlace {
  int turn, slice;   // turn < 0: no tile
};
// Workgroups count themselves: number `id` takes slice id % slices of the tile whose
// turn is id / slices.  A counter that something else wrote to (a second call on the
// same workspace, which is an error) may give any number: those beyond the last
// workgroup's have no place.
PRISM_HOST_DEVICE inline TilePlace tile_place(unsigned id, int tiles, int slices) {
  const unsigned turn = id / (unsigned)slices;
  if (turn >= (unsigned)tiles) return TilePlace{-1, 0};
  return TilePlace{(int)turn, (int)(id - turn * (unsigned)slices)};
}

}  // namespace prism
