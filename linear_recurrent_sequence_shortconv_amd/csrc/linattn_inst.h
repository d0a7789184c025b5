// Instances of the chunk kernel by operand size (included by one source per
// storage type).
#pragma once

#include "linattn_kernel.h"

namespace prism {

template <typename E, int DA, int NCT>
hipError_t la_pass_da(const LaArgs<E>& a, bool precise, hipStream_t s) {
  if (precise) return la_launch<E, DA, NCT, true, true>(a, s);
  return la_launch<E, DA, NCT, false, true>(a, s);
}

template <typename E>
hipError_t launch_la_pass(const LaArgs<E>& a, int dim, bool outputs, bool precise, hipStream_t s) {
  if (!outputs) {
    if (dim <= 32) return la_launch<E, 32, 1, false, false>(a, s);
    if (dim <= 64) return la_launch<E, 64, 1, false, false>(a, s);
    return la_launch<E, 128, 2, false, false>(a, s);
  }
  if (dim <= 32) return la_pass_da<E, 32, 1>(a, precise, s);
  if (dim <= 64) return la_pass_da<E, 64, 1>(a, precise, s);
  return la_pass_da<E, 128, 2>(a, precise, s);
}

}  // namespace prism
