// Instances of the chunk kernel by operand size (included by one source per
// storage type).
#pragma once

#include "linattn_kernel.h"

namespace prism {

template <typename E, int DA, int NCT>
hipError_t la_pass_da(const LaArgs<E>& a, LaPass kind, hipStream_t s) {
  constexpr bool HALF = sizeof(E) == 2;   // (fp32 operands are one piece in every kind)
  constexpr int THREE = HALF ? 3 : 1, TWO = HALF ? 2 : 1;
  switch (kind) {
    case LA_STATES: return la_launch<E, DA, NCT, false, false, TWO>(a, s);
    case LA_STATES_FP32: return la_launch<E, DA, NCT, false, false, THREE>(a, s);
    case LA_OUT: return la_launch<E, DA, NCT, false, true, TWO>(a, s);
    case LA_OUT_STATE: return la_launch<E, DA, NCT, false, true, THREE>(a, s);
    case LA_OUT_DOTS: return la_launch<E, DA, NCT, true, true, THREE>(a, s);
  }
  return hipErrorInvalidValue;
}

template <typename E>
hipError_t launch_la_pass(const LaArgs<E>& a, int dim, LaPass kind, hipStream_t s) {
  if (dim <= 32) return la_pass_da<E, 32, 1>(a, kind, s);
  if (dim <= 64) return la_pass_da<E, 64, 1>(a, kind, s);
  return la_pass_da<E, 128, 2>(a, kind, s);
}

}  // namespace prism
