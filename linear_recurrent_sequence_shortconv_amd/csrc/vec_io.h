// Vectors of a lane: V consecutive values of a row in the storage type, as raw
// words, and as fp32; sums over groups of lanes.
#pragma once

#include "prism_common.h"

namespace prism {

template <typename E, int V> struct VecIo;
template <> struct VecIo<bf16, 8> {
  typedef uint4 raw;
  __device__ static inline void unpack(const raw& w, float (&x)[8]) {
    const unsigned u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  __device__ static inline raw pack(const float (&x)[8]) {
    bf16 b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = (bf16)x[i];
    raw w;
    __builtin_memcpy(&w, b, 16);
    return w;
  }
};
template <> struct VecIo<bf16, 4> {
  typedef uint2 raw;
  __device__ static inline void unpack(const raw& w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x << 16);
    x[1] = __uint_as_float(w.x & 0xffff0000u);
    x[2] = __uint_as_float(w.y << 16);
    x[3] = __uint_as_float(w.y & 0xffff0000u);
  }
  __device__ static inline raw pack(const float (&x)[4]) {
    const bf16 b[4] = {(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3]};
    raw w;
    __builtin_memcpy(&w, b, 8);
    return w;
  }
};
template <> struct VecIo<bf16, 2> {
  typedef unsigned raw;
  __device__ static inline void unpack(const raw& w, float (&x)[2]) {
    x[0] = __uint_as_float(w << 16);
    x[1] = __uint_as_float(w & 0xffff0000u);
  }
  __device__ static inline raw pack(const float (&x)[2]) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(raw, __builtin_convertvector((f2){x[0], x[1]}, b2));
  }
};
template <> struct VecIo<bf16, 1> {
  typedef unsigned short raw;
  __device__ static inline void unpack(const raw& w, float (&x)[1]) { x[0] = __uint_as_float((unsigned)w << 16); }
  __device__ static inline raw pack(const float (&x)[1]) {
    const bf16 b = (bf16)x[0];
    raw w;
    __builtin_memcpy(&w, &b, 2);
    return w;
  }
};
template <> struct VecIo<float, 1> {
  typedef float raw;
  __device__ static inline void unpack(const raw& w, float (&x)[1]) { x[0] = w; }
  __device__ static inline raw pack(const float (&x)[1]) { return x[0]; }
};
template <> struct VecIo<float, 4> {
  typedef f32x4 raw;
  __device__ static inline void unpack(const raw& w, float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = w[i];
  }
  __device__ static inline raw pack(const float (&x)[4]) { return raw{x[0], x[1], x[2], x[3]}; }
};

// V values from an address of any alignment (the memory unit takes 16 bytes from
// any), and those behind the first `skip` of them to one: lanes of a row whose width
// is no multiple of V take V values each all the same, the last with values of the
// lane before it in front, which it neither counts nor writes.
template <typename E, int V>
__device__ inline typename VecIo<E, V>::raw load_vec(const E* p) {
  typename VecIo<E, V>::raw w;
  __builtin_memcpy(&w, p, sizeof(w));
  return w;
}
template <typename E, int V>
__device__ inline void store_vec(E* p, const float (&x)[V]) {
  const typename VecIo<E, V>::raw w = VecIo<E, V>::pack(x);
  __builtin_memcpy(p, &w, sizeof(w));
}
template <typename E, int V>
__device__ inline void store_vec(E* p, const float (&x)[V], int skip) {
  if (skip == 0) {
    store_vec<E, V>(p, x);
  } else {
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (i >= skip) p[i] = (E)x[i];
  }
}
// (whole: no lane of the wave skips any)
template <typename E, int V>
__device__ inline void store_vec(E* p, const float (&x)[V], int skip, bool whole) {
  if (whole)
    store_vec<E, V>(p, x);
  else
    store_vec<E, V>(p, x, skip);
}

// Sum over each group of G = 1, 2, .., 32 consecutive lanes, in every lane of
// the group: quad permutations, then mirrors of half rows and rows (whose
// quads already hold equal values), then one exchange between rows.
#define QN_DPP(v, ctrl) \
  __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, (v)), (ctrl), 0xf, 0xf, false))
__device__ inline float group_sum(float v, int G) {
  if (G > 1) v += QN_DPP(v, 0xB1);
  if (G > 2) v += QN_DPP(v, 0x4E);
  if (G > 4) v += QN_DPP(v, 0x141);
  if (G > 8) v += QN_DPP(v, 0x140);
  if (G > 16) v += __shfl_xor(v, 16);
  return v;
}
#undef QN_DPP

}  // namespace prism
