// Gated recurrence h_t = a_t h_{t-1} + u_t, channel by channel, and its
// backward pass: with g_t the gradient of h_t from its own row and the tokens
// behind it,
//   g_t = dh_t + a_{t+1} g_{t+1},  d(a_t) = g_t h_{t-1},  d(u_t) = g_t,
// dhT added at the last token, dh0 = a_1 g_1.  h_{t-1} is read from the forward
// pass's output.
//
// A lane takes V channels of one sequence and walks its tokens.
#include "recurrence_kernel.h"

namespace prism {

namespace {

template <typename E, int V>
__device__ inline void load_v(const void* p, long at, float (&x)[V]) {
  typedef typename VecIo<E, V>::raw raw;
  VecIo<E, V>::unpack(*reinterpret_cast<const raw*>(static_cast<const E*>(p) + at), x);
}
template <typename E, int V>
__device__ inline void store_v(void* p, long at, const float (&x)[V]) {
  typedef typename VecIo<E, V>::raw raw;
  *reinterpret_cast<raw*>(static_cast<E*>(p) + at) = VecIo<E, V>::pack(x);
}

// First row and tokens of sequence b (packed: the largest clamped offset so far
// to the next), by every thread of a workgroup.
__device__ inline void sequence_rows(const RecurrenceArgs& a, int b, int* sm, int& start, int& n) {
  if (!a.cu) {
    start = b * a.T;
    n = a.T;
    return;
  }
  int m = 0;
  for (int j = threadIdx.x; j <= b; j += 256) m = max(m, min(a.cu[j], a.rows));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, __shfl_xor(m, o));
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = m;
  __syncthreads();
  start = max(max(sm[0], sm[1]), max(sm[2], sm[3]));
  n = max(min(a.cu[b + 1], a.rows) - start, 0);
}

template <typename E, int V, int G, bool INP>
__global__ __launch_bounds__(256) void recurrence_walk_kernel(const RecurrenceArgs a, int cb) {
  __shared__ int sm[4];
  const int b = blockIdx.x / cb, c = ((blockIdx.x % cb) * 256 + threadIdx.x) * V;
  int start, n;
  sequence_rows(a, b, sm, start, n);
  if (c >= a.D) return;
  float h[V], lam[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = a.h0 ? a.h0[(long)b * a.D + c + v] : 0.f;
    lam[v] = G == GATE_POWER ? a.lam[c + v] : 0.f;
  }
  auto at = [&](const TokenSteps& s, int t) { return (a.cu ? (start + t) * s.t : b * s.b + t * s.t) + c; };
  for (int t = 0; t < n; ++t) {
    float x[V], f[V], i[V];
    load_v<E, V>(a.x, at(a.sx, t), x);
    load_v<E, V>(a.f, at(a.sf, t), f);
    if (INP) load_v<E, V>(a.i, at(a.si, t), i);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float av, u;
      gate_inputs<E, G, INP>(x[v], f[v], INP ? i[v] : 0.f, lam[v], av, u);
      h[v] = fmaf(av, h[v], u);
    }
    store_v<E, V>(a.h, at(a.sh, t), h);
  }
  if (a.hT) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.hT[(long)b * a.D + c + v] = h[v];
  }
}

template <typename E, int V, int G, bool INP>
__global__ __launch_bounds__(256) void recurrence_walk_bwd_kernel(const RecurrenceArgs a, int cb) {
  __shared__ int sm[4];
  const int b = blockIdx.x / cb, c = ((blockIdx.x % cb) * 256 + threadIdx.x) * V;
  int start, n;
  sequence_rows(a, b, sm, start, n);
  if (c >= a.D) return;
  float carry[V], lam[V], dlam[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    carry[v] = a.dhT ? a.dhT[(long)b * a.D + c + v] : 0.f;
    lam[v] = G == GATE_POWER ? a.lam[c + v] : 0.f;
    dlam[v] = 0.f;
  }
  auto at = [&](const TokenSteps& s, int t) { return (a.cu ? (start + t) * s.t : b * s.b + t * s.t) + c; };
  for (int t = n - 1; t >= 0; --t) {
    float x[V], f[V], i[V], g[V], before[V], dx[V], df[V], di[V];
    load_v<E, V>(a.x, at(a.sx, t), x);
    load_v<E, V>(a.f, at(a.sf, t), f);
    if (INP) load_v<E, V>(a.i, at(a.si, t), i);
    load_v<E, V>(a.dh, at(a.sdh, t), g);
    if (t > 0) {
      load_v<E, V>(a.h, at(a.sh, t - 1), before);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) before[v] = a.h0 ? a.h0[(long)b * a.D + c + v] : 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float av, cv, dl;
      gate_values<E, G>(f[v], lam[v], av, cv);
      g[v] += carry[v];
      carry[v] = av * g[v];
      gate_gradients<E, G, INP>(x[v], f[v], INP ? i[v] : 0.f, lam[v], before[v], g[v], dx[v], df[v], di[v], dl);
      dlam[v] += dl;
    }
    store_v<E, V>(a.dx, at(a.sdx, t), dx);
    store_v<E, V>(a.df, at(a.sdf, t), df);
    if (INP) store_v<E, V>(a.di, at(a.sdi, t), di);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (a.dh0) a.dh0[(long)b * a.D + c + v] = carry[v];
    if (G == GATE_POWER) a.part[(long)b * a.D + c + v] = dlam[v];
  }
}

template <typename E, int V, int G, bool INP>
hipError_t run_walk(const RecurrenceArgs& a, hipStream_t s) {
  const int cb = (a.D + 256 * V - 1) / (256 * V);
  if (a.B == 0) return hipSuccess;
  hipLaunchKernelGGL((recurrence_walk_kernel<E, V, G, INP>), dim3((unsigned)cb * a.B), dim3(256), 0, s, a, cb);
  return hipGetLastError();
}
template <typename E, int V, int G, bool INP>
hipError_t run_walk_bwd(const RecurrenceArgs& a, hipStream_t s) {
  const int cb = (a.D + 256 * V - 1) / (256 * V);
  if (a.B > 0) {
    hipLaunchKernelGGL((recurrence_walk_bwd_kernel<E, V, G, INP>), dim3((unsigned)cb * a.B), dim3(256), 0, s, a, cb);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (G == GATE_POWER) return launch_column_sums(a.part, a.B, a.D, a.D, 0, a.dlam, s);
  return hipSuccess;
}

// bf16 channels two a lane where every row starts at a multiple of 4 bytes.
template <typename E>
bool pairs(const RecurrenceArgs& a, bool bwd) {
  if (sizeof(E) == 4) return false;
  long m = a.D | a.sx.b | a.sx.t | a.sf.b | a.sf.t | a.sh.b | a.sh.t;
  uintptr_t p = (uintptr_t)a.x | (uintptr_t)a.f | (uintptr_t)a.i | (uintptr_t)a.h;
  if (a.i) m |= a.si.b | a.si.t;
  if (bwd) {
    m |= a.sdh.b | a.sdh.t | a.sdx.b | a.sdx.t | a.sdf.b | a.sdf.t;
    p |= (uintptr_t)a.dh | (uintptr_t)a.dx | (uintptr_t)a.df | (uintptr_t)a.di;
    if (a.i) m |= a.sdi.b | a.sdi.t;
  }
  return m % 2 == 0 && p % 4 == 0;
}

template <typename E, int V, bool BWD, int G>
hipError_t run_gate(const RecurrenceArgs& a, hipStream_t s) {
  if (a.i) return BWD ? run_walk_bwd<E, V, G, true>(a, s) : run_walk<E, V, G, true>(a, s);
  return BWD ? run_walk_bwd<E, V, G, false>(a, s) : run_walk<E, V, G, false>(a, s);
}
template <typename E, int V, bool BWD>
hipError_t run_v(const RecurrenceArgs& a, hipStream_t s) {
  if (a.gate == GATE_LOG) return run_gate<E, V, BWD, GATE_LOG>(a, s);
  if (a.gate == GATE_SIGMOID) return run_gate<E, V, BWD, GATE_SIGMOID>(a, s);
  return run_gate<E, V, BWD, GATE_POWER>(a, s);
}
template <typename E, bool BWD>
hipError_t run(const RecurrenceArgs& a, hipStream_t s) {
  if constexpr (sizeof(E) == 2) {
    if (pairs<E>(a, BWD)) return run_v<E, 2, BWD>(a, s);
  }
  return run_v<E, 1, BWD>(a, s);
}

}  // namespace

size_t recurrence_part_bytes(int B, int D) { return (size_t)B * D * sizeof(float); }

template <typename E>
hipError_t launch_recurrence(const RecurrenceArgs& a, hipStream_t s) {
  return run<E, false>(a, s);
}
template <typename E>
hipError_t launch_recurrence_bwd(const RecurrenceArgs& a, hipStream_t s) {
  return run<E, true>(a, s);
}
template hipError_t launch_recurrence<bf16>(const RecurrenceArgs&, hipStream_t);
template hipError_t launch_recurrence<float>(const RecurrenceArgs&, hipStream_t);
template hipError_t launch_recurrence_bwd<bf16>(const RecurrenceArgs&, hipStream_t);
template hipError_t launch_recurrence_bwd<float>(const RecurrenceArgs&, hipStream_t);

}  // namespace prism
