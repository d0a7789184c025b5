// Layer norm over the last dimension with the residual sum in front, and its
// backward pass.  For a row of D values
//   s = x + residual,  m = mean(s) (0 by root mean square),
//   r = (mean((s - m)^2) + eps)^(-1/2),  u = (s - m) r,  y = u w + b,
// and, from the row x that was normalised, with g = dy w,
//   dx = r (g - mean(g) - u mean(g u)) + dh   (mean(g) only with the mean),
//   dw = sum over rows of dy u,  db = sum over rows of dy.
//
// Memory bound: every row is read once and written once.  A row stays in the
// registers of a group of lanes, of a wave, or of a workgroup of up to 16
// waves, so that mean and deviation are two sums one after the other over
// exact values (the sum of squares less the squared mean would lose the
// deviation of rows far from zero).  The backward pass reads no statistics: it
// forms them again from the row that it holds anyway.
#include "block_ops.h"
#include "vec_io.h"

namespace prism {

namespace {

// Sums over the team of a row: G lanes of a wave (G <= 64), or all waves of the
// workgroup (G > 64) through LDS, in a fixed order.  `turn` counts the sums: two
// rows of LDS in turn, so that a wave that is ahead writes where nobody reads.
template <int N>
__device__ inline void team_sums(float (&v)[N], int G, float (*sm)[16][2], int& turn) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = G >= 64 ? wave_sum(v[n]) : group_sum(v[n], G);
  if (G <= 64) return;
  const int wave = threadIdx.x / WAVE, nw = G / WAVE;
  float(*s)[2] = sm[turn & 1];
  ++turn;
  if ((threadIdx.x & (WAVE - 1)) == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) s[wave][n] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = 0.f;
  for (int k = 0; k < nw; ++k) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += s[k][n];
  }
}

__device__ inline long row_at(const Strides& s, long row, int T, int H) {
  if (T == 1 && H == 1) return row * s.b;
  const int r = (int)row, bt = r / H, h = r - bt * H, b = bt / T, t = bt - b * T;
  return b * s.b + t * s.t + h * s.h;
}

// Lane `lane` of the team holds vectors lane + j G, j < NV, of V values.
template <typename E, int V, int NV>
__global__ __launch_bounds__(1024) void layer_norm_kernel(const LayerNormArgs a, int G) {
  typedef VecIo<E, V> IO;
  typedef typename IO::raw raw;
  __shared__ float sm[2][16][2];
  int turn = 0;
  const int lane = threadIdx.x & (G - 1), teams = blockDim.x / G;
  const float inv = 1.f / (float)a.D;
  int at[NV];
  bool on[NV];
  raw rw[NV], rb[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (lane + j * G) * V;
    on[j] = c < a.D;
    at[j] = on[j] ? c : 0;
    if (a.w) rw[j] = *reinterpret_cast<const raw*>(static_cast<const E*>(a.w) + at[j]);
    if (a.b) rb[j] = *reinterpret_cast<const raw*>(static_cast<const E*>(a.b) + at[j]);
  }
  // (every team of the workgroup makes every round: the sums have barriers)
  for (long base = (long)blockIdx.x * teams; base < a.rows; base += (long)gridDim.x * teams) {
    const long want = base + threadIdx.x / G;
    const bool live = want < a.rows;
    const long row = live ? want : a.rows - 1;
    const E* x = static_cast<const E*>(a.x) + row_at(a.sx, row, a.T, a.H);
    float s[NV][V];
    float sum[1] = {0.f};
    raw rx[NV], rr[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) rx[j] = *reinterpret_cast<const raw*>(x + at[j]);
    if (a.r) {
      const E* r = static_cast<const E*>(a.r) + row_at(a.sr, row, a.T, a.H);
#pragma unroll
      for (int j = 0; j < NV; ++j) rr[j] = *reinterpret_cast<const raw*>(r + at[j]);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      IO::unpack(rx[j], s[j]);
      if (a.r) {
        float q[V];
        IO::unpack(rr[j], q);
#pragma unroll
        for (int i = 0; i < V; ++i) s[j][i] += q[i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) sum[0] += on[j] ? s[j][i] : 0.f;
    }
    if (a.h && live) {
      E* h = static_cast<E*>(a.h) + row_at(a.sh, row, a.T, a.H);
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on[j]) *reinterpret_cast<raw*>(h + at[j]) = IO::pack(s[j]);
    }
    float m = 0.f;
    if (a.center) {
      team_sums<1>(sum, G, sm, turn);
      m = sum[0] * inv;
    }
    float sq[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[j][i] -= m;
        sq[0] += on[j] ? s[j][i] * s[j][i] : 0.f;
      }
    team_sums<1>(sq, G, sm, turn);
    const float r = rsqrtf(fmaf(sq[0], inv, a.eps));
    if (!live) continue;
    E* y = static_cast<E*>(a.y) + row_at(a.sy, row, a.T, a.H);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[V], b[V];
      if (a.w) IO::unpack(rw[j], w);
      if (a.b) IO::unpack(rb[j], b);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v = s[j][i] * r;
        if (a.w) v *= w[i];
        if (a.b) v += b[i];
        s[j][i] = v;
      }
      if (on[j]) *reinterpret_cast<raw*>(y + at[j]) = IO::pack(s[j]);
    }
  }
}

// A workgroup's rows are summed for the weights in registers, then over its
// teams (in the wave, then over the waves through LDS), and written as one
// partial [2][D] for each workgroup.
template <typename E, int V, int NV>
__global__ __launch_bounds__(1024) void layer_norm_bwd_kernel(const LayerNormArgs a, int G) {
  typedef VecIo<E, V> IO;
  typedef typename IO::raw raw;
  __shared__ float sm[2][16][2];
  __shared__ float cols[NV * V * WAVE];
  int turn = 0;
  const int lane = threadIdx.x & (G - 1), teams = blockDim.x / G;
  const float inv = 1.f / (float)a.D;
  int at[NV];
  bool on[NV];
  raw rw[NV];
  float dw[NV][V], db[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (lane + j * G) * V;
    on[j] = c < a.D;
    at[j] = on[j] ? c : 0;
    if (a.w) rw[j] = *reinterpret_cast<const raw*>(static_cast<const E*>(a.w) + at[j]);
#pragma unroll
    for (int i = 0; i < V; ++i) dw[j][i] = db[j][i] = 0.f;
  }
  for (long base = (long)blockIdx.x * teams; base < a.rows; base += (long)gridDim.x * teams) {
    const long want = base + threadIdx.x / G;
    const bool live = want < a.rows;
    const long row = live ? want : a.rows - 1;
    const E* x = static_cast<const E*>(a.x) + row_at(a.sx, row, a.T, a.H);
    const E* dy = static_cast<const E*>(a.dy) + row_at(a.sy, row, a.T, a.H);
    raw rx[NV], rg[NV], rh[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) rx[j] = *reinterpret_cast<const raw*>(x + at[j]);
#pragma unroll
    for (int j = 0; j < NV; ++j) rg[j] = *reinterpret_cast<const raw*>(dy + at[j]);
    if (a.dh) {
      const E* dh = static_cast<const E*>(a.dh) + row_at(a.sr, row, a.T, a.H);
#pragma unroll
      for (int j = 0; j < NV; ++j) rh[j] = *reinterpret_cast<const raw*>(dh + at[j]);
    }
    float u[NV][V], g[NV][V];
    float one[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      IO::unpack(rx[j], u[j]);
      IO::unpack(rg[j], g[j]);
      float w[V];
      if (a.w) IO::unpack(rw[j], w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        one[0] += on[j] ? u[j][i] : 0.f;
        one[1] += on[j] ? (a.w ? g[j][i] * w[i] : g[j][i]) : 0.f;
      }
    }
    float m = 0.f, mg = 0.f;
    if (a.center) {
      team_sums<2>(one, G, sm, turn);
      m = one[0] * inv;
      mg = one[1] * inv;
    }
    float two[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[V];
      if (a.w) IO::unpack(rw[j], w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        u[j][i] -= m;
        const float q = a.w ? g[j][i] * w[i] : g[j][i];
        two[0] += on[j] ? u[j][i] * u[j][i] : 0.f;
        two[1] += on[j] ? u[j][i] * q : 0.f;
      }
    }
    team_sums<2>(two, G, sm, turn);
    const float r = rsqrtf(fmaf(two[0], inv, a.eps));
    const float mu = two[1] * inv * r;   // mean of g u
    if (!live) continue;
    E* dx = static_cast<E*>(a.dx) + row_at(a.sh, row, a.T, a.H);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[V], v[V];
      if (a.w) IO::unpack(rw[j], w);
      if (a.dh) IO::unpack(rh[j], v);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float un = u[j][i] * r;
        const float q = a.w ? g[j][i] * w[i] : g[j][i];
        const float d = r * (q - mg - un * mu);
        v[i] = a.dh ? d + v[i] : d;
        dw[j][i] = fmaf(g[j][i], un, dw[j][i]);
        db[j][i] += g[j][i];
      }
      if (on[j]) *reinterpret_cast<raw*>(dx + at[j]) = IO::pack(v);
    }
  }
  if (!a.part) return;
  float* out = a.part + (long)blockIdx.x * 2 * a.D;
  for (int k = 0; k < 2; ++k) {
    float(&d)[NV][V] = k ? db : dw;
    for (int mask = G; mask < WAVE; mask <<= 1) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) d[j][i] += __shfl_xor(d[j][i], mask);
    }
    if (G < (int)blockDim.x) {   // the waves one after the other
      const int wave = threadIdx.x / WAVE, nw = blockDim.x / WAVE;
      for (int w = 0; w < nw; ++w) {
        __syncthreads();
        if (wave == w && (int)(threadIdx.x & (WAVE - 1)) < G) {
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
              float& c = cols[(j * V + i) * WAVE + lane];
              d[j][i] += w ? c : 0.f;
              c = d[j][i];
            }
        }
      }
      if (wave != nw - 1) continue;
    }
    if ((int)(threadIdx.x & (WAVE - 1)) < G || G > WAVE) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (on[j]) out[(long)k * a.D + at[j] + i] = d[j][i];
    }
  }
}

int pow2_at_least(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

// Dimensions whose steps follow from one another in every tensor are taken as
// one, which leaves rows of one step (T = H = 1) in most calls.
void merge_rows(LayerNormArgs& a, bool bwd) {
  if (a.rows == 0) return;
  Strides* const all[4] = {&a.sx, &a.sy, a.r || a.dh ? &a.sr : nullptr, bwd || a.h ? &a.sh : nullptr};
  long n[3] = {a.rows / ((long)a.T * a.H), a.T, a.H}, step[4][3] = {};
  for (int k = 0; k < 4; ++k)
    if (all[k]) {
      step[k][0] = all[k]->b;
      step[k][1] = all[k]->t;
      step[k][2] = all[k]->h;
    }
  for (int o = 1; o >= 0; --o) {   // dimension o with the one inside it
    bool one = true;
    for (int k = 0; k < 4; ++k) one = one && (n[o + 1] == 1 || n[o] == 1 || step[k][o] == step[k][o + 1] * n[o + 1]);
    if (!one) continue;
    for (int k = 0; k < 4; ++k)
      if (n[o + 1] > 1) step[k][o] = step[k][o + 1];
    n[o] *= n[o + 1];
    for (int i = o + 1; i < 2; ++i) {   // those inside move out by one
      n[i] = n[i + 1];
      for (int k = 0; k < 4; ++k) step[k][i] = step[k][i + 1];
    }
    n[2] = 1;
    for (int k = 0; k < 4; ++k) step[k][2] = 0;
  }
  a.T = (int)n[1];
  a.H = (int)n[2];
  for (int k = 0; k < 4; ++k)
    if (all[k]) *all[k] = Strides{step[k][0], step[k][1], step[k][2]};
}

// Vectors of 16 bytes where every row starts at a multiple of them and has a
// whole number of them, else single values.
bool aligned(const LayerNormArgs& a, bool bwd, int V, int size) {
  long m = a.D | a.sx.b | a.sx.t | a.sx.h | a.sy.b | a.sy.t | a.sy.h;
  uintptr_t p = (uintptr_t)a.x | (uintptr_t)a.w | (uintptr_t)a.b;
  if (a.r || a.dh) m |= a.sr.b | a.sr.t | a.sr.h;
  if (bwd || a.h) m |= a.sh.b | a.sh.t | a.sh.h;
  p |= (uintptr_t)a.r | (uintptr_t)a.y | (uintptr_t)a.h | (uintptr_t)a.dy | (uintptr_t)a.dh | (uintptr_t)a.dx;
  return m % V == 0 && p % (V * size) == 0;
}

struct Shape {
  int G, NV, block;
};
// Lanes, vectors a lane and workgroup for rows of n vectors, `most` vectors a
// lane at most.
Shape shape_of(int n, int most) {
  Shape s;
  if (n <= WAVE) {
    s.G = pow2_at_least(n);
    s.NV = 1;
    s.block = 256;
    return s;
  }
  s.NV = pow2_at_least((n + WAVE - 1) / WAVE);
  s.G = WAVE;
  while (s.NV > most) {
    s.NV /= 2;
    s.G *= 2;
  }
  s.block = s.G > WAVE ? s.G : 256;
  return s;
}

constexpr int LN_PARTS = 512;   // workgroups of the backward kernel with weights, at most

template <typename E, int V, int NV>
hipError_t run_fwd(const LayerNormArgs& a, const Shape& p, hipStream_t s) {
  const long teams = p.block / p.G;
  long grid = (a.rows + teams - 1) / teams;
  if (grid > 4096) grid = 4096;
  hipLaunchKernelGGL((layer_norm_kernel<E, V, NV>), dim3((unsigned)grid), dim3(p.block), 0, s, a, p.G);
  return hipGetLastError();
}
template <typename E, int V, int NV>
hipError_t run_bwd(const LayerNormArgs& a, const Shape& p, hipStream_t s) {
  const long teams = p.block / p.G;
  long grid = (a.rows + teams - 1) / teams;
  if (grid > LN_PARTS) grid = LN_PARTS;
  if (grid > 0) {
    hipLaunchKernelGGL((layer_norm_bwd_kernel<E, V, NV>), dim3((unsigned)grid), dim3(p.block), 0, s, a, p.G);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.dw) {
    const hipError_t e = launch_column_sums(a.part, (int)grid, 2L * a.D, a.D, 0, a.dw, s);
    if (e != hipSuccess) return e;
  }
  if (a.db) return launch_column_sums(a.part + a.D, (int)grid, 2L * a.D, a.D, 0, a.db, s);
  return hipSuccess;
}

}  // namespace

size_t layer_norm_part_bytes(int D) { return (size_t)LN_PARTS * 2 * D * sizeof(float); }

template <typename E>
hipError_t launch_layer_norm(const LayerNormArgs& in, hipStream_t s) {
  LayerNormArgs a = in;
  merge_rows(a, false);
  constexpr int V = 16 / sizeof(E);
  if (aligned(a, false, V, sizeof(E))) {
    const Shape p = shape_of((a.D + V - 1) / V, 32 / V);
    if (p.NV == 1) return run_fwd<E, V, 1>(a, p, s);
    if (p.NV == 2) return run_fwd<E, V, 2>(a, p, s);
    if (p.NV == 4) return run_fwd<E, V, 4>(a, p, s);
    return run_fwd<E, V, 32 / V>(a, p, s);
  }
  const Shape p = shape_of(a.D, 16);
  if (p.NV == 1) return run_fwd<E, 1, 1>(a, p, s);
  if (p.NV <= 4) return run_fwd<E, 1, 4>(a, p, s);
  return run_fwd<E, 1, 16>(a, p, s);
}

template <typename E>
hipError_t launch_layer_norm_bwd(const LayerNormArgs& in, hipStream_t s) {
  LayerNormArgs a = in;
  merge_rows(a, true);
  constexpr int V = 16 / sizeof(E);
  if (aligned(a, true, V, sizeof(E))) {
    const Shape p = shape_of((a.D + V - 1) / V, 16 / V);
    if (p.NV == 1) return run_bwd<E, V, 1>(a, p, s);
    if (p.NV == 2) return run_bwd<E, V, 2>(a, p, s);
    return run_bwd<E, V, 16 / V>(a, p, s);
  }
  const Shape p = shape_of(a.D, 16);
  if (p.NV == 1) return run_bwd<E, 1, 1>(a, p, s);
  if (p.NV <= 4) return run_bwd<E, 1, 4>(a, p, s);
  return run_bwd<E, 1, 16>(a, p, s);
}

template hipError_t launch_layer_norm<bf16>(const LayerNormArgs&, hipStream_t);
template hipError_t launch_layer_norm<float>(const LayerNormArgs&, hipStream_t);
template hipError_t launch_layer_norm_bwd<bf16>(const LayerNormArgs&, hipStream_t);
template hipError_t launch_layer_norm_bwd<float>(const LayerNormArgs&, hipStream_t);

}  // namespace prism
