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
// waves (but for 8 to 9 of 128 registers a lane in bf16, with dh, and 5 to 23 in
// fp32, which the backward pass of more than 8192 values spills), so that mean and deviation are two sums one after the other over the
// values themselves (the sum of squares less the squared mean would lose the
// deviation of rows far from zero).  The backward pass reads no statistics: it
// forms them again from the row that it holds anyway.
//
// bf16, 2048 channels: 8 x 2048 rows with a residual and the sum 48 us, 5.6 TB/s,
// without 26 us, 5.1 TB/s; backward, 16384 rows with dh 56 us with the sums of
// partials (4), 4.8 TB/s.  What is left there: a row's two sums wait for its waves,
// and registers for 16 values of three rows and of dw and db leave 2 waves a SIMD to
// hide that.  fp32, 8192 rows of 2048 with dh: backward 52 us, 5.2 TB/s.
//
// Errors of fp32 results against 64 bits (2-norms): y 5e-8 to 6e-8 and dx 6e-8 to 7e-8,
// as elementary operations in fp32 have them; dw and db, where a lane adds a
// workgroup's rows one after the other, 1.4e-7 to 1.7e-7 (elementary sums: 0.9e-7 of
// 4995 rows of 48, 1.5e-7 and 1.9e-7 of 4096 and 16384 rows of 2048 and 1000).
#include "block_ops.h"
#include "vec_io.h"

namespace prism {

namespace {

// Sums over the team of a row: G lanes of a wave (G <= 64), or G / 64 waves of
// the workgroup through LDS, in a fixed order.  `turn` counts the sums: two rows
// of LDS in turn, so that a wave that is ahead writes where nobody reads.
template <int N>
__device__ inline void team_sums(float (&v)[N], int G, float (*sm)[16][2], int& turn) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = G >= WAVE ? wave_sum(v[n]) : group_sum(v[n], G);
  if (G <= WAVE) return;
  const int wave = threadIdx.x / WAVE, nw = G / WAVE, first = wave & -nw;
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
    for (int n = 0; n < N; ++n) v[n] += s[first + k][n];
  }
}

// A vector of ones or zeros in the place of weights that are not given.
template <typename E, int V>
__device__ inline typename VecIo<E, V>::raw weight(const void* p, int at, float other) {
  if (p) return load_vec<E, V>(static_cast<const E*>(p) + at);
  float x[V];
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = other;
  return VecIo<E, V>::pack(x);
}

__device__ inline long row_at(const Strides& s, long row, int T, int H) {
  if (T == 1 && H == 1) return row * s.b;
  const int r = (int)row, bt = r / H, h = r - bt * H, b = bt / T, t = bt - b * T;
  return b * s.b + t * s.t + h * s.h;
}

// Lane `lane` of the team holds vectors lane + j G, j < NV, of V values; 8 waves a
// SIMD hide the loads (the next row on its way as well gained nothing).
// ODD: the row's last vector is no whole one, and begins before its place.
template <typename E, int V, int NV, int NT, bool ODD, bool RES>
__global__ __launch_bounds__(NT) void layer_norm_kernel(const LayerNormArgs a, int G) {
  typedef VecIo<E, V> IO;
  typedef typename IO::raw raw;
  __shared__ float sm[2][16][2];
  int turn = 0;
  const int lane = threadIdx.x & (G - 1), teams = blockDim.x / G;
  const float inv = 1.f / (float)a.D;
  int at[NV], skip[NV];   // values at + skip .. at + V - 1 are the lane's (skip = V: none)
  raw rw[NV], rb[NV], rx[NV], rr[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (lane + j * G) * V;
    at[j] = c >= a.D ? 0 : ODD ? min(c, a.D - V) : c;
    skip[j] = c >= a.D ? V : ODD ? c - at[j] : 0;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    rw[j] = weight<E, V>(a.w, at[j], 1.f);
    rb[j] = weight<E, V>(a.b, at[j], 0.f);
  }
  auto mine = [&](int j, int i) { return ODD ? i >= skip[j] : skip[j] == 0; };
  // (every team of the workgroup makes every round: the sums have barriers)
  for (long base = (long)blockIdx.x * teams; base < a.rows; base += (long)gridDim.x * teams) {
    const long want = base + threadIdx.x / G;
    const bool live = want < a.rows;
    const long row = live ? want : a.rows - 1;
    const E* x = static_cast<const E*>(a.x) + row_at(a.sx, row, a.T, a.H);
#pragma unroll
    for (int j = 0; j < NV; ++j) rx[j] = load_vec<E, V>(x + at[j]);
    if (RES) {
      const E* r = static_cast<const E*>(a.r) + row_at(a.sr, row, a.T, a.H);
#pragma unroll
      for (int j = 0; j < NV; ++j) rr[j] = load_vec<E, V>(r + at[j]);
    }
    float s[NV][V];
    float sum[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      IO::unpack(rx[j], s[j]);
      if (RES) {
        float q[V];
        IO::unpack(rr[j], q);
#pragma unroll
        for (int i = 0; i < V; ++i) s[j][i] += q[i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) sum[0] += mine(j, i) ? s[j][i] : 0.f;
    }
    if (RES && a.h && live) {
      E* h = static_cast<E*>(a.h) + row_at(a.sh, row, a.T, a.H);
#pragma unroll
      for (int j = 0; j < NV; ++j)
        store_vec<E, V>(h + at[j], s[j], skip[j]);
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
        sq[0] += mine(j, i) ? s[j][i] * s[j][i] : 0.f;
      }
    team_sums<1>(sq, G, sm, turn);
    const float r = rsqrtf(fmaf(sq[0], inv, a.eps));
    if (!live) continue;
    E* y = static_cast<E*>(a.y) + row_at(a.sy, row, a.T, a.H);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[V], b[V];
      IO::unpack(rw[j], w);
      IO::unpack(rb[j], b);
#pragma unroll
      for (int i = 0; i < V; ++i) s[j][i] = fmaf(s[j][i] * r, w[i], b[i]);
      store_vec<E, V>(y + at[j], s[j], skip[j]);
    }
  }
}

// A workgroup's rows are summed for the weights in registers, then over its
// teams (in the wave, then over the waves through LDS), and written as one
// partial [2][D] for each workgroup.  The next row of a team is on its way while
// the sums of one are joined (16384 rows of 2048 with dh: 56 us; without, 67).
template <typename E, int V, int NV, int NT, bool ODD, bool DH>
__global__ __launch_bounds__(NT) void layer_norm_bwd_kernel(const LayerNormArgs a, int G) {
  typedef VecIo<E, V> IO;
  typedef typename IO::raw raw;
  constexpr bool PF = NT < 1024;   // (1024 threads have no registers for it)
  __shared__ float sm[2][16][2];
  __shared__ float cols[2 * NV * V * (NT < 1024 ? NT / 2 : 1)];   // (of two teams or more; 1024 threads are one)
  int turn = 0;
  const int lane = threadIdx.x & (G - 1), teams = blockDim.x / G;
  const float inv = 1.f / (float)a.D;
  int at[NV], skip[NV];   // values at + skip .. at + V - 1 are the lane's (skip = V: none)
  raw rw[NV], rx[NV], rg[NV], rh[NV];
  float dw[NV][V], db[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (lane + j * G) * V;
    at[j] = c >= a.D ? 0 : ODD ? min(c, a.D - V) : c;
    skip[j] = c >= a.D ? V : ODD ? c - at[j] : 0;
#pragma unroll
    for (int i = 0; i < V; ++i) dw[j][i] = db[j][i] = 0.f;
  }
  auto mine = [&](int j, int i) { return ODD ? i >= skip[j] : skip[j] == 0; };
  auto load = [&](long want) {
    const long row = want < a.rows ? want : a.rows - 1;
    const E* x = static_cast<const E*>(a.x) + row_at(a.sx, row, a.T, a.H);
    const E* dy = static_cast<const E*>(a.dy) + row_at(a.sy, row, a.T, a.H);
#pragma unroll
    for (int j = 0; j < NV; ++j) rx[j] = load_vec<E, V>(x + at[j]);
#pragma unroll
    for (int j = 0; j < NV; ++j) rg[j] = load_vec<E, V>(dy + at[j]);
  };
  const long step = (long)gridDim.x * teams;
  long base = (long)blockIdx.x * teams;
  if (PF) load(base + threadIdx.x / G);
#pragma unroll
  for (int j = 0; j < NV; ++j) rw[j] = weight<E, V>(a.w, at[j], 1.f);
  for (; base < a.rows; base += step) {
    const long row = base + threadIdx.x / G;
    const bool live = row < a.rows;
    if (!PF) load(row);
    if (DH) {
      const E* dh = static_cast<const E*>(a.dh) + row_at(a.sr, live ? row : a.rows - 1, a.T, a.H);
#pragma unroll
      for (int j = 0; j < NV; ++j) rh[j] = load_vec<E, V>(dh + at[j]);
    }
    float u[NV][V], g[NV][V];
    float one[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      IO::unpack(rx[j], u[j]);
      IO::unpack(rg[j], g[j]);
      float w[V];
      IO::unpack(rw[j], w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        one[0] += mine(j, i) ? u[j][i] : 0.f;
        one[1] += mine(j, i) ? g[j][i] * w[i] : 0.f;
      }
    }
    if (PF && base + step < a.rows) load(row + step);
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
      IO::unpack(rw[j], w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        u[j][i] -= m;
        two[0] += mine(j, i) ? u[j][i] * u[j][i] : 0.f;
        two[1] += mine(j, i) ? u[j][i] * (g[j][i] * w[i]) : 0.f;
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
      IO::unpack(rw[j], w);
      if (DH) IO::unpack(rh[j], v);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float un = u[j][i] * r;
        const float d = r * (fmaf(g[j][i], w[i], -mg) - un * mu);
        v[i] = DH ? d + v[i] : d;
        dw[j][i] = fmaf(g[j][i], un, dw[j][i]);
        db[j][i] += g[j][i];
      }
      store_vec<E, V>(dx + at[j], v, skip[j]);
    }
  }
  if (!a.part) return;
  float* out = a.part + (long)blockIdx.x * 2 * a.D;
  auto each = [&](auto f) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) f(dw[j][i], j, i, 0), f(db[j][i], j, i, 1);
  };
  for (int mask = G; mask < WAVE; mask <<= 1) each([&](float& d, int, int, int) { d += __shfl_xor(d, mask); });
  // the teams, or, where a wave has several, the waves, one after the other
  const int per = G > WAVE ? G : WAVE, part = threadIdx.x / per, n = blockDim.x / per;
  for (int w = 0; w < n; ++w) {
    if (w) __syncthreads();
    if (part == w)
      each([&](float& d, int j, int i, int k) {
        float& c = cols[((j * V + i) * 2 + k) * per + lane];
        if (w) d += c;
        if (w < n - 1) c = d;
      });
  }
  if (part != n - 1 || (G < WAVE && (int)(threadIdx.x & (WAVE - 1)) >= G)) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (skip[j] == V) continue;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!ODD || i >= skip[j]) out[at[j] + i] = dw[j][i];
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!ODD || i >= skip[j]) out[a.D + at[j] + i] = db[j][i];
  }
}

// Dimensions whose steps follow from one another in every tensor are taken as
// one, which leaves rows of one step (T = H = 1) in most calls, without divisions
// (8 x 2048 rows of 2048 48 us in place of 54; 16 times as many of 128 27 for 32).
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

struct Shape {
  int G, NV, block;
};
// Lanes, vectors a lane and threads a workgroup for rows of n vectors, `most`
// vectors a lane unless a row needs more than 1024 lanes of them.
Shape shape_of(int n, int most, int block) {
  Shape s;
  s.NV = 1;
  s.G = 1;
  while (s.G < WAVE && s.G < n) s.G *= 2;
  while (s.G * s.NV < n) {
    if (s.NV < most || s.G == 1024)
      s.NV *= 2;
    else
      s.G *= 2;
  }
  s.block = s.G > block ? s.G : block;
  return s;
}

// Values a lane, forward: 16, for fewer waves that a row's sums wait for (bf16 rows
// of 2048 without a residual, 8 x 2048 of them, 26 us in place of 31 with 8; 2048 of
// 8192 14 in place of 17.5, with a residual 26 in place of 33), or 8, for more of them
// on a SIMD, where a lane would hold twice the bytes and a row has few waves anyway
// (bf16 with a residual below 4096, fp32 below 8192 values: 8 x 2048 rows of 2048 with
// a residual 48 us, with 16 values 49.5; fp32 4096 rows of 2048 23.7 and 24.9).
// Backward, where the weights' sums want few workgroups with many rows each, 16 (56 us,
// 8 values 62 for 16384 rows of 2048, with 256 workgroups of 512 threads).
constexpr int LN_LANE = 8, LN_LANE_WIDE = 16, LN_LANE_BWD = 16;
template <typename E>
int lane_of(const LayerNormArgs& a, bool bwd) {
  if (bwd) return LN_LANE_BWD;
  return a.D >= 8192 || (sizeof(E) == 2 && (!a.r || a.D >= 4096)) ? LN_LANE_WIDE : LN_LANE;
}
// Workgroups of the backward kernel, at most: one a CU, of 512 threads, where their
// partials are wide (16384 rows of 2048: 56 us; two of 256 threads 58, 1024 rows of
// 4096 18 and 21), two of 256 threads from 1024 channels (16384 rows of 1536 43 us; one
// of 512 threads 47), four where rows are short and a wave has few bytes on their way
// (65536 rows of 256: with 512 workgroups 35 us, 1024 28, 2048 34).
int parts_of(int D) { return D >= 2048 ? 256 : D >= 1024 ? 512 : 1024; }

template <typename E, int V, int NV, int NT, bool ODD>
hipError_t run_fwd(const LayerNormArgs& a, const Shape& p, hipStream_t s) {
  const long teams = p.block / p.G;
  long grid = (a.rows + teams - 1) / teams;
  if (grid > (1 << 20)) grid = 1 << 20;
  if (a.r)
    hipLaunchKernelGGL((layer_norm_kernel<E, V, NV, NT, ODD, true>), dim3((unsigned)grid), dim3(p.block), 0, s, a, p.G);
  else
    hipLaunchKernelGGL((layer_norm_kernel<E, V, NV, NT, ODD, false>), dim3((unsigned)grid), dim3(p.block), 0, s, a, p.G);
  return hipGetLastError();
}
template <typename E, int V, int NV, int NT, bool ODD>
hipError_t run_bwd(const LayerNormArgs& a, const Shape& p, hipStream_t s) {
  const long teams = p.block / p.G;
  long grid = (a.rows + teams - 1) / teams;
  // (two rows a team before there are more than one a CU: 4096 rows of 512 11.4 us in
  // place of 13.5, of 1024 19 in place of 28)
  if (grid > 256) grid = grid > 512 ? grid / 2 : 256;
  if (grid > parts_of(a.D)) grid = parts_of(a.D);
  if (grid > 0) {
    const dim3 blocks((unsigned)grid), threads(p.block);
    if (a.dh)
      hipLaunchKernelGGL((layer_norm_bwd_kernel<E, V, NV, NT, ODD, true>), blocks, threads, 0, s, a, p.G);
    else
      hipLaunchKernelGGL((layer_norm_bwd_kernel<E, V, NV, NT, ODD, false>), blocks, threads, 0, s, a, p.G);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.part) return launch_column_sums(a.part, (int)grid, a.D, 1, a.dw, a.db, s);
  return hipSuccess;
}

// (a row of more than a wave has as many vectors a lane as a lane may have, or, of
// more than 1024 lanes, more)
template <typename E, int V, int NV, bool ODD, bool BWD>
hipError_t run_nv(const LayerNormArgs& a, const Shape& p, hipStream_t s) {
  constexpr int least = BWD ? LN_LANE_BWD : LN_LANE, most = BWD ? LN_LANE_BWD : LN_LANE_WIDE;
  if constexpr (NV * V >= least) {
    if constexpr (BWD) {
      if (p.block > 512) return run_bwd<E, V, NV, 1024, ODD>(a, p, s);
      if (p.block > 256) return run_bwd<E, V, NV, 512, ODD>(a, p, s);
    } else {
      if (p.block > 256) return run_fwd<E, V, NV, 1024, ODD>(a, p, s);
    }
  }
  if constexpr (NV * V <= most) {
    if constexpr (BWD) return run_bwd<E, V, NV, 256, ODD>(a, p, s);
    return run_fwd<E, V, NV, 256, ODD>(a, p, s);
  }
  return hipErrorInvalidValue;
}
// (16384 values are at most 16 for each of 1024 lanes)
template <typename E, int V, bool ODD, bool BWD>
hipError_t run_v(const LayerNormArgs& a, hipStream_t s) {
  Shape p = shape_of((a.D + V - 1) / V, lane_of<E>(a, BWD) / V, 256);
  // (backward, workgroups of 512 threads for wide rows, where these leave more than two
  // rows a team: 4096 rows of 2048 21 us in place of 22, 16384 56 in place of 70)
  if (BWD && a.D >= 2048 && p.block == 256 && a.rows > 512L * (256 / p.G)) p.block = 512;
  if (p.NV == 1) return run_nv<E, V, 1, ODD, BWD>(a, p, s);
  if constexpr (V > 1) {
    if (p.NV == 2) return run_nv<E, V, 2, ODD, BWD>(a, p, s);
  }
  if constexpr (V == 4) {
    if (p.NV == 4) return run_nv<E, V, 4, ODD, BWD>(a, p, s);
  }
  return hipErrorInvalidValue;
}
// Vectors of 16 bytes, or single values of rows narrower than that (8 x 2048 rows of
// 2048 in bf16 48 us by vectors, 86 by values, backward 56 and 95; 16384 rows of 1001
// 14 and 27, backward 38 and 47).
template <typename E, bool BWD>
hipError_t run(LayerNormArgs a, hipStream_t s) {
  merge_rows(a, BWD);
  constexpr int V = 16 / sizeof(E);
  if (a.D % V == 0) return run_v<E, V, false, BWD>(a, s);
  return a.D > V ? run_v<E, V, true, BWD>(a, s) : run_v<E, 1, false, BWD>(a, s);
}

}  // namespace

size_t layer_norm_part_bytes(int D) { return (size_t)parts_of(D) * 2 * D * sizeof(float); }

template <typename E>
hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t s) {
  return run<E, false>(a, s);
}
template <typename E>
hipError_t launch_layer_norm_bwd(const LayerNormArgs& a, hipStream_t s) {
  return run<E, true>(a, s);
}
template hipError_t launch_layer_norm<bf16>(const LayerNormArgs&, hipStream_t);
template hipError_t launch_layer_norm<float>(const LayerNormArgs&, hipStream_t);
template hipError_t launch_layer_norm_bwd<bf16>(const LayerNormArgs&, hipStream_t);
template hipError_t launch_layer_norm_bwd<float>(const LayerNormArgs&, hipStream_t);

}  // namespace prism
