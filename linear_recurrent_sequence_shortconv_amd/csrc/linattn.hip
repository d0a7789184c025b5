// Linear attention with a decay for each head: the kernels beside the chunk
// passes (linattn_kernel.h): joining of segment states, the decay gradient,
// sums over heads that share keys and values, and the recurrent step.
#include <type_traits>

#include "operators.h"
#include "prism_common.h"

namespace prism {


namespace {

// ------------------------------------------------------------ segment join
// One thread carries one element of the state over the segments:
// forward X_{s+1} = decay_s X_s + own_s, reverse the other way round.  The
// last segment of a pass has no own state (nothing enters after it).
__global__ __launch_bounds__(256) void la_join_kernel(const LaJoin a) {
  const int per = (a.DD + 255) / 256;
  int id = blockIdx.x;
  const int blk = id % per;
  id /= per;
  const int dir = id % 2, bh = id / 2;
  if (!a.seg[dir]) return;
  const int e = blk * 256 + threadIdx.x;
  if (e >= a.DD) return;
  const int n = seq_len(a.cu, bh / a.H, a.T);
  const int used = max(1, (n + a.seglen - 1) / a.seglen);
  float* seg = a.seg[dir] + (long)bh * a.nseg * a.DD + e;
  const float* dec = a.dec[dir] + (long)bh * a.nseg;
  float x = a.X0[dir] ? a.X0[dir][(long)bh * a.DD + e] : 0.f;
  for (int i = 0; i < used - 1; ++i) {
    const int s = dir ? used - 1 - i : i;
    const float own = seg[(long)s * a.DD];
    seg[(long)s * a.DD] = x;
    x = fmaf(dec[s], x, own);
  }
  seg[(long)(dir ? 0 : used - 1) * a.DD] = x;
}

// ---------------------------------------------------------- decay gradient
// One workgroup a segment: <dS, S> at its end, then the suffix sums of
// q.dq - k.dk (in fp64: differences of long sums), 256 tokens at a time from
// the end.
__global__ __launch_bounds__(256) void la_decay_kernel(const LaDecay a) {
  __shared__ double sm[256];
  const int tid = threadIdx.x;
  const int seg = blockIdx.x % a.nseg, bh = blockIdx.x / a.nseg;
  const int b = bh / a.H, h = bh % a.H;
  const int n = seq_len(a.cu, b, a.T);
  const int s0 = seg * a.seglen, len = min(n - s0, a.seglen);
  if (len <= 0) return;
  const bool last = s0 + len == n;
  const float* R = last ? (a.dST ? a.dST + (long)bh * a.DD : nullptr)
                        : a.segr + ((long)bh * a.nseg + seg) * a.DD;
  const float* X = last ? (a.dST ? a.ST + (long)bh * a.DD : nullptr)
                        : a.segf + ((long)bh * a.nseg + seg + 1) * a.DD;
  double s = 0.0;
  if (R)
    for (int e = tid; e < a.DD; e += 256) s += (double)R[e] * (double)X[e];
  sm[tid] = s;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (tid < o) sm[tid] += sm[tid + o];
    __syncthreads();
  }
  double carry = sm[0];
  __syncthreads();
  const long row0 = a.cu ? (long)a.cu[b] + s0 : s0;
  for (int hi = len; hi > 0; hi -= 256) {
    // thread tid holds token hi - 1 - tid; a prefix sum over the threads
    const int t = hi - 1 - tid;
    double x = 0.0;
    if (t >= 0) {
      for (int p = 0; p < LA_PARTS; ++p) x += (double)a.eq[((long)bh * LA_PARTS + p) * a.T + s0 + t];
      for (int p = 0; p < LA_PARTS; ++p) x -= (double)a.ek[((long)bh * LA_PARTS + p) * a.T + s0 + t];
    }
    sm[tid] = x;
    __syncthreads();
    for (int o = 1; o < 256; o <<= 1) {
      const double y = tid >= o ? sm[tid - o] : 0.0;
      __syncthreads();
      x += y;
      sm[tid] = x;
      __syncthreads();
    }
    if (t >= 0) {
      const long at = (a.cu ? 0 : b * a.sg.b) + (row0 + t) * a.sg.t + h * a.sg.h;
      const float d = a.g[at] < -104.f ? 0.f : (float)(carry + x);
      if (a.tmp)
        a.tmp[(long)bh * a.T + s0 + t] = d;
      else
        a.dg[at] = d;
    }
    carry += sm[255];
    __syncthreads();
  }
}

// One decay a head: the sum of its tokens' gradients over the batch.
__global__ __launch_bounds__(256) void la_decay_head_kernel(const LaDecay a) {
  __shared__ double sm[256];
  const int tid = threadIdx.x, h = blockIdx.x;
  double s = 0.0;
  for (int b = 0; b < a.B; ++b) {
    const int n = seq_len(a.cu, b, a.T);
    const float* x = a.tmp + ((long)b * a.H + h) * a.T;
    for (int t = tid; t < n; t += 256) s += (double)x[t];
  }
  sm[tid] = s;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (tid < o) sm[tid] += sm[tid + o];
    __syncthreads();
  }
  if (tid == 0) a.dg[h * a.sg.h] = (float)sm[0];
}

// ---------------------------------------------------------------- group sum
template <typename E>
__global__ __launch_bounds__(256) void la_group_kernel(const float* __restrict__ part, E* __restrict__ out,
                                                       long n4, int grp, int d4) {
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n4; i += (long)gridDim.x * 256) {
    const long row = i / d4;
    const int c = (int)(i - row * d4);
    const float* p = part + (row * grp * d4 + c) * 4;
    f32x4 s = *reinterpret_cast<const f32x4*>(p);
    for (int k = 1; k < grp; ++k) s += *reinterpret_cast<const f32x4*>(p + (long)k * d4 * 4);
    st_f4(out + i * 4, s);
  }
}

// ------------------------------------------------------------------- step
// S [dv][dk]: LK lanes hold a row (4 values each), RPT rows a thread; the rows
// stay in registers over the call's tokens, so S crosses memory once.
template <typename E, int LK, int RPT>
__global__ __launch_bounds__(256) void la_step_kernel(const LaStepArgs<E> a, int tiles) {
  constexpr int RW = 256 / LK;   // rows side by side in a workgroup
  const int tid = threadIdx.x, l = tid % LK, y = tid / LK;
  const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles;
  const int b = bh / a.H, h = bh % a.H, hk = h / a.grp;
  const int v0 = tile * RW * RPT + y;
  const bool on = 4 * l < a.dk;
  const int k0 = on ? 4 * l : 0;
  const float* Sp = a.S + (long)bh * a.dv * a.dk;
  f32x4 S[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int v = min(v0 + i * RW, a.dv - 1);
    S[i] = *reinterpret_cast<const f32x4*>(Sp + v * a.dk + k0);
  }
  for (int t = 0; t < a.T; ++t) {
    const E* qp = a.q + (b * a.sq.b + t * a.sq.t + h * a.sq.h) + k0;
    const E* kp = a.k + (b * a.sk.b + t * a.sk.t + hk * a.sk.h) + k0;
    const E* vp = a.v + (b * a.sv.b + t * a.sv.t + hk * a.sv.h);
    const f32x4 q = raw4_to_f(ld_raw4(qp)), k = raw4_to_f(ld_raw4(kp));
    const float e = __expf(a.g[b * a.sg.b + t * a.sg.t + h * a.sg.h]);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int v = v0 + i * RW;
      const float vv = to_f(vp[min(v, a.dv - 1)]);
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        S[i][r] = fmaf(e, S[i][r], vv * k[r]);
        s = fmaf(S[i][r], q[r], s);
      }
      if (!on) s = 0.f;
#pragma unroll
      for (int m = 1; m < LK; m <<= 1) s += __shfl_xor(s, m);
      if (l == 0 && v < a.dv) a.o[b * a.so.b + t * a.so.t + h * a.so.h + v] = to_t<E>(a.scale * s);
    }
  }
  float* So = a.S_out + (long)bh * a.dv * a.dk;
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int v = v0 + i * RW;
    if (on && v < a.dv) *reinterpret_cast<f32x4*>(So + v * a.dk + k0) = S[i];
  }
}

template <typename E, int LK>
hipError_t step_lk(const LaStepArgs<E>& a, hipStream_t s) {
  constexpr int RW = 256 / LK;
  const long bh = (long)a.B * a.H;
  // rows a thread: as many as leave a workgroup for each CU, or one
  auto tiles = [&](int rpt) { return (a.dv + RW * rpt - 1) / (RW * rpt); };
  auto go = [&](auto rpt) {
    constexpr int RPT = decltype(rpt)::value;
    const int nt = tiles(RPT);
    hipLaunchKernelGGL((la_step_kernel<E, LK, RPT>), dim3((unsigned)(bh * nt)), dim3(256), 0, s, a, nt);
    return hipGetLastError();
  };
  if (bh * tiles(4) >= 1024) return go(std::integral_constant<int, 4>());
  if (bh * tiles(2) >= 512) return go(std::integral_constant<int, 2>());
  return go(std::integral_constant<int, 1>());
}

}  // namespace

hipError_t launch_la_join(const LaJoin& a, hipStream_t s) {
  const unsigned grid = (unsigned)((long)a.B * a.H * 2 * ((a.DD + 255) / 256));
  hipLaunchKernelGGL(la_join_kernel, dim3(grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_la_decay(const LaDecay& a, hipStream_t s) {
  if (a.B > 0) {
    hipLaunchKernelGGL(la_decay_kernel, dim3((unsigned)((long)a.B * a.H * a.nseg)), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.tmp) return hipSuccess;
  hipLaunchKernelGGL(la_decay_head_kernel, dim3(a.H), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_la_group_sum(const float* part, E* out, long rows, int Hk, int grp, int d, hipStream_t s) {
  const long n4 = rows * Hk * (d / 4);
  if (n4 == 0) return hipSuccess;
  const long want = (n4 + 255) / 256;
  hipLaunchKernelGGL((la_group_kernel<E>), dim3((unsigned)(want < 8192 ? want : 8192)), dim3(256), 0, s, part, out,
                     n4, grp, d / 4);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_la_step(const LaStepArgs<E>& a, hipStream_t s) {
  if (a.dk <= 16) return step_lk<E, 4>(a, s);
  if (a.dk <= 32) return step_lk<E, 8>(a, s);
  if (a.dk <= 64) return step_lk<E, 16>(a, s);
  return step_lk<E, 32>(a, s);
}

template hipError_t launch_la_group_sum<bf16>(const float*, bf16*, long, int, int, int, hipStream_t);
template hipError_t launch_la_group_sum<float>(const float*, float*, long, int, int, int, hipStream_t);
template hipError_t launch_la_step<bf16>(const LaStepArgs<bf16>&, hipStream_t);
template hipError_t launch_la_step<float>(const LaStepArgs<float>&, hipStream_t);

}  // namespace prism
