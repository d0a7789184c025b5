// Linear attention with a decay for each head: the kernels beside the chunk
// passes (linattn_kernel.h): joining of segment states, the decay gradient,
// sums over heads that share keys and values, and the recurrent step.
#include "operators.h"
#include "prism_common.h"

namespace prism {

namespace {

// ------------------------------------------------------------ segment join
// One thread carries four elements of the state over the segments:
// forward X_{s+1} = decay_s X_s + own_s, reverse the other way round.  The
// last segment of a pass has no own state (nothing enters after it).  Reads and
// writes each state once; bound by latency (eight states requested together):
// 16 heads of 128 x 128, 32 segments, 67 MB in 14 us.
__global__ __launch_bounds__(256) void la_join_kernel(const LaJoin a) {
  const int per = (a.DD + 1023) / 1024;
  int id = blockIdx.x;
  const int blk = id % per;
  id /= per;
  const int dir = a.seg[1] ? id % 2 : 0, bh = a.seg[1] ? id / 2 : id;
  __shared__ int sm[4];
  long first = 0;
  int n = a.T;
  if (a.cu) la_sequence(a.cu, a.N, a.T, bh / a.H, threadIdx.x, sm, first, n);
  const int e = blk * 1024 + 4 * threadIdx.x;
  if (e >= a.DD) return;   // (DD is a multiple of 256)
  const int used = max(1, (n + a.seglen - 1) / a.seglen);
  float* seg = a.seg[dir] + (long)bh * a.nseg * a.DD + e;
  const float* dec = a.dec[dir] + (long)bh * a.nseg;
  auto at = [&](int x) { return reinterpret_cast<f32x4*>(seg + (long)x * a.DD); };
  f32x4 x = a.X0[dir] ? *reinterpret_cast<const f32x4*>(a.X0[dir] + (long)bh * a.DD + e) : f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int U = 8;   // own states requested together
  for (int i0 = 0; i0 < used - 1; i0 += U) {
    f32x4 own[U];
    float d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(i0 + u, used - 2), s = dir ? used - 1 - i : i;
      own[u] = *at(s);
      d[u] = dec[s];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < used - 1) {
        *at(dir ? used - 1 - (i0 + u) : i0 + u) = x;
        x = x * d[u] + own[u];
      }
  }
  *at(dir ? 0 : used - 1) = x;
}

// ---------------------------------------------------------- decay gradient
// One workgroup a segment: <dS, S> at its end, then the suffix sums of
// q.dq - k.dk (in fp64: differences of long sums), 1024 tokens at a time from
// the end, four a thread.  Anchored at each segment's end, so that the segments
// need not wait for one another.  Bound by latency: 8 x 2048 tokens, 16 heads of
// 128, 2 segments: 13.6 us for 34 MB of states, 8 MB of row sums and 2 MB of g
// and dg (25 with a token a thread and the states requested one by one).
__global__ __launch_bounds__(256) void la_decay_kernel(const LaDecay a) {
  __shared__ double sm[8];
  const int tid = threadIdx.x;
  // (the heads of one stretch of tokens on one XCD: their values of g and dg
  // share cache lines)
  int id = xcd_swizzle((int)blockIdx.x, (int)gridDim.x);
  const int h = id % a.H;
  id /= a.H;
  const int seg = id % a.nseg, b = id / a.nseg, bh = b * a.H + h;
  __shared__ int sq[4];
  long first = 0;
  int n = a.T;
  if (a.cu) la_sequence(a.cu, a.N, a.T, b, tid, sq, first, n);
  const int s0 = seg * a.seglen, len = min(n - s0, a.seglen);
  if (len <= 0) return;
  // S and dS at the segment's end: the caller's after the last token, else the
  // states that enter the next segment and (in reverse) this one
  const bool last = s0 + len == n;
  const int used = (n + a.seglen - 1) / a.seglen;
  const long o = (long)bh * a.DD;
  double s = 0.0;
  if (!last || a.dST) {
    constexpr int U = 8;   // pieces of each state requested together
    const long sg0 = (long)bh * a.nseg;
    for (int e0 = 4 * tid; e0 < a.DD; e0 += 1024 * U) {
      f32x4 r[U], x[U];
      auto at = [&](int u) { return min(e0 + 1024 * u, a.DD - 4); };
      auto load = [&](f32x4 (&y)[U], const float* p) {
#pragma unroll
        for (int u = 0; u < U; ++u) y[u] = *reinterpret_cast<const f32x4*>(p + at(u));
      };
      // the state entering a segment, from the own states before it
      auto enter = [&](f32x4 (&y)[U], const float* own, const float* dec, const float* X0, int from, int to, int step) {
        if (X0) {
          load(y, X0 + o);
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u) y[u] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        for (int i = from; i != to; i += step) {
          f32x4 z[U];
          load(z, own + (sg0 + i) * a.DD);
          const float d = dec[sg0 + i];
#pragma unroll
          for (int u = 0; u < U; ++u) y[u] = y[u] * d + z[u];
        }
      };
      if (last) {
        load(r, a.dST + o);
        load(x, a.ST + o);
      } else if (a.joined) {
        load(r, a.segr + (sg0 + seg) * a.DD);
        load(x, a.segf + (sg0 + seg + 1) * a.DD);
      } else {
        enter(r, a.segr, a.decr, a.dST, used - 1, seg, -1);
        enter(x, a.segf, a.decf, a.S0, 0, seg + 1, 1);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (e0 + 1024 * u < a.DD) {
#pragma unroll
          for (int k = 0; k < 4; ++k) s += (double)r[u][k] * (double)x[u][k];
        }
    }
  }
  const int lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if (lane == 0) sm[wave] = s;
  __syncthreads();
  double carry = (sm[0] + sm[1]) + (sm[2] + sm[3]);
  const long row0 = first + s0;
  const long at0 = (a.cu ? 0 : (long)b * a.T) + row0;   // the segment's first row of all rows
  const float* eq = a.eq + (long)h * LA_PARTS * a.rows + at0;
  const float* ek = a.ek + (long)h * LA_PARTS * a.rows + at0;
  const float* pg = a.g + ((a.cu ? 0 : b * a.sg.b) + row0 * a.sg.t + h * a.sg.h);
  // thread tid holds the U tokens hi - 1 - U tid - r, r = 0 .. U - 1, of a block
  // of 256 U (prefix sums over r, then over the threads)
  constexpr int U = 4;
  int buf = 4;
  for (int hi = len; hi > 0; hi -= 256 * U) {
    const int t0 = hi - 1 - U * tid;
    float q[U][LA_PARTS], k[U][LA_PARTS], g[U];
#pragma unroll
    for (int r = 0; r < U; ++r) {
      const int t = max(t0 - r, 0);
#pragma unroll
      for (int p = 0; p < LA_PARTS; ++p) {
        q[r][p] = eq[p * a.rows + t];
        k[r][p] = ek[p * a.rows + t];
      }
      g[r] = pg[(long)t * a.sg.t];
    }
    double x[U];
#pragma unroll
    for (int r = 0; r < U; ++r) {
      x[r] = 0.0;
#pragma unroll
      for (int p = 0; p < LA_PARTS; ++p) x[r] += (double)q[r][p] - (double)k[r][p];
      if (t0 - r < 0) x[r] = 0.0;
      if (r > 0) x[r] += x[r - 1];
    }
    double run = x[U - 1];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double y = __shfl_up(run, o);
      if (lane >= o) run += y;
    }
    if (lane == 63) sm[buf + wave] = run;
    __syncthreads();
    double before = carry + (run - x[U - 1]);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w < wave) before += sm[buf + w];
      carry += sm[buf + w];
    }
    buf ^= 4;   // (the other four sums: one barrier a block)
#pragma unroll
    for (int r = 0; r < U; ++r) {
      const int t = t0 - r;
      if (t < 0) continue;
      const float d = g[r] < -104.f ? 0.f : (float)(before + x[r]);
      if (a.per_head)
        a.tmp[(long)h * a.rows + at0 + t] = d;
      else
        a.dg[(a.cu ? 0 : b * a.sg.b) + (row0 + t) * a.sg.t + h * a.sg.h] = d;
    }
  }
}

// One decay a head: the sum of its tokens' gradients over the batch.
__global__ __launch_bounds__(256) void la_decay_head_kernel(const LaDecay a) {
  __shared__ double sm[256];
  const int tid = threadIdx.x, h = blockIdx.x;
  double s = 0.0;
  int m = a.cu ? min(max(a.cu[0], 0), a.N) : 0;   // (the clamped offsets, as la_sequence has them)
  for (int b = 0; b < a.B; ++b) {
    int n = a.T;
    long first = (long)b * a.T;
    if (a.cu) {
      const int end = max(m, min(a.cu[b + 1], a.N));
      first = m;
      n = min(end - m, a.T);
      m = end;
    }
    const float* x = a.tmp + (long)h * a.rows + first;
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
// dk, dv of the heads that share them, in order (fp32 sums, rounded once).
// Memory bound: 2 x 4096 tokens, 16 heads on 4, 134 MB read and 17 written in 24
// us, 6.3 TB/s (the partial sums are partly still in the last-level cache).
template <typename E>
__global__ __launch_bounds__(256) void la_group_kernel(const float* __restrict__ dkp, const float* __restrict__ dvp,
                                                       E* __restrict__ dk, E* __restrict__ dv, long nk4, long n4,
                                                       int grp, int dk4, int dv4) {
  for (long j = (long)blockIdx.x * 256 + threadIdx.x; j < n4; j += (long)gridDim.x * 256) {
    const bool keys = j < nk4;
    const long i = keys ? j : j - nk4;
    const int d4 = keys ? dk4 : dv4;
    const long row = i / d4;
    const int c = (int)(i - row * d4);
    const float* p = (keys ? dkp : dvp) + (row * grp * d4 + c) * 4;
    f32x4 s = *reinterpret_cast<const f32x4*>(p);
    for (int k = 1; k < grp; ++k) s += *reinterpret_cast<const f32x4*>(p + (long)k * d4 * 4);
    st_f4((keys ? dk : dv) + i * 4, s);
  }
}

// ------------------------------------------------------------------- step
// S [dv][dk]: LK lanes hold a row (4 values each), RPT rows a thread; the rows
// stay in registers over the call's tokens, so S crosses memory once.  Memory
// bound by S, read and written: one token of 64 sequences, 16 heads of 128 x 128,
// 134 MB in 24 us, 5.6 TB/s (30 us with one row a thread, 24 with four).
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
    const float e = expf(a.g[b * a.sg.b + t * a.sg.t + h * a.sg.h]);
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
  constexpr int RPT = 2, RW = 256 / LK;
  const int tiles = (a.dv + RW * RPT - 1) / (RW * RPT);
  hipLaunchKernelGGL((la_step_kernel<E, LK, RPT>), dim3((unsigned)((long)a.B * a.H * tiles)), dim3(256), 0, s, a,
                     tiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_la_join(const LaJoin& a, hipStream_t s) {
  const unsigned grid = (unsigned)((long)a.B * a.H * (a.seg[1] ? 2 : 1) * ((a.DD + 1023) / 1024));
  hipLaunchKernelGGL(la_join_kernel, dim3(grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_la_decay(const LaDecay& a, hipStream_t s) {
  if (a.B > 0) {
    hipLaunchKernelGGL(la_decay_kernel, dim3((unsigned)((long)a.B * a.H * a.nseg)), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.per_head) return hipSuccess;
  hipLaunchKernelGGL(la_decay_head_kernel, dim3(a.H), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_la_group_sum(const float* dkp, const float* dvp, E* dk, E* dv, long rows, int Hk, int grp, int dimk,
                               int dimv, hipStream_t s) {
  const long nk4 = rows * Hk * (dimk / 4), n4 = nk4 + rows * Hk * (dimv / 4);
  if (n4 == 0) return hipSuccess;
  const long want = (n4 + 255) / 256;
  hipLaunchKernelGGL((la_group_kernel<E>), dim3((unsigned)(want < 8192 ? want : 8192)), dim3(256), 0, s, dkp, dvp, dk,
                     dv, nk4, n4, grp, dimk / 4, dimv / 4);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_la_step(const LaStepArgs<E>& a, hipStream_t s) {
  if (a.dk <= 16) return step_lk<E, 4>(a, s);
  if (a.dk <= 32) return step_lk<E, 8>(a, s);
  if (a.dk <= 64) return step_lk<E, 16>(a, s);
  return step_lk<E, 32>(a, s);
}

template hipError_t launch_la_group_sum<bf16>(const float*, const float*, bf16*, bf16*, long, int, int, int, int,
                                              hipStream_t);
template hipError_t launch_la_group_sum<float>(const float*, const float*, float*, float*, long, int, int, int, int,
                                               hipStream_t);
template hipError_t launch_la_step<bf16>(const LaStepArgs<bf16>&, hipStream_t);
template hipError_t launch_la_step<float>(const LaStepArgs<float>&, hipStream_t);

}  // namespace prism
