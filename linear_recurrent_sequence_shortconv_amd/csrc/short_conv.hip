// Depthwise causal convolution over the last K tokens with its activation, and
// its backward pass.  Channel by channel,
//   z_t = bias + sum_{j < K} w_j x_{t-j},  y_t = z_t, or z_t sigma(z_t) (silu),
// with the K - 1 tokens before the sequence from `hist` (nullptr: zeros), and,
// with g_t = dy_t act'(z_t) (z formed again from x),
//   dx_t = sum_j w_j g_{t+j},  dw_j = sum_t g_t x_{t-j},  dbias = sum_t g_t,
// the dx of the tokens before the sequence being dhist.
//
// Memory bound: a wave walks a strip of tokens with V channels a lane, so that
// each value is read once but for the K - 1 rows in front of a strip (backward:
// behind it too), which the wave next to it reads at the same time.  The rows
// before the current one, and in the backward pass the g before it, stay in
// registers.  bf16, K = 4, silu, 8 x 2048 tokens of 2048 channels: 26 us, 5.2 TB/s;
// backward 49 us with the sums of partials, 4.1 TB/s.  What is left: the start of a
// strip, whose first rows nothing hides, and backward the arithmetic (the vector
// units' issue of sigma, its slope and 8 products a value).
#include <type_traits>

#include "block_ops.h"
#include "vec_io.h"

namespace prism {

namespace {

constexpr int SC_WAVES = 4;
constexpr int SC_STRIP = 32, SC_STRIP_BWD = 64;   // tokens

// sigma, for bf16 results by the hardware's exponential and reciprocal (1 ulp
// each; the argument's rounding adds 2^-24 of its size).
template <typename E>
__device__ inline float sigma(float z) {
  if constexpr (sizeof(E) == 2) return __builtin_amdgcn_rcpf(1.f + __expf(-z));
  return 1.f / (1.f + expf(-z));
}

template <typename E, int V>
__device__ inline void load_row(const E* p, float (&x)[V]) {
  VecIo<E, V>::unpack(load_vec<E, V>(p), x);
}

// Row e - start of a sequence, or of the rows before it.
template <typename E, int V, int K>
__device__ inline void load_past(const ShortConvArgs& a, const E* x, int b, int t, int c, float (&v)[V]) {
  if (t >= 0) {
    load_row<E, V>(x + t * a.sx.t + c, v);
  } else if (a.hist) {
    load_row<E, V>(static_cast<const E*>(a.hist) + ((long)b * (K - 1) + K - 1 + t) * a.D + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.f;
  }
}

// The lane's taps, w [D][K].
template <typename E, int V, int K>
__device__ inline void load_taps(const void* w, int c, float (&t)[K][V]) {
  typedef typename VecIo<E, V>::raw raw;
  E e[V * K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const raw r = load_vec<E, V>(static_cast<const E*>(w) + (long)c * K + k * V);
    __builtin_memcpy(e + k * V, &r, sizeof(raw));
  }
#pragma unroll
  for (int j = 0; j < K; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) t[j][i] = to_f(e[i * K + j]);
}

// A workgroup's waves take neighbouring strips of the same channels.  The lane's
// channels are c + skip .. c + V - 1 (skip = V: none).
struct Place {
  int blk, strip, c, skip;
  bool whole;   // no lane of the wave skips any
};
template <int V>
__device__ inline Place place_of(int D, int cw) {
  Place p;
  const int id = blockIdx.x;
  p.blk = id / cw;
  p.strip = __builtin_amdgcn_readfirstlane(p.blk * SC_WAVES + threadIdx.x / WAVE);
  const int c = ((id - p.blk * cw) * WAVE + (threadIdx.x & (WAVE - 1))) * V;
  p.c = c < D ? min(c, D - V) : 0;
  p.skip = c < D ? c - p.c : V;
  p.whole = __all(p.skip == 0);
  return p;
}

template <typename E>
__device__ inline const E* sequence_base(const void* p, const TokenSteps& s, const int* cu, const Sequence& q) {
  return static_cast<const E*>(p) + (cu ? q.start * s.t : q.b * s.b);
}

// Workgroups behind those of the strips take a sequence each: one without tokens
// leaves its history as it was.
template <typename W>
__device__ inline void leave_history(const ShortConvArgs& a, int b, int n, W* dst, const W* src) {
  __shared__ int sm[4];
  if (!dst || !empty_sequence(a.cu, a.T, a.rows, b, sm)) return;
  for (int e = threadIdx.x; e < n; e += SC_WAVES * WAVE) dst[(long)b * n + e] = src ? src[(long)b * n + e] : W(0.f);
}

// The first K - 1 tokens of a sequence, which read hist, belong to the strip of
// its first token, whose wave also writes hist_out: hist may be updated in place.
template <typename E, int V, int K, bool SILU>
__global__ __launch_bounds__(SC_WAVES * WAVE) void short_conv_kernel(const ShortConvArgs a, int cw, int S, int strips) {
  typedef VecIo<E, V> IO;
  typedef typename IO::raw raw;
  constexpr int U = 4;
  if ((int)blockIdx.x >= strips) {
    leave_history(a, blockIdx.x - strips, (K - 1) * a.D, static_cast<E*>(a.hist_out), static_cast<const E*>(a.hist));
    return;
  }
  const Place p = place_of<V>(a.D, cw);
  const int lo = p.strip * S, hi = min(lo + S, a.rows);
  if (lo >= a.rows) return;
  float w[K][V], bias[V];
  load_taps<E, V, K>(a.w, p.c, w);
  if (a.b) {
    load_row<E, V>(static_cast<const E*>(a.b) + p.c, bias);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = 0.f;
  }
  int row = lo;
  while (row < hi) {
    const Sequence q = find_sequence(a.cu, a.B, a.T, a.rows, row);
    if (q.b < 0 || q.b >= a.B) {
      row = q.end;
      continue;
    }
    const bool mine = q.start >= lo;
    if (!mine) row = max(row, min(q.start + K - 1, q.end));
    const int stop = max(min(q.end, hi), mine ? min(q.end, q.start + K - 1) : 0);
    if (row >= stop) {
      row = max(row, stop);
      continue;
    }
    const E* x = sequence_base<E>(a.x, a.sx, a.cu, q);
    E* y = const_cast<E*>(sequence_base<E>(a.y, a.sy, a.cu, q));
    float past[K - 1][V];   // past[j]: row - 1 - j
#pragma unroll
    for (int j = 0; j < K - 1; ++j) load_past<E, V, K>(a, x, q.b, row - q.start - 1 - j, p.c, past[j]);
    if (mine && a.hist_out) {
      float last[K - 1][V];
      const int n = q.end - q.start;
#pragma unroll
      for (int m = 0; m < K - 1; ++m) load_past<E, V, K>(a, x, q.b, n - (K - 1) + m, p.c, last[m]);
#pragma unroll
      for (int m = 0; m < K - 1; ++m)
        store_vec<E, V>(static_cast<E*>(a.hist_out) + ((long)q.b * (K - 1) + m) * a.D + p.c, last[m], p.skip, p.whole);
    }
    raw in[U], ahead[U];
    auto load = [&](raw(&r)[U], int row) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        r[u] = load_vec<E, V>(x + (long)(min(row + u, stop - 1) - q.start) * a.sx.t + p.c);
    };
    load(ahead, row);
    auto rows = [&](int row, auto inner) {   // INNER: U rows, and a whole wave
      constexpr bool INNER = decltype(inner)::value;
#pragma unroll
      for (int u = 0; u < U; ++u) in[u] = ahead[u];
      if (row + U < stop) load(ahead, row + U);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float now[V], z[V];
        IO::unpack(in[u], now);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          z[i] = fmaf(w[0][i], now[i], bias[i]);
#pragma unroll
          for (int j = 1; j < K; ++j) z[i] = fmaf(w[j][i], past[j - 1][i], z[i]);
          if (SILU) z[i] *= sigma<E>(z[i]);
#pragma unroll
          for (int j = K - 2; j > 0; --j) past[j][i] = past[j - 1][i];
          past[0][i] = now[i];
        }
        if (INNER || row + u < stop)
          store_vec<E, V>(y + (long)(row + u - q.start) * a.sy.t + p.c, z, INNER ? 0 : p.skip, INNER || p.whole);
      }
    };
    for (; row < stop; row += U) {
      if (p.whole && row + U <= stop)
        rows(row, std::true_type());
      else
        rows(row, std::false_type());
    }
    row = stop;
  }
}

// Rows lo .. hi - 1 of dx come from g up to K - 1 rows further; the sums over
// tokens take the g of lo .. hi - 1 alone.  The waves' sums are joined through
// LDS one after the other, and leave as one partial [K + 1][D] a workgroup.
template <typename E, int V, int K, bool SILU>
__global__ __launch_bounds__(SC_WAVES * WAVE, V == 4 ? 4 : 8) void short_conv_bwd_kernel(const ShortConvArgs a, int cw,
                                                                                       int S, int strips) {
  typedef VecIo<E, V> IO;
  typedef typename IO::raw raw;
  constexpr int U = 4;
  __shared__ float sm[(K + 1) * V][WAVE];
  if ((int)blockIdx.x >= strips) {
    leave_history<float>(a, blockIdx.x - strips, (K - 1) * a.D, a.dhist, nullptr);
    return;
  }
  const Place p = place_of<V>(a.D, cw);
  const int lo = min(p.strip * S, a.rows), hi = min(lo + S, a.rows);
  float w[K][V], bias[V], dw[K + 1][V];
  load_taps<E, V, K>(a.w, p.c, w);
  if (a.b) {
    load_row<E, V>(static_cast<const E*>(a.b) + p.c, bias);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = 0.f;
  }
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[j][i] = 0.f;
  int at = lo;
  while (at < hi) {
    const Sequence q = find_sequence(a.cu, a.B, a.T, a.rows, at);
    if (q.b < 0 || q.b >= a.B) {
      at = q.end;
      continue;
    }
    const E* x = sequence_base<E>(a.x, a.sx, a.cu, q);
    const E* dy = sequence_base<E>(a.dy, a.sy, a.cu, q);
    E* dx = const_cast<E*>(sequence_base<E>(a.dx, a.sd, a.cu, q));
    const int own = min(q.end, hi), stop = own + K - 1;   // rows of g, zero from q.end on
    float past[K - 1][V], gp[K - 1][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      load_past<E, V, K>(a, x, q.b, at - q.start - 1 - j, p.c, past[j]);
#pragma unroll
      for (int i = 0; i < V; ++i) gp[j][i] = 0.f;
    }
    // U rows from `row`; INNER: all of them the strip's, behind its first K - 1, and
    // the wave whole
    auto rows = [&](int row, auto inner) {
      constexpr bool INNER = decltype(inner)::value;
      raw in[U], gr[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long t = (INNER ? row + u : min(row + u, q.end - 1)) - q.start;
        in[u] = load_vec<E, V>(x + t * a.sx.t + p.c);
        gr[u] = load_vec<E, V>(dy + t * a.sy.t + p.c);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = row + u;
        float now[V], g[V], out[V];
        IO::unpack(in[u], now);
        IO::unpack(gr[u], g);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (SILU) {
            float z = fmaf(w[0][i], now[i], bias[i]);
#pragma unroll
            for (int j = 1; j < K; ++j) z = fmaf(w[j][i], past[j - 1][i], z);
            const float s = sigma<E>(z);
            g[i] *= s * fmaf(z, 1.f - s, 1.f);
          }
          if (!INNER && r >= q.end) g[i] = 0.f;
          if (INNER || r < own) {
            dw[0][i] = fmaf(g[i], now[i], dw[0][i]);
#pragma unroll
            for (int j = 1; j < K; ++j) dw[j][i] = fmaf(g[i], past[j - 1][i], dw[j][i]);
            dw[K][i] += g[i];
          }
          // dx of row r - (K - 1)
          out[i] = w[K - 1][i] * g[i];
#pragma unroll
          for (int j = 0; j < K - 1; ++j) out[i] = fmaf(w[K - 2 - j][i], gp[j][i], out[i]);
#pragma unroll
          for (int j = K - 2; j > 0; --j) {
            past[j][i] = past[j - 1][i];
            gp[j][i] = gp[j - 1][i];
          }
          past[0][i] = now[i];
          gp[0][i] = g[i];
        }
        const int e = r - (K - 1);
        if (INNER || r < stop) {
          if (INNER || e >= at) {
            store_vec<E, V>(dx + (long)(e - q.start) * a.sd.t + p.c, out, INNER ? 0 : p.skip, INNER || p.whole);
          } else if (at == q.start && a.dhist) {
            float* d = a.dhist + ((long)q.b * (K - 1) + (r - q.start)) * a.D + p.c;
#pragma unroll
            for (int i = 0; i < V; ++i)
              if (i >= p.skip) d[i] = out[i];
          }
        }
      }
    };
    int row = at;
    rows(row, std::false_type());
    row += U;   // (U >= K - 1)
    if (p.whole)
      for (; row + U <= own; row += U) rows(row, std::true_type());
    for (; row < stop; row += U) rows(row, std::false_type());
    at = own;
  }
  const int wave = threadIdx.x / WAVE, lane = threadIdx.x & (WAVE - 1);
  for (int k = 0; k < SC_WAVES; ++k) {
    __syncthreads();
    if (wave != k) continue;
#pragma unroll
    for (int j = 0; j <= K; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float& s = sm[j * V + i][lane];
        s = k ? s + dw[j][i] : dw[j][i];
        if (k == SC_WAVES - 1 && i >= p.skip) a.part[((long)p.blk * (K + 1) + j) * a.D + p.c + i] = s;
      }
  }
}

// Tokens a strip, fewer (to 4) where that leaves under two waves a SIMD.  (8 x 2048
// tokens of 2048 channels, strips of 16, 32 and 64: 31, 28 and 31 us; backward,
// where a strip also walks K - 1 rows twice on either side, 59, 53 and 51.)
int parts_of(int rows, int S) { return (int)((rows + S * SC_WAVES - 1L) / (S * SC_WAVES)); }
// (longer strips where a launch would have 2^32 threads)
int launchable(int rows, int D, int S) {
  while ((D + 255L) / 256 * parts_of(rows, S) >= (1L << 23)) S *= 2;
  return S;
}
int strip_tokens(int rows, int D, int S) {
  const long waves = (D + 255) / 256;
  while (S > 4 && (rows + S - 1L) / S * waves < 2048) S /= 2;
  return launchable(rows, D, S);
}

// Workgroups for sequences that may be empty and have a result all the same.
int empties(const ShortConvArgs& a, const void* result) {
  return result && result != a.hist && (a.cu || a.T == 0) ? a.B : 0;
}

// (a dense sequence of at most 8 tokens is a strip of its own)
template <typename E, int V, int K>
hipError_t run_fwd(const ShortConvArgs& a, hipStream_t s) {
  const int cw = (a.D + WAVE * V - 1) / (WAVE * V);
  const int S = !a.cu && a.T <= 8 && a.T > 0 ? launchable(a.rows, a.D, a.T) : strip_tokens(a.rows, a.D, SC_STRIP);
  const int strips = cw * parts_of(a.rows, S);
  const dim3 grid((unsigned)strips + empties(a, a.hist_out));
  if (grid.x == 0) return hipSuccess;
  if (a.silu)
    hipLaunchKernelGGL((short_conv_kernel<E, V, K, true>), grid, dim3(SC_WAVES * WAVE), 0, s, a, cw, S, strips);
  else
    hipLaunchKernelGGL((short_conv_kernel<E, V, K, false>), grid, dim3(SC_WAVES * WAVE), 0, s, a, cw, S, strips);
  return hipGetLastError();
}
template <typename E, int V, int K>
hipError_t run_bwd(const ShortConvArgs& a, hipStream_t s) {
  const int cw = (a.D + WAVE * V - 1) / (WAVE * V), S = strip_tokens(a.rows, a.D, SC_STRIP_BWD);
  const int parts = parts_of(a.rows, S), strips = cw * parts;
  const dim3 grid((unsigned)strips + empties(a, a.dhist));
  if (grid.x > 0) {
    if (a.silu)
      hipLaunchKernelGGL((short_conv_bwd_kernel<E, V, K, true>), grid, dim3(SC_WAVES * WAVE), 0, s, a, cw, S, strips);
    else
      hipLaunchKernelGGL((short_conv_bwd_kernel<E, V, K, false>), grid, dim3(SC_WAVES * WAVE), 0, s, a, cw, S, strips);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return launch_column_sums(a.part, parts, a.D, K, a.dw, a.db, s);
}

// Channels a lane: four, or one of rows narrower than that.  (8 x 2048 tokens of 2048
// channels 28 us with four, 36 with one, backward 51 and 57, of 1001 channels 18 and
// 23, backward 39 and 42; eight bf16 take the registers of half the waves: 32 us,
// backward 61.)
template <typename E, bool BWD, int K>
hipError_t run_k(const ShortConvArgs& a, hipStream_t s) {
  if (a.D >= 4) return BWD ? run_bwd<E, 4, K>(a, s) : run_fwd<E, 4, K>(a, s);
  return BWD ? run_bwd<E, 1, K>(a, s) : run_fwd<E, 1, K>(a, s);
}
template <typename E, bool BWD>
hipError_t run(const ShortConvArgs& a, hipStream_t s) {
  if (a.K == 2) return run_k<E, BWD, 2>(a, s);
  if (a.K == 3) return run_k<E, BWD, 3>(a, s);
  return run_k<E, BWD, 4>(a, s);
}

}  // namespace

size_t short_conv_part_bytes(int rows, int D, int K) {
  return (size_t)parts_of(rows, strip_tokens(rows, D, SC_STRIP_BWD)) * (K + 1) * D * sizeof(float);
}

template <typename E>
hipError_t launch_short_conv(const ShortConvArgs& a, hipStream_t s) {
  return run<E, false>(a, s);
}
template <typename E>
hipError_t launch_short_conv_bwd(const ShortConvArgs& a, hipStream_t s) {
  return run<E, true>(a, s);
}
template hipError_t launch_short_conv<bf16>(const ShortConvArgs&, hipStream_t);
template hipError_t launch_short_conv<float>(const ShortConvArgs&, hipStream_t);
template hipError_t launch_short_conv_bwd<bf16>(const ShortConvArgs&, hipStream_t);
template hipError_t launch_short_conv_bwd<float>(const ShortConvArgs&, hipStream_t);

}  // namespace prism
