// Query / key normalisation for each head with the rotation by position, and
// its backward pass.  For a row x of d values (one token, one head):
//   r = (c sum x^2 + eps)^(-1/2),  y = r x w,  z = y with its first `rot`
//   values turned in pairs by angle_i = 2 pi p F_i 2^-64,
// and, with dy = dz turned back, h = dy w and u = r x,
//   dx = r (h - c u (u . h)),  dw = sum over rows of dy u
// (by u, of size 1: r^3 would leave fp32's range for rows shorter than 1e-13 or
// longer than 1e13, whose gradients are well within it).
//
// Memory bound: a row is read once and written once (backward: x and dz read,
// dx written), everything else stays in registers.  A row belongs to a group
// of G lanes; a lane owns P = d / (2 V G) <= 1 pair of 16-byte (8-byte) vectors
// that hold both members of V rotation pairs, so turning needs no exchange
// between lanes and the row sums are DPP sums over the group.  The groups of a
// team, at most a wave, share one token: its V angles are formed once in each
// lane and used for all its heads.  (A workgroup a token took 83 us in place of
// 48 for 8 x 2048 tokens of 16 + 16 heads, and nothing less for 64 tokens.)
//
// Measured, bf16, d = 128: forward, 8 x 2048 tokens of 16 + 16 heads, 268 MB,
// 48 us, 5.6 TB/s (a copy of this size runs at 5.3 TB/s); backward with weights,
// 16384 tokens of 16 + 4 heads, 252 MB, 50 us, 5.0 TB/s.  One token for each of
// 64 sequences: 5 us, the launch and one memory latency.
#include "operators.h"
#include "prism_common.h"

namespace prism {

namespace {

constexpr int QN_NT = 256;

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
template <> struct VecIo<float, 4> {
  typedef f32x4 raw;
  __device__ static inline void unpack(const raw& w, float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = w[i];
  }
  __device__ static inline raw pack(const float (&x)[4]) { return raw{x[0], x[1], x[2], x[3]}; }
};

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

// Where the lane's two vectors lie in a row, and the first rotation pair of
// the lane (-1: its values pass).
struct LanePlace {
  int a, b, pair;
  bool on;
};
template <int V, bool IL>
__device__ inline LanePlace lane_place(int p, int d, int rot) {
  LanePlace q;
  q.on = p < d / (2 * V);
  if (!q.on) p = 0;
  if (IL) {
    q.a = 2 * V * p;
    q.b = q.a + V;
    q.pair = q.a < rot ? V * p : -1;
  } else {
    const int np = rot / (2 * V);
    q.a = p < np ? V * p : rot + 2 * V * (p - np);
    q.b = p < np ? rot / 2 + V * p : q.a + V;
    q.pair = p < np ? V * p : -1;
  }
  return q;
}

// cos, sin of the lane's V angles.  The phase p F mod 2^64 is exact; its upper
// 32 bits, as a signed number rounded to fp32, keep the angle to 2^-32 of a turn
// and 2^-24 of its size (an fp32 product p * frequency would lose position's
// bits).  For bf16 the hardware's
// sine and cosine of turns do (absolute error about 2^-20; the outputs are
// rounded at 2^-9); fp32 takes the library's.
template <typename E, int V>
__device__ inline void lane_angles(const QkNormArgs& g, long tok, const LanePlace& q, float (&cs)[V],
                                   float (&sn)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  if (g.rot > 0 && q.pair >= 0) {
    const unsigned long long p = (unsigned long long)(long long)g.pos[tok];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const unsigned long long ph = p * (unsigned long long)g.turns[q.pair + i];
      const float f = (float)(int)(unsigned)(ph >> 32);
      if (sizeof(E) == 2) {
        sn[i] = __builtin_amdgcn_sinf(f * 0x1p-32f);
        cs[i] = __builtin_amdgcn_cosf(f * 0x1p-32f);
      } else {
        sincospif(f * 0x1p-31f, &sn[i], &cs[i]);
      }
    }
  }
}

// Turns the lane's pairs: S = +1 forward, -1 back.
template <int V, bool IL, int S>
__device__ inline void turn(float (&a)[V], float (&b)[V], const float (&cs)[V], const float (&sn)[V]) {
  if (IL) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float s0 = S * sn[i], s1 = S * sn[V / 2 + i];
      const float x0 = a[2 * i], x1 = a[2 * i + 1], y0 = b[2 * i], y1 = b[2 * i + 1];
      a[2 * i] = x0 * cs[i] - x1 * s0;
      a[2 * i + 1] = x1 * cs[i] + x0 * s0;
      b[2 * i] = y0 * cs[V / 2 + i] - y1 * s1;
      b[2 * i + 1] = y1 * cs[V / 2 + i] + y0 * s1;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float s = S * sn[i], x = a[i], y = b[i];
      a[i] = x * cs[i] - y * s;
      b[i] = y * cs[i] + x * s;
    }
  }
}

// Row addresses of head h (q heads first, then k heads) of token (b, t).
template <typename E>
__device__ inline const E* row_of(const void* q, const void* k, const Strides& sq, const Strides& sk,
                                  int h, int Hq, int b, int t) {
  return h < Hq ? static_cast<const E*>(q) + (b * sq.b + t * sq.t + h * sq.h)
                : static_cast<const E*>(k) + (b * sk.b + t * sk.t + (h - Hq) * sk.h);
}

template <typename E, int V>
__device__ inline void load_w(const void* w, const LanePlace& q, float (&wa)[V], float (&wb)[V]) {
  typedef typename VecIo<E, V>::raw raw;
  if (w) {
    VecIo<E, V>::unpack(*reinterpret_cast<const raw*>(static_cast<const E*>(w) + q.a), wa);
    VecIo<E, V>::unpack(*reinterpret_cast<const raw*>(static_cast<const E*>(w) + q.b), wb);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) wa[i] = wb[i] = 1.f;
  }
}

// G lanes a row, tg groups a token (both powers of two, G * tg <= 64).
template <typename E, int V, bool IL>
__global__ __launch_bounds__(QN_NT) void qk_norm_kernel(const QkNormArgs g, int G, int tg) {
  typedef VecIo<E, V> IO;
  typedef typename IO::raw raw;
  constexpr int U = 4;   // rows of a group in flight
  const int tid = threadIdx.x, lane = tid & (G - 1);
  const int grp = tid / G, team = grp / tg, gi = grp & (tg - 1);
  const int teams = QN_NT / (G * tg);
  const int H = g.Hq + g.Hk;
  const LanePlace q = lane_place<V, IL>(lane, g.d, g.rot);
  const long N = (long)g.B * g.T;
  float wqa[V], wqb[V], wka[V], wkb[V];
  load_w<E, V>(g.wq, q, wqa, wqb);
  load_w<E, V>(g.wk, q, wka, wkb);
  for (long tok = (long)blockIdx.x * teams + team; tok < N; tok += (long)gridDim.x * teams) {
    const int b = (int)(tok / g.T), t = (int)(tok - (long)b * g.T);
    float cs[V], sn[V];
    bool first = true;
    for (int h0 = gi; h0 < H; h0 += U * tg) {
      raw ra[U], rb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = min(h0 + u * tg, H - 1);
        const E* x = row_of<E>(g.xq, g.xk, g.sxq, g.sxk, h, g.Hq, b, t);
        ra[u] = *reinterpret_cast<const raw*>(x + q.a);
        rb[u] = *reinterpret_cast<const raw*>(x + q.b);
      }
      if (first) lane_angles<E, V>(g, tok, q, cs, sn);
      first = false;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * tg;
        float xa[V], xb[V];
        IO::unpack(ra[u], xa);
        IO::unpack(rb[u], xb);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(xa[i], xa[i], fmaf(xb[i], xb[i], ss));
        ss = group_sum(q.on ? ss : 0.f, G);
        const float r = rsqrtf(fmaf(g.c, ss, g.eps));
        const bool isq = h < g.Hq;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          xa[i] *= r * (isq ? wqa[i] : wka[i]);
          xb[i] *= r * (isq ? wqb[i] : wkb[i]);
        }
        turn<V, IL, 1>(xa, xb, cs, sn);
        if (h < H && q.on) {
          E* y = const_cast<E*>(row_of<E>(g.yq, g.yk, g.syq, g.syk, h, g.Hq, b, t));
          *reinterpret_cast<raw*>(y + q.a) = IO::pack(xa);
          *reinterpret_cast<raw*>(y + q.b) = IO::pack(xb);
        }
      }
    }
  }
}

// The rows of q or of k (the first nq workgroups take q: one kind's weights and
// sums in a workgroup's registers).  The weight gradients of a workgroup's rows
// are summed in registers over its tokens, then over its groups (in the wave,
// then over the waves through LDS), and written as one partial [d] for each
// workgroup.
template <typename E, int V, bool IL, bool DW>
__global__ __launch_bounds__(QN_NT) void qk_norm_bwd_kernel(const QkNormArgs g, int G, int nq, int tgq, int tgk) {
  typedef VecIo<E, V> IO;
  typedef typename IO::raw raw;
  const bool isq = (int)blockIdx.x < nq;
  const int blk = isq ? blockIdx.x : blockIdx.x - nq, nblk = isq ? nq : gridDim.x - nq;
  const int tg = isq ? tgq : tgk, H = isq ? g.Hq : g.Hk;
  const void *px = isq ? g.xq : g.xk, *pz = isq ? g.gq : g.gk;
  void* py = isq ? g.yq : g.yk;
  const Strides sx = isq ? g.sxq : g.sxk, sg = isq ? g.sgq : g.sgk, sy = isq ? g.syq : g.syk;
  const int tid = threadIdx.x, lane = tid & (G - 1);
  const int grp = tid / G, team = grp / tg, gi = grp & (tg - 1);
  const int teams = QN_NT / (G * tg);
  const LanePlace q = lane_place<V, IL>(lane, g.d, g.rot);
  const long N = (long)g.B * g.T;
  float wa[V], wb[V], da[V], db[V];
  load_w<E, V>(isq ? g.wq : g.wk, q, wa, wb);
#pragma unroll
  for (int i = 0; i < V; ++i) da[i] = db[i] = 0.f;
  for (long tok = (long)blk * teams + team; tok < N; tok += (long)nblk * teams) {
    const int b = (int)(tok / g.T), t = (int)(tok - (long)b * g.T);
    const E* x = static_cast<const E*>(px) + (b * sx.b + t * sx.t);
    const E* dz = static_cast<const E*>(pz) + (b * sg.b + t * sg.t);
    E* dx = static_cast<E*>(py) + (b * sy.b + t * sy.t);
    float cs[V], sn[V];
    bool first = true;
    // (a row at a time: two in flight measured 3 us slower, of 57, by their registers)
    for (int h = gi; h < H; h += tg) {
      const raw ra = *reinterpret_cast<const raw*>(x + h * sx.h + q.a);
      const raw rb = *reinterpret_cast<const raw*>(x + h * sx.h + q.b);
      const raw rc = *reinterpret_cast<const raw*>(dz + h * sg.h + q.a);
      const raw rd = *reinterpret_cast<const raw*>(dz + h * sg.h + q.b);
      if (first) lane_angles<E, V>(g, tok, q, cs, sn);
      first = false;
      float xa[V], xb[V], ga[V], gb[V];
      IO::unpack(ra, xa);
      IO::unpack(rb, xb);
      IO::unpack(rc, ga);
      IO::unpack(rd, gb);
      turn<V, IL, -1>(ga, gb, cs, sn);
      float ss = 0.f, xh = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ss = fmaf(xa[i], xa[i], fmaf(xb[i], xb[i], ss));
        xh = fmaf(xa[i] * wa[i], ga[i], fmaf(xb[i] * wb[i], gb[i], xh));
      }
      ss = group_sum(q.on ? ss : 0.f, G);
      xh = group_sum(q.on ? xh : 0.f, G);
      const float r = rsqrtf(fmaf(g.c, ss, g.eps));
      const float m = g.c * (r * xh);   // c u.h
      if (q.on) {
        float ya[V], yb[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float ua = r * xa[i], ub = r * xb[i];
          ya[i] = r * fmaf(-m, ua, wa[i] * ga[i]);
          yb[i] = r * fmaf(-m, ub, wb[i] * gb[i]);
          if (DW) {
            da[i] = fmaf(ua, ga[i], da[i]);
            db[i] = fmaf(ub, gb[i], db[i]);
          }
        }
        *reinterpret_cast<raw*>(dx + h * sy.h + q.a) = IO::pack(ya);
        *reinterpret_cast<raw*>(dx + h * sy.h + q.b) = IO::pack(yb);
      }
    }
  }
  if constexpr (DW) {
    __shared__ float sm[QN_NT / WAVE][2][V * 32];
    const int wave = tid / WAVE, wl = tid & (WAVE - 1);
    auto fold = [&](float (&v)[V], int row) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        for (int m = G; m < WAVE; m <<= 1) v[i] += __shfl_xor(v[i], m);
        if (wl < G) sm[wave][row][V * wl + i] = v[i];
      }
    };
    fold(da, 0);
    fold(db, 1);
    __syncthreads();
    float* out = g.part + (long)blockIdx.x * g.d;
    for (int e = tid; e < 2 * V * G; e += QN_NT) {
      const int row = e / (V * G), j = e % (V * G);
      const LanePlace w = lane_place<V, IL>(j / V, g.d, g.rot);
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < QN_NT / WAVE; ++k) s += sm[k][row][j];
      if (w.on) out[(row ? w.b : w.a) + j % V] = s;
    }
  }
}

// Column sums of the partial rows [d]: the first nq give dwq, the others dwk.
// 32 columns a workgroup, 32 threads on each column taking every 32nd row,
// joined through LDS in a fixed order.
__global__ __launch_bounds__(1024) void qk_norm_dw_kernel(const float* __restrict__ part, int nq, int n, int d,
                                                          float* __restrict__ dwq,
                                                          float* __restrict__ dwk) {
  __shared__ float sm[32][33];
  const int c = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  const bool isq = blockIdx.y == 0;
  float* out = isq ? dwq : dwk;
  if (!out) return;
  float s = 0.f;
  if (col < d) {
#pragma unroll 8
    for (int r = (isq ? 0 : nq) + y; r < (isq ? nq : n); r += 32) s += part[(long)r * d + col];
  }
  sm[y][c] = s;
  __syncthreads();
  if (y == 0 && col < d) {
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) x += sm[k][c];
    out[col] = x;
  }
}

constexpr int QN_PARTS = 1024;   // workgroups of the backward kernel with weights, at most

int pow2_at_least(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

// The forward pass takes vectors of 8 bf16 where every row offset is a multiple
// of 16 bytes, else of 4 (8 x 2048 tokens, 16 + 16 heads of 128: 48 us with 8,
// 56 with 4).  The backward pass always takes 4, for its registers (the same
// shape: 82 us with 4, 85 with 8).
bool wide(const QkNormArgs& a) {
  if (a.d % 16 || a.rot % 16) return false;
  long m = a.sxq.b | a.sxq.t | a.sxq.h | a.syq.b | a.syq.t | a.syq.h;
  if (a.Hk) m |= a.sxk.b | a.sxk.t | a.sxk.h | a.syk.b | a.syk.t | a.syk.h;
  return m % 8 == 0;
}

// Groups a token: a wave's, never more than there are heads.
int team_groups(int G, int H) {
  const int most = WAVE / G, need = pow2_at_least(H);
  return most < need ? most : need;
}

template <typename E, int V>
hipError_t run_fwd(const QkNormArgs& a, hipStream_t s) {
  const int G = pow2_at_least(a.d / (2 * V)), tg = team_groups(G, a.Hq + a.Hk), teams = QN_NT / (G * tg);
  const long N = (long)a.B * a.T;
  long grid = (N + teams - 1) / teams;
  if (grid > (1 << 20)) grid = 1 << 20;
  if (a.interleaved)
    hipLaunchKernelGGL((qk_norm_kernel<E, V, true>), dim3((unsigned)grid), dim3(QN_NT), 0, s, a, G, tg);
  else
    hipLaunchKernelGGL((qk_norm_kernel<E, V, false>), dim3((unsigned)grid), dim3(QN_NT), 0, s, a, G, tg);
  return hipGetLastError();
}

template <typename E, bool IL>
hipError_t run_bwd(const QkNormArgs& a, hipStream_t s) {
  constexpr int V = 4;
  const int G = pow2_at_least(a.d / (2 * V));
  const long N = (long)a.B * a.T;
  const bool dw = a.dwq || a.dwk;
  // workgroups for q and for k: as many as there are teams of tokens, at most
  // `most` in the proportion of their heads
  const long most = dw ? QN_PARTS : (1 << 20);
  auto blocks = [&](int H, int tg) -> long {
    if (H == 0 || N == 0) return 0;
    const int teams = QN_NT / (G * tg);
    const long want = (N + teams - 1) / teams, room = most * H / (a.Hq + a.Hk);
    return want < room ? want : (room > 1 ? room : 1);
  };
  const int tgq = team_groups(G, a.Hq), tgk = a.Hk ? team_groups(G, a.Hk) : 1;
  const long nq = blocks(a.Hq, tgq), nk = blocks(a.Hk, tgk);
  if (N > 0) {
    const dim3 grid((unsigned)(nq + nk));
    if (dw)
      hipLaunchKernelGGL((qk_norm_bwd_kernel<E, V, IL, true>), grid, dim3(QN_NT), 0, s, a, G, (int)nq, tgq, tgk);
    else
      hipLaunchKernelGGL((qk_norm_bwd_kernel<E, V, IL, false>), grid, dim3(QN_NT), 0, s, a, G, (int)nq, tgq, tgk);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dw) {
    hipLaunchKernelGGL(qk_norm_dw_kernel, dim3((a.d + 31) / 32, 2), dim3(1024), 0, s, a.part, (int)nq, (int)(nq + nk),
                       a.d, a.dwq, a.dwk);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace

// (with few heads of one kind its share may round up to one more)
size_t qk_norm_part_bytes(int d) { return (size_t)(QN_PARTS + 1) * d * sizeof(float); }

template <typename E>
hipError_t launch_qk_norm(const QkNormArgs& a, hipStream_t s) {
  if constexpr (sizeof(E) == 2) {
    if (wide(a)) return run_fwd<E, 8>(a, s);
  }
  return run_fwd<E, 4>(a, s);
}
template <typename E>
hipError_t launch_qk_norm_bwd(const QkNormArgs& a, hipStream_t s) {
  return a.interleaved ? run_bwd<E, true>(a, s) : run_bwd<E, false>(a, s);
}
template hipError_t launch_qk_norm<bf16>(const QkNormArgs&, hipStream_t);
template hipError_t launch_qk_norm<float>(const QkNormArgs&, hipStream_t);
template hipError_t launch_qk_norm_bwd<bf16>(const QkNormArgs&, hipStream_t);
template hipError_t launch_qk_norm_bwd<float>(const QkNormArgs&, hipStream_t);

}  // namespace prism
