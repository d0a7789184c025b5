// Linear attention with a decay for each head, over chunks of 32 tokens
// (LaRole in operators.h has the formula).  In a chunk entered with state X,
// with the cumulative log2 decays G_1 .. G_C of its tokens (Gamma_ti = 2^(G_t - G_i)):
//   out = s_in (Gamma o A B^T)_{i<=t} C + s_row 2^G o (A X)
//   X'  = 2^{G_C} X + s_upd B^T (2^{G_C - G} o C)
// (reverse: i >= t, Gamma_ti = 2^(G_i - G_t), 2^{G_C - G_t} and 2^{G_i}).
//
// One workgroup of four waves carries X over its segment's chunks; a wave owns
// 16 NCT of its columns (all DA rows) in fp32 accumulators.  The tiles of A, B
// and C are fetched one chunk ahead in registers and staged in LDS, the only
// data the waves share: with a column of out^T and of X in one wave, what one
// product leaves in accumulators is the next product's operand in the same
// lanes, so neither X nor Gamma o A B^T passes through LDS.  An accumulator
// tile holds rows 4 g + r (g = lane / 16) of one column, a k-contiguous operand
// 8 consecutive k (bf16) of one row at 8 g; the 32 rows of two tiles are
// therefore assigned to them as 8 g + r and 8 g + 4 + r (the row order of a
// product's left operand is free).  Each wave forms the scores for itself.
// The staged tiles are double buffered: one barrier a chunk.  The decays are
// summed for 256 tokens at a time, one token a thread.
//
// Operand rounding (bf16): A, B, C are the inputs themselves.  2^{G_C-G} C, fp32,
// enters the state's sum as three bf16 pieces (the state is an fp32 result: one
// piece would leave it 2e-3 off).  Gamma o A B^T and the copy of X in the
// readout are rounded once to bf16 (out is bf16: each adds what the final
// rounding adds), or, with PR, taken in three pieces as well (the gradient of
// g is a difference of large sums of q . dq and k . dk).
#pragma once

#include <type_traits>

#include "operators.h"
#include "prism_common.h"

namespace prism {

constexpr int LA_NW = LA_PARTS, LA_NT = LA_NW * WAVE;

// ROWS x COLS of T in registers as 16-byte pieces; rows >= nv and columns >=
// nc (a multiple of the piece) are zeros.  Loads read the nearest valid piece
// in their place, so none sits in a branch.
template <typename E, int ROWS, int COLS>
struct LaTile {
  static constexpr int VN = 16 / (int)sizeof(E);
  static constexpr int VPR = COLS / VN;
  static constexpr int NU = ROWS * VPR;
  static constexpr int PER = (NU + LA_NT - 1) / LA_NT;
  uint4 v[PER];
  int nv, nc;
  __device__ inline void load(const E* g, long stride, int nvalid, int ncols, int tid) {
    nv = nvalid;
    nc = ncols;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int u = min(tid + p * LA_NT, NU - 1);
      const int r = min(u / VPR, nv - 1), c = min((u % VPR) * VN, nc - VN);
      v[p] = ld16(reinterpret_cast<const char*>(g) +
                  ((unsigned)r * (unsigned)stride + (unsigned)c) * (unsigned)sizeof(E));
    }
  }
  // (the fill is a uniform branch of its own: most chunks are whole)
  __device__ inline void store(E* s, int ld, int tid) {
    if (nv < ROWS || nc < COLS) {
#pragma unroll
      for (int p = 0; p < PER; ++p) {
        const int u = tid + p * LA_NT;
        const bool in = u / VPR < nv && (u % VPR) * VN < nc;
        v[p].x = in ? v[p].x : 0u;
        v[p].y = in ? v[p].y : 0u;
        v[p].z = in ? v[p].z : 0u;
        v[p].w = in ? v[p].w : 0u;
      }
    }
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int u = tid + p * LA_NT;
      if (NU % LA_NT == 0 || u < NU) st16(s + (u / VPR) * ld + (u % VPR) * VN, v[p]);
    }
  }
};

// 16-byte operands: KV values of one row at KV (lane / 16), so one instruction
// (bf16) or four (fp32) contract KG values.
template <typename E> struct La16;
template <> struct La16<bf16> {
  static constexpr int KV = 8, KG = 32, UPG = 2;
  typedef bf16x8 frag;
  __device__ static inline f32x4 mma(const frag& a, const frag& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  // row of an accumulator tile (u-th of its group) -> index in the group
  __device__ static inline int row(int u, int p) { return 8 * (p >> 2) + 4 * u + (p & 3); }
  // first of the four indexes that lane group g holds of tile u
  __device__ static inline int first(int u, int g) { return 8 * g + 4 * u; }
  // (index row(u, lane & 15), k at k0 + 8 g) of a tile stored [k][index]
  __device__ static inline frag trans(const bf16* p, int ld, int i0, int u, int k0, int lane, bool mapped) {
    const int j = lane & 15;
    const bf16* a = p + (k0 + 8 * (lane >> 4) + (j >> 2)) * ld + i0 + (mapped ? 8 * (j & 3) + 4 * u : 4 * (j & 3));
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a + 4 * ld));
    const short __attribute__((ext_vector_type(8))) w = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    frag f;
    __builtin_memcpy(&f, &w, 16);
    return f;
  }
};
template <> struct La16<float> {
  static constexpr int KV = 4, KG = 16, UPG = 1;
  typedef f32x4 frag;
  __device__ static inline f32x4 mma(const frag& a, const frag& b, f32x4 c) {
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
    return c;
  }
  __device__ static inline int row(int, int p) { return p; }
  __device__ static inline int first(int, int g) { return 4 * g; }
  __device__ static inline frag trans(const float* p, int ld, int i0, int, int k0, int lane, bool) {
    const float* a = p + (k0 + 4 * (lane >> 4)) * ld + i0 + (lane & 15);
    return frag{a[0], a[ld], a[2 * ld], a[3 * ld]};
  }
};

// x[0 .. KV) as NS operands whose sum is x to NS times E's precision
template <int NS>
__device__ inline void la_pieces(const float (&x)[8], bf16x8 (&f)[NS]) {
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = x[j];
#pragma unroll
  for (int k = 0; k < NS; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[k][j] = (bf16)y[j];
      if (k + 1 < NS) y[j] -= (float)f[k][j];
    }
}
template <int NS>
__device__ inline void la_pieces(const float (&x)[4], f32x4 (&f)[NS]) {
  static_assert(NS == 1, "fp32 is one piece");
  f[0] = f32x4{x[0], x[1], x[2], x[3]};
}

// log2 decay of a token; below -150 (exp underflows well before) it counts as
// -150: infinite values would leave inf - inf between two tokens behind them.
__device__ inline double la_log2(float g) { return (double)(g < -150.f ? -150.f : g) * 1.4426950408889634; }

template <typename E, int DA, int NCT, bool PR, bool OUT>
__global__ __launch_bounds__(LA_NT, 2) void la_pass_kernel(const LaArgs<E> args) {
  typedef La16<E> M;
  typedef typename M::frag frag;
  constexpr int CH = LA_CHUNK;
  constexpr bool HALF = sizeof(E) == 2;
  constexpr int NV = 64 * NCT;                    // columns of X
  constexpr int KG = M::KG, KV = M::KV, UPG = M::UPG;
  constexpr int AT = DA / 16, AG = DA / KG;       // tiles and groups of X's rows
  constexpr int TG = CH / KG;                     // groups of the chunk's tokens
  constexpr int NSU = HALF ? 3 : 1;               // pieces of the state's summand
  constexpr int NSX = HALF && PR ? 3 : 1;         // of X and of Gamma o A B^T in out
  constexpr int LA = ldpad<E>(DA), LC = ldpad<E>(NV);
  // (fp32 rows of 128 take too much LDS for two workgroups a CU with two buffers)
  constexpr int NBUF = OUT && !HALF && DA == 128 ? 1 : 2;
  constexpr int CPB = LA_NT / CH;                 // chunks of a batch of decays
  __shared__ __attribute__((aligned(16))) E sb_[NBUF][CH * LA];
  __shared__ __attribute__((aligned(16))) E sc_[NBUF][CH * LC];
  __shared__ __attribute__((aligned(16))) E sa_[NBUF][OUT ? CH * LA : 8];
  // per token: signed cumulative decays in its chunk (two floats), row and
  // column factors; per chunk: its decay, also as a log.  Two batches.
  __shared__ __attribute__((aligned(16))) float sgh[2][LA_NT], sgl[2][LA_NT], sra[2][LA_NT], srt[2][LA_NT];
  __shared__ float sgc[2][CPB];
  __shared__ double sgt[2][CPB];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, gq = lane >> 4;

  int id = xcd_swizzle((int)blockIdx.x, (int)gridDim.x);
  const LaRole<E>& R = args.r[id % args.nroles];
  id /= args.nroles;
  const int seg = id % args.nseg, bh = id / args.nseg;
  const int b = bh / args.H, h = bh % args.H;
  const int nc = R.dc;
  const bool rev = R.rev != 0;

  // the segment's tokens
  const int n = seq_len(args.cu, b, args.T);
  const int used = max(1, (n + args.seglen - 1) / args.seglen);   // segments with tokens (or one)
  if (seg >= used) return;
  const int s0 = seg * args.seglen, len = min(n - s0, args.seglen);
  const bool last = rev ? seg == 0 : seg == used - 1;   // of the pass: its state leaves
  if (!OUT && last) return;                             // nothing enters after it
  const long row0 = args.cu ? (long)args.cu[b] + s0 : s0;
  auto at = [&](const E* p, const Strides& s, int grp) {
    return p + ((args.cu ? 0 : b * s.b) + row0 * s.t + (long)(h / grp) * s.h);
  };
  const E* pa = OUT ? at(R.a, R.sa, R.ga) : nullptr;
  const E* pb = at(R.b, R.sb, R.gb);
  const E* pc = at(R.c, R.sc, R.gc);
  const float* pg = args.g + ((args.cu ? 0 : b * args.sg.b) + row0 * args.sg.t + h * args.sg.h);

  // X: tile (i, j) holds rows KG (i / UPG) + first(i % UPG, g) + r, column cw + 16 j + l16
  const int cw = wave * 16 * NCT;
  f32x4 X[AT][NCT];
#pragma unroll
  for (int i = 0; i < AT; ++i)
#pragma unroll
    for (int j = 0; j < NCT; ++j) X[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto state_each = [&](auto&& f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < AT; ++i)
#pragma unroll
      for (int j = 0; j < NCT; ++j) {
        const int a0 = KG * (i / UPG) + M::first(i % UPG, gq), c = cw + 16 * j + l16;
        if (a0 < R.da && c < nc) f(X[i][j], (long)a0 * R.xa + (long)c * R.xc);
      }
  };
  auto state_load = [&](const float* src) __attribute__((always_inline)) {
    state_each([&](f32x4& x, long o) __attribute__((always_inline)) {
      if (R.xa == 1) {
        x = *reinterpret_cast<const f32x4*>(src + o);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = src[o + (long)r * R.xa];
      }
    });
  };
  auto state_store = [&](float* dst) __attribute__((always_inline)) {
    state_each([&](f32x4& x, long o) __attribute__((always_inline)) {
      if (R.xa == 1) {
        *reinterpret_cast<f32x4*>(dst + o) = x;
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) dst[o + (long)r * R.xa] = x[r];
      }
    });
  };
  const long segoff = ((long)bh * args.nseg + seg) * args.DD;
  if (OUT) {
    if (args.nseg > 1)
      state_load(R.seg + segoff);
    else if (R.X0)
      state_load(R.X0 + (long)bh * args.DD);
  }

  // what the loop uses of the arguments, in registers
  const int sgn = rev ? -1 : 1;
  const float s_in = R.s_in;
  const bool wide = R.out32 != nullptr, dots = PR && R.e != nullptr;
  const int ot = (int)R.so.t, et = (int)R.se.t;
  const long o0 = (args.cu ? 0 : b * R.so.b) + row0 * R.so.t + h * R.so.h + cw + 4 * gq;
  E* const po = R.out + o0;
  float* const po32 = R.out32 + o0;
  const E* const pe =
      R.e + ((args.cu ? 0 : b * R.se.b) + row0 * R.se.t + (long)(h / R.ge) * R.se.h + cw + 4 * gq);
  float* const pd = R.edot + ((long)bh * LA_NW + wave) * args.T + s0;

  const int nch = (len + CH - 1) / CH;
  auto first_of = [&](int it) { return (rev ? nch - 1 - it : it) * CH; };
  LaTile<E, OUT ? CH : 16, DA> ta;
  LaTile<E, CH, DA> tb;
  LaTile<E, CH, NV> tc;
  auto fetch = [&](int t0) __attribute__((always_inline)) {
    const int nv = min(CH, len - t0);
    tb.load(pb + (long)t0 * R.sb.t, R.sb.t, nv, R.da, tid);
    if (OUT) ta.load(pa + (long)t0 * R.sa.t, R.sa.t, nv, R.da, tid);
    tc.load(pc + (long)t0 * R.sc.t, R.sc.t, nv, nc, tid);
  };
  // a thread's token in the batch of chunks from `it` on (tokens past the
  // segment decay by nothing), its cumulative decay in its chunk, its factors
  float gv = 0.f;
  const int bq = tid / CH, bj = tid % CH;
  auto batch_token = [&](int it) { return it + bq < nch ? first_of(it + bq) + bj : len; };
  auto batch_load = [&](int it) __attribute__((always_inline)) {
    gv = pg[(long)min(batch_token(it), len - 1) * args.sg.t];
  };
  auto batch_scan = [&](int it) __attribute__((always_inline)) {
    const int buf = (it / CPB) & 1;
    double x = batch_token(it) < len ? la_log2(gv) : 0.0;
#pragma unroll
    for (int o = 1; o < CH; o <<= 1) {
      const double y = __shfl_up(x, o, CH);
      if (bj >= o) x += y;
    }
    const double tot = __shfl(x, CH - 1, CH);
    const double y = rev ? -x : x;
    const float hi = (float)y;
    sgh[buf][tid] = hi;
    sgl[buf][tid] = (float)(y - (double)hi);
    const float from = __builtin_amdgcn_exp2f((float)x), to = __builtin_amdgcn_exp2f((float)(tot - x));
    sra[buf][tid] = R.s_row * (rev ? to : from);
    srt[buf][tid] = R.s_upd * (rev ? from : to);
    if (bj == 0) {
      sgc[buf][bq] = __builtin_amdgcn_exp2f((float)tot);
      sgt[buf][bq] = tot;
    }
  };

  double total = 0.0;
  if (nch > 0) {
    fetch(first_of(0));
    batch_load(0);
  }

  for (int it = 0; it < nch; ++it) {
    const int t0 = first_of(it), nv = min(CH, len - t0);
    if (it % CPB == 0) {
      batch_scan(it);
      batch_load(min(it + CPB, nch - 1));
    }
    const int bat = (it / CPB) & 1, boff = (it % CPB) * CH;
    const float *gh = &sgh[bat][boff], *gl = &sgl[bat][boff], *ra = &sra[bat][boff], *rt = &srt[bat][boff];
    E *sa = sa_[it % NBUF], *sb = sb_[it % NBUF], *sc = sc_[it % NBUF];
    tb.store(sb, LA, tid);
    if constexpr (OUT) ta.store(sa, LA, tid);
    tc.store(sc, LC, tid);
    __syncthreads();
    fetch(first_of(min(it + 1, nch - 1)));   // (past the end: the last chunk again)

    f32x4 acc[NCT][2];                       // out^T, [tile of columns][tile of t]
    if constexpr (OUT) {
      f32x4 p[2][2];                         // scores^T, [tile of i][tile of t]
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        p[0][j] = p[1][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < NCT; ++c) acc[c][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int k = 0; k < AG; ++k) {
        frag fa[2], fb[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          fa[j] = *reinterpret_cast<const frag*>(sa + (16 * j + l16) * LA + KV * gq + KG * k);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          fb[i] = *reinterpret_cast<const frag*>(sb + (KG * (i / UPG) + M::row(i % UPG, l16)) * LA + KV * gq + KG * k);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) p[i][j] = M::mma(fb[i], fa[j], p[i][j]);
#pragma unroll
        for (int c = 0; c < NCT; ++c) {
          float x[KV];
#pragma unroll
          for (int u = 0; u < UPG; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) x[4 * u + r] = X[UPG * k + u][c][r];
          frag fx[NSX];
          la_pieces(x, fx);
#pragma unroll
          for (int s = 0; s < NSX; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[c][j] = M::mma(fx[s], fa[j], acc[c][j]);
        }
      }
      // readout factors; Gamma and the mask
      frag fp[TG][2][NSX];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = 16 * j + l16;
        const float f = ra[t], hi = gh[t], lo = gl[t];
#pragma unroll
        for (int c = 0; c < NCT; ++c) acc[c][j] *= f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int i0 = KG * (i / UPG) + M::first(i % UPG, gq);
          const f32x4 ghi = *reinterpret_cast<const f32x4*>(gh + i0);
          const f32x4 glo = *reinterpret_cast<const f32x4*>(gl + i0);
          const int ahead = sgn * (t - i0);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float dif = hi - ghi[r];
            if (!HALF || PR) dif += lo - glo[r];
            // (masked: 2^-inf; a select of the exponent keeps this free of branches)
            dif = ahead >= sgn * r ? dif : -__builtin_inff();
            p[i][j][r] *= s_in * __builtin_amdgcn_exp2f(dif);
          }
        }
#pragma unroll
        for (int q = 0; q < TG; ++q) {
          float y[KV];
#pragma unroll
          for (int u = 0; u < UPG; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) y[4 * u + r] = p[q * UPG + u][j][r];
          la_pieces(y, fp[q][j]);
        }
      }
#pragma unroll
      for (int q = 0; q < TG; ++q)
#pragma unroll
        for (int c = 0; c < NCT; ++c) {
          const frag fc = M::trans(sc, LC, cw + 16 * c, 0, KG * q, lane, false);
#pragma unroll
          for (int s = 0; s < NSX; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[c][j] = M::mma(fc, fp[q][j][s], acc[c][j]);
        }
    }

    // X' = 2^{G_C} X + B^T (factor o C)
    const float gc = sgc[bat][it % CPB];
    if (!OUT) total += sgt[bat][it % CPB];
#pragma unroll
    for (int i = 0; i < AT; ++i)
#pragma unroll
      for (int j = 0; j < NCT; ++j) X[i][j] *= gc;
#pragma unroll
    for (int q = 0; q < TG; ++q) {
      frag fc[NCT][NSU];
#pragma unroll
      for (int c = 0; c < NCT; ++c) {
        const frag raw = M::trans(sc, LC, cw + 16 * c, 0, KG * q, lane, false);
        float x[KV];
#pragma unroll
        for (int v = 0; v < KV; v += 4) {
          const f32x4 f = *reinterpret_cast<const f32x4*>(rt + KG * q + KV * gq + v);
#pragma unroll
          for (int r = 0; r < 4; ++r) x[v + r] = f[r] * to_f(raw[v + r]);
        }
        la_pieces(x, fc[c]);
      }
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        const frag fb = M::trans(sb, LA, HALF ? KG * (i / UPG) : 16 * i, i % UPG, KG * q, lane, true);
#pragma unroll
        for (int s = 0; s < NSU; ++s)
#pragma unroll
          for (int c = 0; c < NCT; ++c) X[i][c] = M::mma(fb, fc[c][s], X[i][c]);
      }
    }

    // out, and its dots with the rows of e
    if constexpr (OUT) {
      auto out_each = [&](auto&& f) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < NCT; ++c)
            if (16 * j + l16 < nv && cw + 16 * c + 4 * gq < nc) f(j, c, (long)(t0 + 16 * j + l16));
      };
      if (wide)
        out_each([&](int j, int c, long t) { st_f4(po32 + t * ot + 16 * c, acc[c][j]); });
      else
        out_each([&](int j, int c, long t) { st_f4(po + t * ot + 16 * c, acc[c][j]); });
      if (dots) {
        float dot[2] = {0.f, 0.f};
        out_each([&](int j, int c, long t) {
          const f32x4 x = raw4_to_f(ld_raw4(pe + t * et + 16 * c));
          dot[j] += (acc[c][j][0] * x[0] + acc[c][j][1] * x[1]) + (acc[c][j][2] * x[2] + acc[c][j][3] * x[3]);
        });
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          dot[j] += __shfl_xor(dot[j], 16);
          dot[j] += __shfl_xor(dot[j], 32);
          if (gq == 0 && 16 * j + l16 < nv) pd[t0 + 16 * j + l16] = dot[j];
        }
      }
    }
    if (NBUF == 1) __syncthreads();
  }

  if (OUT) {
    if (last && R.fin) state_store(R.fin + (long)bh * args.DD);
  } else {
    state_store(R.seg + segoff);
    if (tid == 0) R.segdec[(long)bh * args.nseg + seg] = __builtin_amdgcn_exp2f((float)total);
  }
}

// Launch of one instance; DA and NCT by the operands' size.
template <typename E, int DA, int NCT, bool PR, bool OUT>
hipError_t la_launch(const LaArgs<E>& a, hipStream_t s) {
  const unsigned grid = (unsigned)((long)a.B * a.H * a.nseg * a.nroles);
  hipLaunchKernelGGL((la_pass_kernel<E, DA, NCT, PR, OUT>), dim3(grid), dim3(LA_NT), 0, s, a);
  return hipGetLastError();
}

}  // namespace prism
