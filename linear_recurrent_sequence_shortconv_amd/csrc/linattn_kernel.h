// Linear attention with a decay for each head, over chunks of 32 tokens
// (LaRole in operators.h has the formula).  With u_t the log2 decay from the
// chunk's entry to token t in the direction of the pass (forward: G_t, the sum
// of the decays up to t; reverse: G_C - G_t), a chunk entered with state X gives
//   out_t = s_row 2^{u_t} A_t (X + s_upd sum_{i <= t} 2^{-u_i} B_i C_i^T)
//   X'    = 2^{G_C} (X + s_upd sum_i 2^{-u_i} B_i C_i^T)
// (reverse: i >= t; s_row s_upd = s_in).  X is kept without the decay: with F
// the log2 decay since X was last brought up to date, the registers hold
// 2^{-F} X, rows are read out with 2^{F + u_t} and added with 2^{-(F + u_i)},
// so that a chunk costs no pass over X and no decay between pairs of tokens.
// That holds while F + u stays within +-48; X is brought up to date (F = 0)
// every 256 tokens, 128 where 256 leave this range, or when a chunk would leave
// it, and a chunk that leaves it by itself (a decay by 2^-48 within 32 tokens, a
// reset) takes the form with
// Gamma_ti = 2^{u_t - u_i} on each pair and 2^{G_C - u_i} on each added row.
//
// One workgroup of four waves carries X over its segment's chunks; a wave owns
// 16 NCT of its columns (all DA rows) in fp32 accumulators.  The tiles of A, B
// and C are fetched one chunk ahead in registers and staged in LDS, the only
// data the waves share: with a column of out^T and of X in one wave, what one
// product leaves in accumulators is the next product's operand in the same
// lanes, so neither X nor the scores pass through LDS.  An accumulator
// tile holds rows 4 g + r (g = lane / 16) of one column, a k-contiguous operand
// 8 consecutive k (bf16) of one row at 8 g; the 32 state rows of two tiles are
// therefore assigned to them as 8 g + r and 8 g + 4 + r (the row order of a
// product's left operand is free), while tokens, which both operands of their
// products read transposed, are contracted in the accumulators' order (in the
// other one the scores' reads of B met in LDS banks: 4 of 10 cycles).  Each
// wave forms the scores for itself.
// The staged tiles are double buffered: one barrier a chunk.  The decays are
// summed for 256 tokens at a time, one token a thread.
//
// Bound by the latency chain of a chunk, not by one unit.  bf16, 128 x 128, in
// cycles: 5800 for a workgroup alone on a CU, 7200 for two together, of which
// scores and readout take 1700, their product with C 630, the update of X 2000,
// the rest waits for loads, LDS stores, barrier and decays; matrix units are
// busy 25 %, the vector ALU 30 to 40 %, LDS 24 %.  8 x 2048 tokens, 16 heads of
// 128: 83 us for out (4 reads and writes of 67 MB; 3.2 TB/s), 36 for the states
// before it; with its dots (a gradient and the rows for dg) 118 each.
// The sizes taken: chunks of 32 tokens (64: 88 us where 32 took 82: more
// products, fewer workgroups a CU), 32 columns of X a wave and four waves (eight
// waves of 16 columns: 110), tiles fetched one chunk ahead (two: no gain, for
// more registers).
//
// Operand rounding (bf16): A, B, C are the inputs themselves.  2^{-(F+u)} C, fp32,
// enters the state's sum as three bf16 pieces where the state is an fp32 result
// (one piece would leave it 2e-3 off, two 3e-6), as two where only out, bf16,
// comes of it.  The scaled scores and the copy of X in the
// readout are rounded once to bf16 (out is bf16: each adds what the final
// rounding adds), or, with PR, taken in three pieces as well (the gradient of
// g is a difference of large sums of q . dq and k . dk: 2048 tokens, with two
// pieces dg is off by 1.1e-5, with three by 6e-7, at 341 and 358 us for the
// whole backward pass of 8 x 2048 tokens, 16 heads).
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
  unsigned row[PER], col[PER];   // byte offsets
  unsigned step;
  int nv, nc;
  __device__ inline void place(long stride, int ncols, int tid) {
    nc = ncols;
    step = (unsigned)stride * (unsigned)sizeof(E);
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int u = min(tid + p * LA_NT, NU - 1);
      row[p] = (unsigned)(u / VPR) * step;
      col[p] = (unsigned)min((u % VPR) * VN, nc - VN) * (unsigned)sizeof(E);
    }
  }
  __device__ inline void load(const E* g, int nvalid) {
    nv = nvalid;
    const unsigned end = (unsigned)(nvalid - 1) * step;
#pragma unroll
    for (int p = 0; p < PER; ++p) v[p] = ld16(reinterpret_cast<const char*>(g) + (min(row[p], end) + col[p]));
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

// 16-byte operands: KV values of one row in each lane, so one instruction (bf16)
// or four (fp32) contract KG values.  A group of KG tokens is contracted in the
// order of the accumulators: lane group g has tokens 16 u + 4 g + r (u-th tile).
// A group of KG state rows in the order of a k-contiguous operand: 8 g + j.
template <typename E> struct La16;
template <> struct La16<bf16> {
  static constexpr int KV = 8, KG = 32, UPG = 2;
  typedef bf16x8 frag;
  __device__ static inline f32x4 mma(const frag& a, const frag& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  // first of the four state rows that lane group g holds of a group's tile u
  __device__ static inline int first(int u, int g) { return 8 * g + 4 * u; }
  // Column i0 + (lane & 15) of a tile stored [token][column], at the group's
  // tokens from k0 on; STATE: column i0 + the state row of (lane & 15) in tile u.
  template <bool STATE>
  __device__ static inline frag trans(const bf16* p, int ld, int i0, int u, int k0, int lane) {
    const int j = lane & 15;
    const bf16* a = p + (k0 + 4 * (lane >> 4) + (j >> 2)) * ld + i0 + (STATE ? 8 * (j & 3) + 4 * u : 4 * (j & 3));
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a + 16 * ld));
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
  __device__ static inline int first(int, int g) { return 4 * g; }
  template <bool STATE>
  __device__ static inline frag trans(const float* p, int ld, int i0, int, int k0, int lane) {
    const float* a = p + (k0 + 4 * (lane >> 4)) * ld + i0 + (lane & 15);
    return frag{a[0], a[ld], a[2 * ld], a[3 * ld]};
  }
};

// x[0 .. KV) as NS operands whose sum is x to NS times E's precision
template <int NS>
__device__ inline void la_pieces(const float (&x)[8], bf16x8 (&f)[NS]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    float a = x[j], b = x[j + 1];
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      // (a pair is rounded by one instruction and taken apart by two)
      const bf16x2 w = __builtin_convertvector((f32x2{a, b}), bf16x2);
      f[k][j] = w[0];
      f[k][j + 1] = w[1];
      if (k + 1 < NS) {
        const unsigned u = __builtin_bit_cast(unsigned, w);
        a -= __uint_as_float(u << 16);
        b -= __uint_as_float(u & 0xffff0000u);
      }
    }
  }
}
template <int NS>
__device__ inline void la_pieces(const float (&x)[4], f32x4 (&f)[NS]) {
  static_assert(NS == 1, "fp32 is one piece");
  f[0] = f32x4{x[0], x[1], x[2], x[3]};
}

// Four values at element `at` of a buffer from a wave-uniform address; nothing
// is written where the byte offset passes the buffer's 2^31 - 1 bytes, as that
// of LA_NOWHERE does (a chunk's own are under 32 rows of 2^22 elements).
constexpr unsigned LA_NOWHERE = 0x60000000u;   // (2 and 4 times it, mod 2^32, are 2^31 or more)
__device__ inline __amdgpu_buffer_rsrc_t la_buffer(void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(p, 0, 0x7fffffff, 0x00020000);
}
__device__ inline void la_store4(__amdgpu_buffer_rsrc_t p, unsigned at, const f32x4& x, float) {
  typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), p, at * 4u, 0, 0);
}
__device__ inline void la_store4(__amdgpu_buffer_rsrc_t p, unsigned at, const f32x4& x, bf16) {
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  const bf16 b[4] = {(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3]};
  u32x2 w;
  __builtin_memcpy(&w, b, 8);
  __builtin_amdgcn_raw_buffer_store_b64(w, p, at * 2u, 0, 0);
}

// log2 decay of a token; below -150 (exp underflows well before) it counts as
// -150: infinite values would leave inf - inf between two tokens behind them.
__device__ inline double la_log2(float g) { return (double)(g < -150.f ? -150.f : g) * 1.4426950408889634; }

// 2^e for an exponent in fp64: the whole part goes to the exponent bits, so the
// factor is good to 2^-23 however far e is from 0 (an fp32 e of 80 is not known
// to better than 4e-6).
__device__ inline float la_exp2(double e) {
  const double n = rint(e);
  return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f((float)(e - n)), (int)fmin(fmax(n, -400.0), 400.0));
}

// log2 range of the factors kept without the decay.  They enlarge sums of
// products by up to 2^48, so that those below 2^76 stay finite in fp32.  (With 80
// a v k^T of 2^48 overflows; 8 x 2048 tokens, 16 heads of 128, learned decays of a
// gate near 0.86, backward: 355 us with 80, 359 with 48, 368 with 40 and no halves
// of a batch; of a gate near 0.5: 371 with 80, 377 with 48.)
constexpr double LA_RANGE = 48.0;

// Inclusive prefix sum over each 32 lanes: shifts within rows of 16 lanes, then
// the first row's sum to the second (lane 15 to the row behind it).
template <int CTRL, int ROWS>
__device__ inline double la_dpp(double x) {
  const long long b = __builtin_bit_cast(long long, x);
  const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)b, CTRL, ROWS, 0xf, ROWS == 0xf);
  const unsigned hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, ROWS, 0xf, ROWS == 0xf);
  return __builtin_bit_cast(double, (long long)(((unsigned long long)hi << 32) | lo));
}
__device__ inline double la_scan32(double x) {
  x += la_dpp<0x111, 0xf>(x);
  x += la_dpp<0x112, 0xf>(x);
  x += la_dpp<0x114, 0xf>(x);
  x += la_dpp<0x118, 0xf>(x);
  x += la_dpp<0x142, 0xa>(x);
  return x;
}
// Sum over each 32 lanes, in the last of them
__device__ inline float la_sum32(float x) {
  x = row16_sum(x);
  const int b = __builtin_bit_cast(int, x);
  return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, b, 0x142, 0xa, 0xf, false));
}

template <typename E, int DA, int NCT, bool PR, bool OUT, int PIECES>
__global__ __launch_bounds__(LA_NT, 2) void la_pass_kernel(const LaArgs<E> args) {
  typedef La16<E> M;
  typedef typename M::frag frag;
  constexpr int CH = LA_CHUNK;
  constexpr bool HALF = sizeof(E) == 2;
  constexpr int NV = 64 * NCT;                    // columns of X
  constexpr int KG = M::KG, KV = M::KV, UPG = M::UPG;
  constexpr int AT = DA / 16, AG = DA / KG;       // tiles and groups of X's rows
  constexpr int TG = CH / KG;                     // groups of the chunk's tokens
  constexpr int NSU = HALF ? PIECES : 1;          // pieces of the state's summand
  constexpr int NSX = HALF && PR ? 3 : 1;         // of X and of Gamma o A B^T in out
  constexpr int LA = ldpad<E>(DA), LC = ldpad<E>(NV);
  // (fp32 rows of 128 take too much LDS for two workgroups a CU with two buffers)
  constexpr int NBUF = OUT && !HALF && DA == 128 ? 1 : 2;
  constexpr int CPB = LA_NT / CH;                 // chunks of a batch of decays
  __shared__ __attribute__((aligned(16))) E sb_[NBUF][CH * LA];
  __shared__ __attribute__((aligned(16))) E sc_[NBUF][CH * LC];
  __shared__ __attribute__((aligned(16))) E sa_[NBUF][OUT ? CH * LA : 8];
  // per token: u (two floats), readout and update factors; per chunk: factors of
  // X before its readout and before its update, and whether it takes the form
  // with Gamma.  Two batches.
  __shared__ __attribute__((aligned(16))) float suh[2][LA_NT], sul[2][LA_NT], sra[2][LA_NT], srt[2][LA_NT];
  __shared__ float sm0[2][CPB], sm1[2][CPB];
  __shared__ int strong[2][CPB];
  __shared__ double stot[CPB];
  __shared__ float spos[CPB];
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
  __shared__ int sseq[LA_NW];
  long first = 0;
  int n = args.T;
  if (args.cu) la_sequence(args.cu, args.N, args.T, b, tid, sseq, first, n);
  const int used = max(1, (n + args.seglen - 1) / args.seglen);   // segments with tokens (or one)
  if (seg >= used) return;
  const int s0 = seg * args.seglen, len = min(n - s0, args.seglen);
  const bool last = rev ? seg == 0 : seg == used - 1;   // of the pass: its state leaves
  if (!OUT && last) return;                             // nothing enters after it
  const long row0 = first + s0;
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
    if (args.nseg > 1 && args.joined) {
      state_load(R.seg + segoff);
    } else {
      if (R.X0) state_load(R.X0 + (long)bh * args.DD);
      // the segments before this one (in the pass's direction), by their own states
      for (int i = 0; i < (rev ? used - 1 - seg : seg); ++i) {
        const long s = (long)bh * args.nseg + (rev ? used - 1 - i : i);
        const float dec = R.segdec[s];
        const float* src = R.seg + s * args.DD;
        state_each([&](f32x4& x, long o) __attribute__((always_inline)) {
          if (R.xa == 1) {
            x = x * dec + *reinterpret_cast<const f32x4*>(src + o);
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = fmaf(x[r], dec, src[o + (long)r * R.xa]);
          }
        });
      }
    }
  }

  // what the loop uses of the arguments, in registers
  const float s_in = R.s_in;
  const bool wide = R.out32 != nullptr, dots = PR && R.e != nullptr;
  const long ot = R.so.t, et = R.se.t;
  const long o0 = (args.cu ? 0 : b * R.so.b) + row0 * ot + h * R.so.h;
  const long e0 = (args.cu ? 0 : b * R.se.b) + row0 * et + (long)(h / R.ge) * R.se.h;
  float* const pd = R.edot + ((long)h * LA_NW + wave) * args.rows + ((args.cu ? 0 : (long)b * args.T) + row0);
  // the lane's place in a chunk's output and e rows (elements)
  unsigned ol[2], el[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    ol[j] = (unsigned)(16 * j + l16) * (unsigned)ot + (unsigned)(cw + 4 * gq);
    el[j] = (unsigned)(16 * j + l16) * (unsigned)et + (unsigned)(cw + 4 * gq);
  }
  // masked scores: bits kept of each value of p[i][j] (its i against its t)
  auto keep = [&](int i, int j, int r) {
    const int ii = 16 * i + 4 * gq + r, t = 16 * j + l16;
    return rev ? ii >= t : ii <= t;
  };

  const int nch = (len + CH - 1) / CH;
  auto first_of = [&](int it) { return (rev ? nch - 1 - it : it) * CH; };
  LaTile<E, OUT ? CH : 16, DA> ta;
  LaTile<E, CH, DA> tb;
  LaTile<E, CH, NV> tc;
  if (OUT) ta.place(R.sa.t, R.da, tid);
  tb.place(R.sb.t, R.da, tid);
  tc.place(R.sc.t, nc, tid);
  auto fetch = [&](int t0) __attribute__((always_inline)) {
    const int nv = min(CH, len - t0);
    tb.load(pb + (long)t0 * R.sb.t, nv);
    if (OUT) ta.load(pa + (long)t0 * R.sa.t, nv);
    tc.load(pc + (long)t0 * R.sc.t, nv);
  };
  // a thread's token in the batch of chunks from `it` on (tokens past the
  // segment decay by nothing), and its factors
  float gv = 0.f;
  double F = 0.0, total = 0.0;
  const int bq = tid / CH, bj = tid % CH;
  auto batch_token = [&](int it) { return it + bq < nch ? first_of(it + bq) + bj : len; };
  auto batch_load = [&](int it) __attribute__((always_inline)) {
    gv = pg[(long)min(batch_token(it), len - 1) * args.sg.t];
  };
  auto batch_scan = [&](int it) __attribute__((always_inline)) {
    const int buf = (it / CPB) & 1;
    double x = batch_token(it) < len ? la_log2(gv) : 0.0;
    float pos = (float)fmax(x, 0.0);
    x = la_scan32(x);
    pos = la_sum32(pos);
    const double tot = __shfl(x, CH - 1, CH);
    const double u = rev ? tot - x : x;
    if (bj == CH - 1) {
      stot[bq] = tot;
      spos[bq] = pos;
    }
    __syncthreads();
    // Every batch starts with X up to date.  u of a chunk lies between its sum
    // less its positive part and its positive part.
    constexpr int HB = CPB / 2;
    double f = 0.0, sums[2] = {0.0, 0.0};   // of each half of the batch
    float ups[2] = {0.f, 0.f};
#pragma unroll
    for (int q = 0; q < CPB; ++q) {
      const double t = stot[q];
      if (q < bq) f += t;
      sums[q / HB] += t;
      ups[q / HB] += spos[q];
    }
    auto within = [](double sum, float up) { return up <= LA_RANGE && sum - up >= -LA_RANGE; };
    const double sum = sums[0] + sums[1];
    double m0 = bq == 0 ? F : 0.0, m1 = 0.0;   // log2 factors of X at this thread's chunk
    bool st = false;
    total += sum;
    if (within(sum, ups[0] + ups[1])) {
      F = sum;
    } else if (within(sums[0], ups[0]) && within(sums[1], ups[1])) {
      if (bq == HB) m0 = sums[0];
      if (bq >= HB) f -= sums[0];
      F = sums[1];
    } else {
      // chunk after chunk (every thread alike).  (A NaN takes the strong form,
      // which spreads it as the recurrence would.)
#pragma unroll 1
      for (int q = 0; q < CPB; ++q) {
        const double t = stot[q], hi = spos[q], lo = t - hi;
        double pre = 0.0, post = 0.0;
        bool s = false;
        if (q == 0 || !(F + lo >= -LA_RANGE && F + hi <= LA_RANGE)) {
          pre = F;
          F = 0.0;
          s = !(lo >= -LA_RANGE && hi <= LA_RANGE);
          if (s) post = t;
        }
        if (q == bq) {
          f = F;
          m0 = pre;
          m1 = post;
          st = s;
        }
        if (!s) F += t;
      }
    }
    const float uh = (float)u;
    suh[buf][tid] = uh;
    sul[buf][tid] = (float)(u - (double)uh);
    sra[buf][tid] = R.s_row * la_exp2(f + u);
    srt[buf][tid] = R.s_upd * la_exp2((st ? tot : -f) - u);
    if (bj == 0) {
      sm0[buf][bq] = la_exp2(m0);
      sm1[buf][bq] = la_exp2(m1);
      strong[buf][bq] = st;
    }
  };
  auto state_scale = [&](float m) __attribute__((always_inline)) {
    if (m != 1.f) {
#pragma unroll
      for (int i = 0; i < AT; ++i)
#pragma unroll
        for (int j = 0; j < NCT; ++j) X[i][j] *= m;
    }
  };

  if (nch > 0) {
    fetch(first_of(0));
    batch_load(0);
  }
  // X here, not at its first use in the loop: a wait there for loads from
  // before the loop would in every chunk wait for the stores of the one before
#pragma unroll
  for (int i = 0; i < AT; ++i)
#pragma unroll
    for (int j = 0; j < NCT; ++j) asm volatile("" : "+v"(X[i][j]));

  for (int it = 0; it < nch; ++it) {
    const int t0 = first_of(it), nv = min(CH, len - t0);
    if (it % CPB == 0) {
      batch_scan(it);
      batch_load(min(it + CPB, nch - 1));
    }
    const int bat = (it / CPB) & 1, boff = (it % CPB) * CH;
    const float *uh = &suh[bat][boff], *ul = &sul[bat][boff], *ra = &sra[bat][boff], *rt = &srt[bat][boff];
    E *sa = sa_[it % NBUF], *sb = sb_[it % NBUF], *sc = sc_[it % NBUF];
    tb.store(sb, LA, tid);
    if constexpr (OUT) ta.store(sa, LA, tid);
    tc.store(sc, LC, tid);
    __syncthreads();
    fetch(first_of(min(it + 1, nch - 1)));   // (past the end: the last chunk again)
    const bool st = __builtin_amdgcn_readfirstlane(strong[bat][it % CPB]) != 0;
    state_scale(sm0[bat][it % CPB]);

    f32x4 acc[NCT][2];                       // out^T, [tile of columns][tile of t]
    if constexpr (OUT) {
      f32x4 p[2][2];                         // scores^T, [tile of i][tile of t]
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        p[0][j] = p[1][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < NCT; ++c) acc[c][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      // (every operand requested before the first product: read as they are
      // used, each group of products would wait out an LDS access)
      frag fa[AG][2], fb[AG][2];
#pragma unroll
      for (int k = 0; k < AG; ++k) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          fa[k][j] = *reinterpret_cast<const frag*>(sa + (16 * j + l16) * LA + KV * gq + KG * k);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          fb[k][i] =
              *reinterpret_cast<const frag*>(sb + (16 * i + l16) * LA + KV * gq + KG * k);
      }
      if (HALF) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < AG; ++k) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) p[i][j] = M::mma(fb[k][i], fa[k][j], p[i][j]);
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
            for (int j = 0; j < 2; ++j) acc[c][j] = M::mma(fx[s], fa[k][j], acc[c][j]);
        }
      }
      // factors of the added rows (or Gamma), the mask, operands
      float fin[2];
      if (!st) {
        fin[0] = ra[l16];
        fin[1] = ra[16 + l16];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const f32x4 f = *reinterpret_cast<const f32x4*>(rt + 16 * i + 4 * gq);
#pragma unroll
          for (int j = 0; j < 2; ++j) p[i][j] *= f;
        }
      } else {
        fin[0] = fin[1] = 1.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float f = ra[16 * j + l16], hi = uh[16 * j + l16], lo = ul[16 * j + l16];
#pragma unroll
          for (int c = 0; c < NCT; ++c) acc[c][j] *= f;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int i0 = 16 * i + 4 * gq;
            const f32x4 vh = *reinterpret_cast<const f32x4*>(uh + i0), vl = *reinterpret_cast<const f32x4*>(ul + i0);
#pragma unroll
            for (int r = 0; r < 4; ++r)
              p[i][j][r] *= s_in * __builtin_amdgcn_exp2f((hi - vh[r]) + (lo - vl[r]));
          }
        }
      }
      frag fp[TG][2][NSX];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < TG; ++q) {
          float y[KV];
#pragma unroll
          for (int u = 0; u < UPG; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              y[4 * u + r] = keep(q * UPG + u, j, r) ? p[q * UPG + u][j][r] : 0.f;
          la_pieces(y, fp[q][j]);
        }
#pragma unroll
      for (int q = 0; q < TG; ++q)
#pragma unroll
        for (int c = 0; c < NCT; ++c) {
          const frag fc = M::template trans<false>(sc, LC, cw + 16 * c, 0, KG * q, lane);
#pragma unroll
          for (int s = 0; s < NSX; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[c][j] = M::mma(fc, fp[q][j][s], acc[c][j]);
        }
#pragma unroll
      for (int c = 0; c < NCT; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[c][j] *= fin[j];
    }

    // the chunk's rows into X
    state_scale(sm1[bat][it % CPB]);
#pragma unroll
    for (int q = 0; q < TG; ++q) {
      frag raw[NCT], fc[NCT][NSU], fb[HALF ? AT : 1];
#pragma unroll
      for (int c = 0; c < NCT; ++c) raw[c] = M::template trans<false>(sc, LC, cw + 16 * c, 0, KG * q, lane);
      f32x4 f[KV / 4];
#pragma unroll
      for (int v = 0; v < KV / 4; ++v) f[v] = *reinterpret_cast<const f32x4*>(rt + KG * q + 16 * v + 4 * gq);
      if (HALF) {
#pragma unroll
        for (int i = 0; i < AT; ++i) fb[HALF ? i : 0] = M::template trans<true>(sb, LA, KG * (i / UPG), i % UPG, KG * q, lane);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int c = 0; c < NCT; ++c) {
        float x[KV];
#pragma unroll
        for (int v = 0; v < KV; ++v) x[v] = f[v / 4][v % 4] * to_f(raw[c][v]);
        la_pieces(x, fc[c]);
      }
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        if (!HALF) fb[0] = M::template trans<true>(sb, LA, 16 * i, 0, KG * q, lane);
#pragma unroll
        for (int s = 0; s < NSU; ++s)
#pragma unroll
          for (int c = 0; c < NCT; ++c) X[i][c] = M::mma(fb[HALF ? i : 0], fc[c][s], X[i][c]);
      }
    }

    // out, and its dots with the rows of e
    if constexpr (OUT) {
      // (buffer stores, whose out-of-range lanes write nothing: a branch around
      // a store hides their number from the wait for the next tiles' loads,
      // which would then wait for the stores as well)
      unsigned os[2][NCT];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int c = 0; c < NCT; ++c)
          os[j][c] = (16 * j + l16 < nv && cw + 16 * c + 4 * gq < nc) ? ol[j] + 16 * c : LA_NOWHERE;
      if (wide) {
        const auto po = la_buffer(R.out32 + (o0 + t0 * ot));
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < NCT; ++c) la_store4(po, os[j][c], acc[c][j], 0.f);
      } else {
        const auto po = la_buffer(R.out + (o0 + t0 * ot));
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < NCT; ++c) la_store4(po, os[j][c], acc[c][j], E(0.f));
      }
      if (dots) {
        const E* const pe = R.e + (e0 + t0 * et);
        float dot[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < NCT; ++c)
            if (16 * j + l16 < nv && cw + 16 * c + 4 * gq < nc) {
              const f32x4 x = raw4_to_f(ld_raw4(pe + (el[j] + 16 * c)));
              dot[j] += (acc[c][j][0] * x[0] + acc[c][j][1] * x[1]) + (acc[c][j][2] * x[2] + acc[c][j][3] * x[3]);
            }
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

  state_scale(la_exp2(F));
  if (OUT) {
    if (last && R.fin) state_store(R.fin + (long)bh * args.DD);
  } else {
    state_store(R.seg + segoff);
    if (tid == 0) R.segdec[(long)bh * args.nseg + seg] = la_exp2(total);
  }
}

// Launch of one instance; DA and NCT by the operands' size.
template <typename E, int DA, int NCT, bool PR, bool OUT, int PIECES>
hipError_t la_launch(const LaArgs<E>& a, hipStream_t s) {
  const unsigned grid = (unsigned)((long)a.B * a.H * a.nseg * a.nroles);
  hipLaunchKernelGGL((la_pass_kernel<E, DA, NCT, PR, OUT, PIECES>), dim3(grid), dim3(LA_NT), 0, s, a);
  return hipGetLastError();
}

}  // namespace prism
