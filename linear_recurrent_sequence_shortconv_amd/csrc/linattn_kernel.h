// Linear attention with a decay for each head, over chunks of CH tokens
// (LaRole in operators.h has the formula).  In a chunk entered with state X,
// with the cumulative log2 decays G_1 .. G_C of its tokens (Gamma_ti = 2^(G_t - G_i)):
//   out = s_in (Gamma o A B^T)_{i<=t} C + s_row 2^G o (A X)
//   X'  = 2^{G_C} X + s_upd B^T (2^{G_C - G} o C)
// (reverse: i >= t, Gamma_ti = 2^(G_i - G_t), 2^{G_C - G_t} and 2^{G_i}).
//
// One workgroup carries a slice of NV columns of X in fp32 accumulators over
// its segment's chunks: the tiles of A, B, C are fetched one chunk ahead in
// registers and staged in LDS, out is formed transposed (a lane then holds
// four consecutive values of one token, stored as one piece), and X goes back
// to LDS once a chunk as the operand of the next readout.
//
// Operand rounding (bf16): A, B, C are the inputs themselves.  2^{G_C-G} C, fp32,
// enters the state's sum as three bf16 pieces (the state is an fp32 result: one
// piece would leave it 2e-3 off).  Gamma o A B^T and the copy of X in the
// readout are rounded once to bf16 (out is bf16: each adds what the final
// rounding adds), or, with PR, taken in three pieces as well (the gradient of
// g is a difference of large sums of q . dq and k . dk).
#pragma once

#include "operators.h"
#include "prism_common.h"

namespace prism {

constexpr int LA_NW = 4, LA_NT = LA_NW * WAVE;

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
  __device__ inline uint4 get(int p, int r, int c) const {
    uint4 w = v[p];
    asm volatile("" : "+v"(w.x), "+v"(w.y), "+v"(w.z), "+v"(w.w));
    return (r < nv && c < nc) ? w : uint4{0u, 0u, 0u, 0u};
  }
  template <typename F>
  __device__ inline void each(int tid, F&& f) const {
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int u = tid + p * LA_NT;
      const int r = u / VPR, c = (u % VPR) * VN;
      if (NU % LA_NT == 0 || u < NU) f(r, c, get(p, r, c));
    }
  }
  __device__ inline void store(E* s, int ld, int tid) const {
    each(tid, [&](int r, int c, const uint4& w) { st16(s + r * ld + c, w); });
  }
};

// x as NS pieces of type E: p[0] + p[1] + .. = x to NS times E's precision
template <typename E, int NS>
__device__ inline void pieces(float x, E (&p)[NS]) {
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    p[i] = to_t<E>(x);
    x -= to_f(p[i]);
  }
}

template <typename E, int DA, int NV, int CH, bool PR, bool OUT>
struct LaShape {
  static constexpr bool HALF = sizeof(E) == 2;
  static constexpr int NSU = HALF ? 3 : 1;              // pieces of the state's summand
  static constexpr int NSX = HALF && PR ? 3 : 1;        // of X in the readout
  static constexpr int NSP = HALF && PR ? 3 : 1;        // of Gamma o A B^T
  static constexpr int LA = ldpad_min<E>(DA), LC = ldpad_min<E>(NV), LP = ldpad_min<E>(CH);
  struct Lds {
    alignas(16) E b[CH * LA];
    alignas(16) E cs[NSU][CH * LC];
    float gh[2][CH], gl[2][CH], ra[2][CH], rc[2][CH], gc[2];
    // (only where outputs are formed)
    alignas(16) E a[OUT ? CH * LA : 8];
    alignas(16) E c[OUT ? CH * LC : 8];
    alignas(16) E p[OUT ? NSP : 1][OUT ? CH * LP : 8];
    alignas(16) E x[OUT ? NSX : 1][OUT ? NV * LA : 8];
  };
};

// log2 decay of a token; below -150 (exp underflows well before) it counts as
// -150: infinite values would leave inf - inf between two tokens behind them.
__device__ inline double la_log2(float g) { return (double)(g < -150.f ? -150.f : g) * 1.4426950408889634; }

template <typename E, int DA, int NV, int CH, bool PR, bool OUT>
__global__ __launch_bounds__(LA_NT) void la_pass_kernel(const LaArgs<E> args) {
  typedef LaShape<E, DA, NV, CH, PR, OUT> SH;
  constexpr int LA = SH::LA, LC = SH::LC, LP = SH::LP;
  __shared__ typename SH::Lds S;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  int id = xcd_swizzle((int)blockIdx.x, (int)gridDim.x);
  const int slice = id % args.nslice;
  id /= args.nslice;
  const LaRole<E>& R = args.r[id % args.nroles];
  id /= args.nroles;
  const int seg = id % args.nseg, bh = id / args.nseg;
  const int b = bh / args.H, h = bh % args.H;
  const int c0 = slice * NV, nc = min(NV, R.dc - c0);
  if (nc <= 0) return;
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
  const E* pc = at(R.c, R.sc, R.gc) + c0;
  const float* pg = args.g + ((args.cu ? 0 : b * args.sg.b) + row0 * args.sg.t + h * args.sg.h);

  // X: columns c0 .. c0 + NV - 1 of the entering state
  Acc<DA, NV, LA_NW> X;
  X.zero();
  auto state_at = [&](int a, int c) { return (long)a * R.xa + (long)(c0 + c) * R.xc; };
  auto state_load = [&](const float* src) {
    for_tiles_ij(X, wave, lane, [&](int i, int j, int a0, int c, const f32x4&) {
      if (a0 < R.da && c < nc) {
        f32x4 w;
        if (R.xa == 1) {
          w = *reinterpret_cast<const f32x4*>(src + state_at(a0, c));
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) w[r] = src[state_at(a0 + r, c)];
        }
        X.v[i][j] = w;
      }
    });
  };
  auto state_store = [&](float* dst) {
    for_tiles(X, wave, lane, [&](int a0, int c, const f32x4& w) {
      if (a0 < R.da && c < nc) {
        if (R.xa == 1) {
          *reinterpret_cast<f32x4*>(dst + state_at(a0, c)) = w;
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) dst[state_at(a0 + r, c)] = w[r];
        }
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
  auto state_to_lds = [&]() {
    for_tiles(X, wave, lane, [&](int a0, int c, const f32x4& w) {
      E pc4[4][SH::NSX];
#pragma unroll
      for (int r = 0; r < 4; ++r) pieces(w[r], pc4[r]);
#pragma unroll
      for (int k = 0; k < SH::NSX; ++k) {
        const E x4[4] = {pc4[0][k], pc4[1][k], pc4[2][k], pc4[3][k]};
        st4(&S.x[k][c * LA + a0], x4);
      }
    });
  };

  const int nch = (len + CH - 1) / CH;
  auto first_of = [&](int it) { return (rev ? nch - 1 - it : it) * CH; };
  LaTile<E, CH, DA> ta, tb;
  LaTile<E, CH, NV> tc;
  float gv = 0.f;
  auto fetch = [&](int t0) {
    const int nv = min(CH, len - t0);
    if (OUT) ta.load(pa + (long)t0 * R.sa.t, R.sa.t, nv, R.da, tid);
    tb.load(pb + (long)t0 * R.sb.t, R.sb.t, nv, R.da, tid);
    tc.load(pc + (long)t0 * R.sc.t, R.sc.t, nv, nc, tid);
    if (wave == 0) gv = pg[(long)(t0 + min(lane, nv - 1)) * args.sg.t];
  };
  // cumulative decays of a chunk of nv tokens (wave 0; tokens past the chunk
  // decay by nothing), and the factors of its rows
  double total = 0.0;
  auto scan = [&](int buf, int nv) {
    double x = lane < nv ? la_log2(gv) : 0.0;
#pragma unroll
    for (int o = 1; o < CH; o <<= 1) {
      const double y = __shfl_up(x, o);
      if (lane >= o) x += y;
    }
    const double tot = __shfl(x, CH - 1);
    if (lane < CH) {
      const float hi = (float)x;
      S.gh[buf][lane] = hi;
      S.gl[buf][lane] = (float)(x - (double)hi);
      const float from = __builtin_amdgcn_exp2f((float)x), to = __builtin_amdgcn_exp2f((float)(tot - x));
      S.ra[buf][lane] = R.s_row * (rev ? to : from);
      S.rc[buf][lane] = R.s_upd * (rev ? from : to);
    }
    if (lane == 0) S.gc[buf] = __builtin_amdgcn_exp2f((float)tot);
    total += tot;
  };

  if (nch > 0) {
    fetch(first_of(0));
    if (wave == 0) scan(0, min(CH, len - first_of(0)));
  }
  if (OUT && nch > 0) state_to_lds();
  __syncthreads();

  for (int it = 0; it < nch; ++it) {
    const int buf = it & 1, t0 = first_of(it), nv = min(CH, len - t0);
    // tiles of this chunk to LDS
    if (OUT) {
      ta.store(S.a, LA, tid);
      tc.store(S.c, LC, tid);
    }
    tb.store(S.b, LA, tid);
    tc.each(tid, [&](int r, int c, const uint4& w) {
      const E* x = reinterpret_cast<const E*>(&w);
      constexpr int VN = LaTile<E, CH, NV>::VN;
      const float f = S.rc[buf][r];
      E q[SH::NSU][VN];
#pragma unroll
      for (int j = 0; j < VN; ++j) {
        E pcs[SH::NSU];
        pieces(to_f(x[j]) * f, pcs);
#pragma unroll
        for (int k = 0; k < SH::NSU; ++k) q[k][j] = pcs[k];
      }
#pragma unroll
      for (int k = 0; k < SH::NSU; ++k) {
        uint4 y;
        __builtin_memcpy(&y, q[k], 16);
        st16(&S.cs[k][r * LC + c], y);
      }
    });
    __syncthreads();
    const int tn = first_of(min(it + 1, nch - 1));   // (past the end: the last chunk again)
    fetch(tn);

    Acc<NV, CH, LA_NW> acc;
    if constexpr (OUT) {
      // transposed: rows i (or c), columns t
      Acc<CH, CH, LA_NW> sc;
      sc.zero();
      gemm_acc<E, CH, CH, DA, LA_NW, true, true>(sc, S.b, LA, S.a, LA, wave, lane);
      acc.zero();
#pragma unroll
      for (int k = 0; k < SH::NSX; ++k)
        gemm_acc<E, NV, CH, DA, LA_NW, true, true>(acc, S.x[k], LA, S.a, LA, wave, lane);
      for_tiles(sc, wave, lane, [&](int i0, int t, const f32x4& w) {
        const float th = S.gh[buf][t], tl = S.gl[buf][t];
        E pc4[4][SH::NSP];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = i0 + r;
          const float dif = (th - S.gh[buf][i]) + (tl - S.gl[buf][i]);
          const float e = __builtin_amdgcn_exp2f(rev ? -dif : dif);
          pieces((rev ? i >= t : i <= t) ? R.s_in * e * w[r] : 0.f, pc4[r]);
        }
#pragma unroll
        for (int k = 0; k < SH::NSP; ++k) {
          const E x4[4] = {pc4[0][k], pc4[1][k], pc4[2][k], pc4[3][k]};
          st4(&S.p[k][t * LP + i0], x4);
        }
      });
      for_tiles_ij(acc, wave, lane, [&](int i, int j, int, int t, const f32x4&) {
        const float f = S.ra[buf][t];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc.v[i][j][r] *= f;
      });
    }
    if (wave == 0 && it + 1 < nch) scan(buf ^ 1, min(CH, len - tn));
    if (OUT) __syncthreads();

    if constexpr (OUT) {
#pragma unroll
      for (int k = 0; k < SH::NSP; ++k)
        gemm_acc<E, NV, CH, CH, LA_NW, false, true>(acc, S.c, LC, S.p[k], LP, wave, lane);
      // out, and its dots with the rows of e
      typedef Tiling<NV, CH, LA_NW> TL;
      float dot[TL::RN];
#pragma unroll
      for (int j = 0; j < TL::RN; ++j) dot[j] = 0.f;
      for_tiles_ij(acc, wave, lane, [&](int, int j, int cl, int t, const f32x4& w) {
        if (t < nv && cl < nc) {
          const long tok = row0 + t0 + t;
          const long o = (args.cu ? 0 : b * R.so.b) + tok * R.so.t + h * R.so.h + c0 + cl;
          if (R.out32)
            st_f4(R.out32 + o, w);
          else
            st_f4(R.out + o, w);
          if (PR && R.e) {
            const f32x4 x = raw4_to_f(ld_raw4(
                R.e + ((args.cu ? 0 : b * R.se.b) + tok * R.se.t + (long)(h / R.ge) * R.se.h + c0 + cl)));
            dot[j] += (w[0] * x[0] + w[1] * x[1]) + (w[2] * x[2] + w[3] * x[3]);
          }
        }
      });
      if (PR && R.e && TL::active(wave)) {
        const int part = slice * TL::WM + wave / TL::WN;
        const int parts = (R.dc + NV - 1) / NV * TL::WM;
#pragma unroll
        for (int j = 0; j < TL::RN; ++j) {
          dot[j] += __shfl_xor(dot[j], 16);
          dot[j] += __shfl_xor(dot[j], 32);
          const int t = TL::n0(wave) + 16 * j + (lane & 15);
          if (lane < 16 && t < nv) R.edot[((long)bh * parts + part) * args.T + s0 + t0 + t] = dot[j];
        }
      }
    }
    // X' = 2^{G_C} X + B^T (factor o C)
    const float gc = S.gc[buf];
    for_tiles_ij(X, wave, lane, [&](int i, int j, int, int, const f32x4&) {
#pragma unroll
      for (int r = 0; r < 4; ++r) X.v[i][j][r] *= gc;
    });
#pragma unroll
    for (int k = 0; k < SH::NSU; ++k)
      gemm_acc<E, DA, NV, CH, LA_NW, false, false>(X, S.b, LA, S.cs[k], LC, wave, lane);
    if (OUT && it + 1 < nch) state_to_lds();
    __syncthreads();
  }

  if (OUT) {
    if (last && R.fin) state_store(R.fin + (long)bh * args.DD);
  } else {
    state_store(R.seg + segoff);
    if (tid == 0 && slice == 0) R.segdec[(long)bh * args.nseg + seg] = __builtin_amdgcn_exp2f((float)total);
  }
}

// Launch of one instance; DA and NV by the operands' size.
template <typename E, int DA, int NV, int CH, bool PR, bool OUT>
hipError_t la_launch(const LaArgs<E>& a, hipStream_t s) {
  const unsigned grid = (unsigned)((long)a.B * a.H * a.nseg * a.nroles * a.nslice);
  hipLaunchKernelGGL((la_pass_kernel<E, DA, NV, CH, PR, OUT>), dim3(grid), dim3(LA_NT), 0, s, a);
  return hipGetLastError();
}

}  // namespace prism
