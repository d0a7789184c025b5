// Host-side declarations of the query / key normalisation and of the linear
// attention, shared by the C-ABI layer (operators_api.cpp) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace prism {

typedef __bf16 bf16;

struct Strides {
  long b, t, h;   // elements between batch entries, tokens, heads
};

// ---------------------------------------------------------------- qk_norm
// One launch covers the query and the key heads: heads 0 .. Hq - 1 are q,
// Hq .. Hq + Hk - 1 are k.
struct QkNormArgs {
  int B, T, Hq, Hk, d, rot;
  float c, eps;                  // r = (c sum x^2 + eps)^(-1/2)
  int interleaved;
  const void *xq, *xk;           // inputs
  const void *wq, *wk;           // weights (nullptr: ones)
  const int* pos;                // [B, T] (nullptr: no rotation)
  const long long* turns;        // [rot / 2]
  const void *gq, *gk;           // output gradients (backward)
  void *yq, *yk;                 // outputs (forward) or input gradients (backward)
  Strides sxq, sxk, sgq, sgk, syq, syk;
  float *part, *dwq, *dwk;       // weight-gradient partials and results (backward)
};
template <typename E> hipError_t launch_qk_norm(const QkNormArgs& a, hipStream_t s);
template <typename E> hipError_t launch_qk_norm_bwd(const QkNormArgs& a, hipStream_t s);
size_t qk_norm_part_bytes(int d);   // room for the weight-gradient partials

// ------------------------------------------------------- linear attention
// Every pass over a sequence is one form: with operand rows A_t, B_t (da
// values) and C_t (dc values), cumulative log decays G_t and a state X [da][dc],
//   forward:  out_t = s_in sum_{i<=t} e^{G_t-G_i} (A_t.B_i) C_i + s_row e^{G_t} A_t X0
//   reverse:  out_t = s_in sum_{i>=t} e^{G_i-G_t} (A_t.B_i) C_i + s_row e^{G_T-G_t} A_t X0
// and the state after the pass is e^{G_T} X0 + s_upd sum_i e^{G_T-G_i} B_i C_i^T
// (reverse: e^{G_i}).  (q, k, v) forward gives o; (dO, v, k) forward dq;
// (v, dO, q) reverse dk; (k, q, dO) reverse dv.
// Rows of sequence b of a packed batch, from the caller's offsets: c'_i = max_{j <= i} clamp(cu[j], 0, N)
// in place of cu[i], and at most T rows, so that every sequence lies inside the N rows and no two overlap
// whatever the offsets are.  Called by all 256 threads of a workgroup; sm: four ints of LDS.
#ifdef __HIPCC__
__device__ inline void la_sequence(const int* cu, int N, int T, int b, int tid, int* sm, long& first, int& n) {
  int m = 0;
  for (int j = tid; j <= b; j += 256) m = max(m, min(cu[j], N));
  const int end = min(cu[b + 1], N);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, __shfl_xor(m, o));
  if ((tid & 63) == 0) sm[tid >> 6] = m;
  __syncthreads();
  m = __builtin_amdgcn_readfirstlane(max(max(sm[0], sm[1]), max(sm[2], sm[3])));
  first = m;
  n = __builtin_amdgcn_readfirstlane(min(max(end - m, 0), T));
}
#endif

template <typename E>
struct LaRole {
  const E *a, *b, *c;
  Strides sa, sb, sc;
  int ga, gb, gc;          // query heads per head of a, b, c
  E* out;                  // strided by so, or
  float* out32;            // fp32, strided by so (one row for each query head)
  Strides so;
  const E* e;              // rows dotted with out (fp32, before rounding), or nullptr
  Strides se;
  int ge;
  float* edot;             // [H][LA_PARTS][rows] partial dots
  int da, dc, rev;
  float s_in, s_row, s_upd;
  const float* X0;         // [B, H, dv, dk] entering state (nullptr: zeros)
  float* fin;              // the same, leaving (nullptr: not wanted)
  float* seg;              // [B * H][nseg][dv * dk] states of the segments (nseg > 1)
  float* segdec;           // [B * H][nseg] decay over a segment (nseg > 1)
  int xa, xc;              // element steps of X's two indexes in those arrays
};
constexpr int LA_ROLES = 3;
// A sequence is cut into nseg segments of `seglen` tokens (a whole number of
// chunks), worked on side by side.
template <typename E>
struct LaArgs {
  int B, T, H, nseg, seglen, nroles;
  int joined;              // role.seg holds entering states, not the segments' own
  int DD;                  // dv * dk
  const int* cu;           // offsets of a packed batch of N rows, or nullptr
  int N;
  long rows;               // N, or B * T
  const float* g;
  Strides sg;
  LaRole<E> r[LA_ROLES];
};
constexpr int LA_CHUNK = 32;   // tokens per chunk
// Partial row dots written for each token (one a wave).
constexpr int LA_PARTS = 4;
// What a pass computes (dim = max(dk, dv)): the segments' own states alone
// (role.seg, role.segdec), as far as bf16 outputs or as fp32 results need them;
// outputs; outputs and a final state (role.fin); outputs, a final state and the
// row dots, every product's bf16 operands in three pieces.
enum LaPass { LA_STATES, LA_STATES_FP32, LA_OUT, LA_OUT_STATE, LA_OUT_DOTS };
template <typename E>
hipError_t launch_la_pass(const LaArgs<E>& a, int dim, LaPass kind, hipStream_t s);

// Segment states in place: own states -> states entering each segment.
struct LaJoin {
  int B, T, H, nseg, seglen, DD;
  const int* cu;
  int N;
  float* seg[2];           // forward, reverse (nullptr: absent)
  const float* dec[2];
  const float* X0[2];
};
hipError_t launch_la_join(const LaJoin& a, hipStream_t s);

// dg from the row dots: dg_t = sum_{i >= t} (q_i.dq_i - k_i.dk_i) + <dS, S> at
// the segment's end.
struct LaDecay {
  int B, T, H, nseg, seglen, DD;
  const int* cu;
  int N;
  long rows;                       // N, or B * T
  const float* g;
  Strides sg;
  const float *eq, *ek;            // [H][LA_PARTS][rows]
  const float *segf, *segr;        // states of the segments, forward and reverse (nseg > 1):
  const float *decf, *decr;        // entering (joined), or their own with their decays
  int joined;
  const float *S0, *ST, *dST;      // first, last state and the latter's gradient (nullptr: zero)
  int per_head;                    // dg is one sum a head (over no sequences: zero)
  float* dg;                       // strided like g, or [H] (strided like its heads), summed from
  float* tmp;                      // [H][rows]
};
hipError_t launch_la_decay(const LaDecay& a, hipStream_t s);

// dk, dv [.., Hk, d] = sums over the grp query heads of each of the fp32 partials [.., H, d]
template <typename E>
hipError_t launch_la_group_sum(const float* dkp, const float* dvp, E* dk, E* dv, long rows, int Hk, int grp, int dimk,
                               int dimv, hipStream_t s);

template <typename E>
struct LaStepArgs {
  int B, T, H, dk, dv, grp;
  float scale;
  const E *q, *k, *v;
  Strides sq, sk, sv, so, sg;
  const float* g;
  const float* S;
  float* S_out;
  E* o;
};
template <typename E> hipError_t launch_la_step(const LaStepArgs<E>& a, hipStream_t s);

}  // namespace prism
