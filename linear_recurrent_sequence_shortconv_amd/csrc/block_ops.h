// Host-side declarations of the operators of a recurrent block (layer norm,
// short convolution, gated recurrence), shared by the C-ABI layer
// (block_ops_api.cpp) and the kernels.
#pragma once

#include "operators.h"

namespace prism {

// Element steps of a token tensor [B, T, D] (packed: [N, D], batch unused).
struct TokenSteps {
  long b, t;
};

// --------------------------------------------------------------- layer norm
struct LayerNormArgs {
  long rows;               // B * T * H rows of D values
  int T, H, D;
  int center;              // 1: mean and deviation, 0: root mean square
  float eps;
  const void *x, *r, *w, *b;
  void *y, *h;             // forward: results; h nullptr: the sum is not wanted
  Strides sx, sr, sy, sh;  // backward: sr of dh, sy of dy, sh of dx
  const void *dy, *dh;
  void* dx;
  float *part, *dw, *db;   // weight-gradient partials and results (nullptr: not wanted)
};
template <typename E> hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t s);
template <typename E> hipError_t launch_layer_norm_bwd(const LayerNormArgs& a, hipStream_t s);
size_t layer_norm_part_bytes(int D);   // room for the weight-gradient partials
constexpr int LN_MAX_D = 16384;

// -------------------------------------------------------- short convolution
struct ShortConvArgs {
  int B, T, D, K;
  int rows;                // N, or B * T
  int silu;
  const int* cu;           // offsets of a packed batch, or nullptr
  const void *x, *w, *b, *hist;
  void *y, *hist_out;
  TokenSteps sx, sy, sd;   // of x, of y / dy, of dx
  const void* dy;
  void* dx;
  float *part, *dw, *db, *dhist;
};
template <typename E> hipError_t launch_short_conv(const ShortConvArgs& a, hipStream_t s);
template <typename E> hipError_t launch_short_conv_bwd(const ShortConvArgs& a, hipStream_t s);
size_t short_conv_part_bytes(int rows, int D, int K);

// --------------------------------------------------------- gated recurrence
// (part: set by the launch)
enum Gate { GATE_LOG, GATE_SIGMOID, GATE_POWER };
struct RecurrenceArgs {
  int B, T, D;
  int rows;                // N, or B * T
  int gate;
  const int* cu;
  const void *x, *f, *i;   // i nullptr: an open input gate
  const float *lam, *h0;
  void* h;
  float* hT;
  TokenSteps sx, sf, si, sh;
  // backward
  const void* dh;
  const float* dhT;
  void *dx, *df, *di;
  float *dh0, *dlam, *part;
  TokenSteps sdh, sdx, sdf, sdi;
};
hipError_t launch_recurrence(const RecurrenceArgs& a, bool f32, bool bwd, void* ws, hipStream_t s);
hipError_t launch_recurrence_step(const RecurrenceArgs& a, bool f32, hipStream_t s);
size_t recurrence_bytes(const RecurrenceArgs& a, bool packed, bool bwd);   // of the workspace

// ------------------------------------------------- partials and sequences
// Sums over partials [K + 1][C] in a fixed order: rows j < K go to out[c * K + j],
// the last to last[c] (each nullptr: not wanted).
hipError_t launch_column_sums(const float* part, int parts, int C, int K, float* out, float* last, hipStream_t s);

#ifdef __HIPCC__
// The sequence that holds row `row` of a batch: rows start .. end - 1 of
// sequence b; b < 0 or b >= B: rows of no sequence.  Packed batches take the
// caller's offsets as c'_i = max_{j <= i} min(max(cu[j], 0), rows), so that the
// sequences lie inside the tensors and do not overlap whatever the offsets are.
struct Sequence {
  int b, start, end;
};
// Called by whole waves with one row each; 256 offsets in one trip to memory.
__device__ inline Sequence find_sequence(const int* cu, int B, int T, int rows, int row) {
  Sequence q;
  if (!cu) {
    q.b = row / T;
    q.start = q.b * T;
    q.end = q.start + T;
    return q;
  }
  const int lane = threadIdx.x & 63;
  int before = 0;   // largest offset not behind the row, of the lane's
  q.b = B;
  q.end = rows;
  for (int j0 = 0; j0 <= B; j0 += 256) {
    int c[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + 64 * u + lane;
      c[u] = j <= B ? min(max(cu[j], 0), rows) : 0;
    }
    bool found = false;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const unsigned long long behind = __ballot(c[u] > row);
      if (!found && behind) {
        const int first = __builtin_ctzll(behind);
        q.b = j0 + 64 * u + first - 1;
        q.end = __builtin_amdgcn_readlane(c[u], first);
        if (lane < first) before = max(before, c[u]);
        found = true;
      } else if (!found) {
        before = max(before, c[u]);
      }
    }
    if (found) break;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) before = max(before, __shfl_xor(before, o));
  q.b = __builtin_amdgcn_readfirstlane(q.b);
  q.start = __builtin_amdgcn_readfirstlane(before);
  q.end = __builtin_amdgcn_readfirstlane(q.end);
  return q;
}

// Whether sequence b has no tokens, which no row of a pass belongs to; by all 256
// threads of a workgroup, sm: four ints of LDS.
__device__ inline bool empty_sequence(const int* cu, int T, int rows, int b, int* sm) {
  if (!cu) return T == 0;
  int m = 0;
  for (int j = threadIdx.x; j <= b; j += 256) m = max(m, min(cu[j], rows));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, __shfl_xor(m, o));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = m;
  __syncthreads();
  return min(cu[b + 1], rows) <= max(max(sm[0], sm[1]), max(sm[2], sm[3]));
}
#endif

}  // namespace prism
