// What the operators of a recurrent block share: column sums of partials, and
// the results of sequences without tokens.
#include "block_ops.h"
#include "prism_common.h"

namespace prism {

namespace {

// 32 columns a workgroup, 32 threads on each column taking every 32nd partial,
// joined through LDS in a fixed order.
__global__ __launch_bounds__(1024) void column_sums_kernel(const float* part, int parts, int C, int K, float* out,
                                                           float* last) {
  __shared__ float sm[32][33];
  const int c = threadIdx.x & 31, y = threadIdx.x >> 5;
  const long n = (long)(K + 1) * C, col = blockIdx.x * 32L + c;
  float s = 0.f;
  if (col < n) {
#pragma unroll 8
    for (int r = y; r < parts; r += 32) s += part[r * n + col];
  }
  sm[y][c] = s;
  __syncthreads();
  if (y == 0 && col < n) {
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) x += sm[k][c];
    const int j = (int)(col / C);
    float* to = j < K ? out : last;
    if (to) to[j < K ? (col - (long)j * C) * K + j : col - (long)j * C] = x;
  }
}

// A workgroup a sequence: whether it is empty from the largest offset up to its
// start and to its end.
template <typename W>
__global__ __launch_bounds__(256) void empty_sequences_kernel(const int* cu, int rows, int T, W* dst, const W* src,
                                                              int n) {
  __shared__ int sm[4];
  const int b = blockIdx.x;
  bool empty = T == 0;
  if (cu) {
    int m = 0;
    for (int j = threadIdx.x; j <= b; j += 256) m = max(m, min(cu[j], rows));
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = max(m, __shfl_xor(m, o));
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = m;
    __syncthreads();
    m = max(max(sm[0], sm[1]), max(sm[2], sm[3]));
    empty = min(cu[b + 1], rows) <= m;
  }
  if (!empty) return;
  for (int e = threadIdx.x; e < n; e += 256) dst[(long)b * n + e] = src ? src[(long)b * n + e] : W(0);
}

}  // namespace

hipError_t launch_column_sums(const float* part, int parts, int C, int K, float* out, float* last, hipStream_t s) {
  hipLaunchKernelGGL(column_sums_kernel, dim3((unsigned)(((K + 1L) * C + 31) / 32)), dim3(1024), 0, s, part, parts, C, K,
                     out, last);
  return hipGetLastError();
}

hipError_t launch_empty_sequences(const int* cu, int B, int rows, int T, void* dst, const void* src, int n, int size,
                                  hipStream_t s) {
  if (B == 0 || n == 0) return hipSuccess;
  if (size == 2)
    hipLaunchKernelGGL((empty_sequences_kernel<unsigned short>), dim3(B), dim3(256), 0, s, cu, rows, T,
                       static_cast<unsigned short*>(dst), static_cast<const unsigned short*>(src), n);
  else
    hipLaunchKernelGGL((empty_sequences_kernel<unsigned>), dim3(B), dim3(256), 0, s, cu, rows, T,
                       static_cast<unsigned*>(dst), static_cast<const unsigned*>(src), n);
  return hipGetLastError();
}

}  // namespace prism
