// What the operators of a recurrent block share: column sums of partials.
#include "block_ops.h"
#include "prism_common.h"

namespace prism {

namespace {

// 32 columns a workgroup, 32 threads on each column taking every 32nd partial,
// joined through LDS in a fixed order: latency bound, 8 loads on their way (256
// partials of 2 x 2048 values, 4 MB, 4 us).
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

}  // namespace

hipError_t launch_column_sums(const float* part, int parts, int C, int K, float* out, float* last, hipStream_t s) {
  hipLaunchKernelGGL(column_sums_kernel, dim3((unsigned)(((K + 1L) * C + 31) / 32)), dim3(1024), 0, s, part, parts, C,
                     K, out, last);
  return hipGetLastError();
}

}  // namespace prism
