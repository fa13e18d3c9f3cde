// Sum over the rows of a matrix of partial sums, in a fixed order.
#pragma once

#include "ssm_device.h"
#include "ssm_internal.h"

namespace ssm {
namespace {

// out[y][c] = sum of part[y]'s n rows at column c (y: blockIdx.y, parts `second` floats apart; NULL outputs are left
// out).  16 columns a workgroup, 64 interleaved sums a column (eight loads of each on their way), joined
// across lanes and then across the 16 waves.
__global__ void __launch_bounds__(1024) k_col_sum(const float* part, float* out0, float* out1, int64_t second,
                                                  int64_t n, int64_t width) {
  __shared__ float s[16][16];
  float* const out = blockIdx.y == 0 ? out0 : out1;
  if (out == nullptr) return;
  const int c = threadIdx.x & 15;
  const int64_t col = (int64_t)blockIdx.x * 16 + c;
  const float* const p = part + (blockIdx.y == 0 ? 0 : second) + col;
  float v = 0.0f;
  if (col < width)
    for (int64_t k = threadIdx.x >> 4; k < n; k += 8 * 64) {
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = k + 64 * i < n ? p[(k + 64 * i) * width] : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v += q[i];
    }
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  if ((threadIdx.x & 48) == 0) s[threadIdx.x / 64][c] = v;
  __syncthreads();
  if (threadIdx.x < 16 && col < width) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) t += s[w][c];
    out[col] = t;
  }
}

hipError_t col_sum(const float* part, float* out0, float* out1, int64_t second, int64_t n, int64_t width,
                   hipStream_t stream) {
  return launch(k_col_sum, dim3((unsigned)((width + 15) / 16), out1 != nullptr ? 2 : 1), dim3(1024), 0, stream, part,
                out0, out1, second, n, width);
}

}  // namespace
}  // namespace ssm
