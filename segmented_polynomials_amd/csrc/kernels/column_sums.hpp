// Sums of columns over partial rows: a workgroup of 1024 takes 32 columns by 32
// interleaved sets of rows, whose sums are added in order.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace segpoly {
namespace kern {

// The column c = 32 blockIdx.x + threadIdx.x % 32 over the rows, `stride` apart,
// of `partial`; the first 32 threads get theirs.
__device__ __forceinline__ float column_sum(const float* __restrict__ partial, int64_t rows, int64_t stride,
                                            int64_t columns, int64_t c) {
  __shared__ float lds[32 * 33];
  const int set = threadIdx.x / 32;
  float s = 0.f;
  if (c < columns) {
#pragma unroll 8
    for (int64_t p = set; p < rows; p += 32) s += partial[p * stride + c];
  }
  lds[set * 33 + threadIdx.x % 32] = s;
  __syncthreads();
  float t = 0.f;
  if (threadIdx.x < 32) {
#pragma unroll
    for (int q = 0; q < 32; ++q) t += lds[q * 33 + threadIdx.x];
  }
  return t;
}

}  // namespace kern
}  // namespace segpoly
