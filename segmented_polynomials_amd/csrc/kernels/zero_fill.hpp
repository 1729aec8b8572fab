// Zeros to up to three buffers, for gradients of no rows.
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

namespace segpoly {
namespace kern {

struct ZeroArgs {
  void* to[3];
  int64_t count[3];
};
template <typename U>
__global__ void __launch_bounds__(256)
zero_kernel(ZeroArgs g) {
  U* to = static_cast<U*>(g.to[blockIdx.y]);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < g.count[blockIdx.y];
       i += static_cast<int64_t>(gridDim.x) * 256)
    to[i] = 0;
}

// `count` elements of `bytes` (2 or 4) each to the buffers that are not null
inline int zero_fill(const ZeroArgs& g, int64_t bytes, hipStream_t st) {
  int64_t most = 0;
  for (int i = 0; i < 3; ++i) most = std::max(most, g.count[i]);
  if (most == 0) return 0;
  const int64_t blocks = std::min<int64_t>((most + 255) / 256, 2048);
  auto* zero = bytes == 4 ? zero_kernel<uint32_t> : zero_kernel<uint16_t>;
  hipLaunchKernelGGL(zero, dim3(static_cast<unsigned>(blocks), 3), dim3(256), 0, st, g);
  return static_cast<int>(hipGetLastError());
}

}  // namespace kern
}  // namespace segpoly
