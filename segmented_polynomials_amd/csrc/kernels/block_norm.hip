// Row loop sizes, the fold of the parameters' gradients and the type dispatch
// of the block norm (block_norm.hpp).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../channel_ops.hpp"
#include "../launch.hpp"
#include "column_sums.hpp"

namespace segpoly {

namespace {

// lanes that hold one row, 8 elements each, and the threads of a workgroup
int64_t row_threads(int64_t dim) {
  int64_t lanes = 16;
  while (lanes < 1024 && lanes * 8 < dim) lanes *= 2;
  return lanes;
}

}  // namespace

int64_t block_norm_even_grid(int64_t steps, int64_t most) {
  if (steps < 1) return 1;
  const int64_t each = (steps + most - 1) / most;
  return (steps + each - 1) / each;
}

int64_t block_norm_parts(int64_t n, int64_t dim) {
  const int64_t lanes = row_threads(dim), threads = std::max<int64_t>(lanes, 256), per = threads / lanes;
  // resident workgroups at the backward's registers: three of 256 threads, 1024 lanes of the wider
  return block_norm_even_grid((n + per - 1) / per, 256 * (threads == 256 ? 3 : 1024 / threads));
}

namespace kern {

// column sums of the partial rows
__global__ void __launch_bounds__(1024)
block_norm_fold_kernel(const float* __restrict__ partial, int64_t parts, int64_t dim, const float* __restrict__ w_post,
                       const float* __restrict__ res_scale, float* __restrict__ gpost, float* __restrict__ gscale,
                       float* __restrict__ gpre) {
  if (blockIdx.y == 1 && !gpre) return;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x % 32;
  const float t = column_sum(partial + blockIdx.y * dim, parts, 2 * dim, dim, c);
  if (threadIdx.x >= 32 || c >= dim) return;
  if (blockIdx.y == 1) {
    gpre[c] = t;
  } else {
    gpost[c] = res_scale ? t * res_scale[c] : t;
    if (gscale) gscale[c] = t * w_post[c];
  }
}

int block_norm_fold(const BlockNormArgs& a) {
  hipLaunchKernelGGL(block_norm_fold_kernel, dim3(static_cast<unsigned>((a.dim + 31) / 32), 2), dim3(1024), 0,
                     static_cast<hipStream_t>(a.stream), static_cast<const float*>(a.workspace), a.parts, a.dim,
                     a.w_post, a.res_scale, a.gpost, a.gscale, a.gpre);
  return static_cast<int>(hipGetLastError());
}

int block_norm_bf16(const BlockNormArgs& a, bool backward);
int block_norm_f16(const BlockNormArgs& a, bool backward);
int block_norm_f32(const BlockNormArgs& a, bool backward);

int block_norm_any(const BlockNormArgs& a, bool backward) {
  if (a.dtype == kChBF16) return block_norm_bf16(a, backward);
  if (a.dtype == kChF16) return block_norm_f16(a, backward);
  return block_norm_f32(a, backward);
}

}  // namespace kern

int launch_block_norm_fwd(const BlockNormArgs& a) { return kern::block_norm_any(a, false); }
int launch_block_norm_bwd(const BlockNormArgs& a) { return kern::block_norm_any(a, true); }

}  // namespace segpoly
