// Type dispatch of the dense layer, and its gradient over no rows.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../channel_ops.hpp"
#include "zero_fill.hpp"

namespace segpoly {
namespace kern {

#define SEGPOLY_DENSE_DECL(name)                              \
  int dense_fwd_##name(const DenseArgs& a, size_t* bytes); \
  int dense_bwd_##name(const DenseArgs& a, size_t* bytes);
SEGPOLY_DENSE_DECL(bf16)
SEGPOLY_DENSE_DECL(f16)
SEGPOLY_DENSE_DECL(f32)
#undef SEGPOLY_DENSE_DECL

int dense_any(const DenseArgs& a, bool backward, size_t* bytes) {
  if (a.dtype == kChBF16) return backward ? dense_bwd_bf16(a, bytes) : dense_fwd_bf16(a, bytes);
  if (a.dtype == kChF16) return backward ? dense_bwd_f16(a, bytes) : dense_fwd_f16(a, bytes);
  return backward ? dense_bwd_f32(a, bytes) : dense_fwd_f32(a, bytes);
}

}  // namespace kern

size_t dense_workspace_bytes(int dtype, int act, int64_t n, int64_t d_in, int64_t d_out, bool backward) {
  if (n == 0) return 0;
  DenseArgs a{};
  a.dtype = dtype, a.act = act, a.n = n, a.d_in = d_in, a.d_out = d_out;
  a.x_stride = d_in, a.gout_stride = d_out, a.residual_stride = d_out;
  size_t bytes = 0;
  kern::dense_any(a, backward, &bytes);
  return bytes;
}

int launch_dense_fwd(const DenseArgs& a) { return kern::dense_any(a, false, nullptr); }
int launch_dense_bwd(const DenseArgs& a) {
  if (a.n > 0) return kern::dense_any(a, true, nullptr);
  return kern::zero_fill({{a.gw, a.gbias, nullptr}, {a.gw ? a.d_out * a.d_in : 0, a.gbias ? a.d_out : 0, 0}},
                         channel_dtype_bytes(a.dtype), static_cast<hipStream_t>(a.stream));
}

}  // namespace segpoly
