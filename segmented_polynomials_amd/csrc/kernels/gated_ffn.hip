// Type dispatch of the gated feed-forward operator, and its gradient over no
// rows.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../channel_ops.hpp"

namespace segpoly {
namespace kern {

#define SEGPOLY_FFN_DECL(name)                                  \
  int ffn_fwd_##name(const GatedFfnArgs& a, size_t* bytes); \
  int ffn_bwd_##name(const GatedFfnArgs& a, size_t* bytes);
SEGPOLY_FFN_DECL(bf16)
SEGPOLY_FFN_DECL(f16)
SEGPOLY_FFN_DECL(f32)
#undef SEGPOLY_FFN_DECL

int ffn_any(const GatedFfnArgs& a, bool backward, size_t* bytes) {
  if (a.dtype == kChBF16) return backward ? ffn_bwd_bf16(a, bytes) : ffn_fwd_bf16(a, bytes);
  if (a.dtype == kChF16) return backward ? ffn_bwd_f16(a, bytes) : ffn_fwd_f16(a, bytes);
  return backward ? ffn_bwd_f32(a, bytes) : ffn_fwd_f32(a, bytes);
}

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

// The weight gradients of no rows: zeros, without a look at the weights, which
// the caller need not have.
int ffn_bwd_no_rows(const GatedFfnArgs& a) {
  if (!a.gw_gate) return 0;
  const int64_t in = a.hidden * a.d_in, out = a.d_out * a.hidden;
  const ZeroArgs g{{a.gw_gate, a.gw_up, a.gw_down}, {in, in, out}};
  const int64_t blocks = std::min<int64_t>((std::max(in, out) + 255) / 256, 2048);
  auto* zero = channel_dtype_bytes(a.dtype) == 4 ? zero_kernel<uint32_t> : zero_kernel<uint16_t>;
  hipLaunchKernelGGL(zero, dim3(static_cast<unsigned>(blocks), 3), dim3(256), 0, static_cast<hipStream_t>(a.stream), g);
  return static_cast<int>(hipGetLastError());
}

}  // namespace kern

size_t gated_ffn_workspace_bytes(int dtype, int64_t n, int64_t d_in, int64_t hidden, int64_t d_out, bool backward) {
  if (n == 0) return 0;
  GatedFfnArgs a{};
  a.dtype = dtype, a.n = n, a.d_in = d_in, a.hidden = hidden, a.d_out = d_out;
  a.x_stride = d_in, a.gout_stride = d_out;
  size_t bytes = 0;
  kern::ffn_any(a, backward, &bytes);
  return bytes;
}

int launch_gated_ffn_fwd(const GatedFfnArgs& a) { return kern::ffn_any(a, false, nullptr); }
int launch_gated_ffn_bwd(const GatedFfnArgs& a) {
  return a.n == 0 ? kern::ffn_bwd_no_rows(a) : kern::ffn_any(a, true, nullptr);
}

}  // namespace segpoly
