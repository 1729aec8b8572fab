// Type dispatch of the gated feed-forward operator.
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

}  // namespace kern

size_t gated_ffn_workspace_bytes(int dtype, int64_t n, int64_t d_in, int64_t hidden, int64_t d_out, bool backward) {
  GatedFfnArgs a{};
  a.dtype = dtype, a.n = n, a.d_in = d_in, a.hidden = hidden, a.d_out = d_out;
  a.x_stride = d_in, a.gout_stride = d_out;
  size_t bytes = 0;
  kern::ffn_any(a, backward, &bytes);
  return bytes;
}

int launch_gated_ffn_fwd(const GatedFfnArgs& a) { return kern::ffn_any(a, false, nullptr); }
int launch_gated_ffn_bwd(const GatedFfnArgs& a) { return kern::ffn_any(a, true, nullptr); }

}  // namespace segpoly
