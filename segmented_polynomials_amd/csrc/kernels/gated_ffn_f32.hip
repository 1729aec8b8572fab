// Gated feed-forward kernels, element type f32 (see gated_ffn.hpp).
#include "gated_ffn.hpp"

namespace segpoly {
namespace kern {

int ffn_fwd_f32(const GatedFfnArgs& a, size_t* bytes) { return ffn_fwd<DtF32>(a, bytes); }
int ffn_bwd_f32(const GatedFfnArgs& a, size_t* bytes) { return ffn_bwd<DtF32>(a, bytes); }

}  // namespace kern
}  // namespace segpoly
