// Gated feed-forward kernels, element type bf16 (see gated_ffn.hpp).
#include "gated_ffn.hpp"

namespace segpoly {
namespace kern {

int ffn_fwd_bf16(const GatedFfnArgs& a, size_t* bytes) { return ffn_fwd<DtBF16>(a, bytes); }
int ffn_bwd_bf16(const GatedFfnArgs& a, size_t* bytes) { return ffn_bwd<DtBF16>(a, bytes); }

}  // namespace kern
}  // namespace segpoly
