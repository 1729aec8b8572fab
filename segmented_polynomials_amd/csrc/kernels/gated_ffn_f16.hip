// Gated feed-forward kernels, element type f16 (see gated_ffn.hpp).
#include "gated_ffn.hpp"

namespace segpoly {
namespace kern {

int ffn_fwd_f16(const GatedFfnArgs& a, size_t* bytes) { return ffn_fwd<DtF16>(a, bytes); }
int ffn_bwd_f16(const GatedFfnArgs& a, size_t* bytes) { return ffn_bwd<DtF16>(a, bytes); }

}  // namespace kern
}  // namespace segpoly
