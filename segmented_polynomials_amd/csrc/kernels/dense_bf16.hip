// Dense layer kernels, element type bf16 (see dense.hpp).
#include "dense.hpp"

namespace segpoly {
namespace kern {

int dense_fwd_bf16(const DenseArgs& a, size_t* bytes) { return dense_fwd<DtBF16>(a, bytes); }
int dense_bwd_bf16(const DenseArgs& a, size_t* bytes) { return dense_bwd<DtBF16>(a, bytes); }

}  // namespace kern
}  // namespace segpoly
