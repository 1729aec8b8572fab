// Dense layer kernels, element type f16 (see dense.hpp).
#include "dense.hpp"

namespace segpoly {
namespace kern {

int dense_fwd_f16(const DenseArgs& a, size_t* bytes) { return dense_fwd<DtF16Plain>(a, bytes); }
int dense_bwd_f16(const DenseArgs& a, size_t* bytes) { return dense_bwd<DtF16>(a, bytes); }

}  // namespace kern
}  // namespace segpoly
