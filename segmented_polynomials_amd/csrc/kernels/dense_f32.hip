// Dense layer kernels, element type f32 (see dense.hpp).
#include "dense.hpp"

namespace segpoly {
namespace kern {

int dense_fwd_f32(const DenseArgs& a, size_t* bytes) { return dense_fwd<DtF32Staged>(a, bytes); }
int dense_bwd_f32(const DenseArgs& a, size_t* bytes) { return dense_bwd<DtF32Staged>(a, bytes); }

}  // namespace kern
}  // namespace segpoly
