// Block norm kernels, element type f16 (see block_norm.hpp).
#include "block_norm.hpp"

namespace segpoly {
namespace kern {

int block_norm_f16(const BlockNormArgs& a, bool backward) { return block_norm_rows<f16>(a, backward); }

}  // namespace kern
}  // namespace segpoly
