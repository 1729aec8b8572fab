// Block norm kernels, element type bf16 (see block_norm.hpp).
#include "block_norm.hpp"

namespace segpoly {
namespace kern {

int block_norm_bf16(const BlockNormArgs& a, bool backward) { return block_norm_rows<bf16>(a, backward); }

}  // namespace kern
}  // namespace segpoly
