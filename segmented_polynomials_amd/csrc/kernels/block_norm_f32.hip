// Block norm kernels, element type f32 (see block_norm.hpp).
#include "block_norm.hpp"

namespace segpoly {
namespace kern {

int block_norm_f32(const BlockNormArgs& a, bool backward) { return block_norm_rows<float>(a, backward); }

}  // namespace kern
}  // namespace segpoly
