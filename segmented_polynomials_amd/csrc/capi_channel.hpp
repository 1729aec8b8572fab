// Checks of arguments shared by the C ABI of the operators on rows of
// channels.  Host code.
#pragma once
#include <initializer_list>
#include <string>

#include "capi_util.hpp"
#include "channel_ops.hpp"
#include "segpoly.h"

namespace segpoly {

inline int launched(int rc, const char* what) {
  if (rc) return fail(SEGPOLY_E_HIP, std::string(what) + " launch: " + hipGetErrorString(static_cast<hipError_t>(rc)));
  return ok();
}

inline int check_dtype(int dtype) {
  if (dtype == SEGPOLY_F64)
    return fail(SEGPOLY_E_UNSUPPORTED, "the invariant-channel operators take float32, bfloat16 and float16");
  if (dtype != SEGPOLY_F32 && dtype != SEGPOLY_BF16 && dtype != SEGPOLY_F16)
    return fail(SEGPOLY_E_INVALID, "bad dtype");
  return SEGPOLY_OK;
}

inline bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// every buffer at a multiple of its element's size
inline int check_aligned(int64_t bytes, std::initializer_list<const void*> buffers) {
  for (const void* p : buffers)
    if (!aligned(p, bytes)) return fail(SEGPOLY_E_INVALID, "misaligned buffer");
  return SEGPOLY_OK;
}
inline int64_t index_bytes(int idx_dtype) { return idx_dtype == SEGPOLY_I32 ? 4 : 8; }

inline int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return SEGPOLY_OK;
  if (!ws) return fail(SEGPOLY_E_INVALID, "null workspace");
  if (!aligned(ws, 256)) return fail(SEGPOLY_E_INVALID, "workspace must be 256-byte aligned");
  if (have < need)
    return fail(SEGPOLY_E_INVALID, "workspace has " + std::to_string(have) + " bytes, needs " + std::to_string(need));
  return SEGPOLY_OK;
}

// the largest width and row stride the kernels' 32-bit offsets take
constexpr int64_t kMaxWidth = int64_t{1} << 21;

// The row stride of a feed-forward operand: that of a single row, or none, is never
// used, whatever the tensor it was taken from.
inline int64_t row_stride(int64_t n, int64_t stride, int64_t width) { return n <= 1 ? width : stride; }

}  // namespace segpoly
