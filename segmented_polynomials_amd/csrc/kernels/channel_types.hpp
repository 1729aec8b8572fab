// Element types of the invariant-channel kernels and their 16-byte accesses.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace segpoly {
namespace kern {

using bf16 = __bf16;
using f16 = _Float16;

template <typename T>
struct Chunk {
  static constexpr int kN = 16 / sizeof(T);  // elements of one 16-byte access
};

// 16 bytes from an address that is only element aligned: global memory
// accesses of this target may be unaligned, so rows of odd widths need no
// narrower loads, only the last chunk of a row does.
template <typename T>
__device__ __forceinline__ void load_chunk(const T* p, int valid, float* v) {
  constexpr int N = Chunk<T>::kN;
  if (valid >= N) {
    T t[N];
    __builtin_memcpy(t, p, 16);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = static_cast<float>(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < valid ? static_cast<float>(p[i]) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void store_chunk(T* p, int valid, const float* v) {
  constexpr int N = Chunk<T>::kN;
  T t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = static_cast<T>(v[i]);
  if (valid >= N) {
    __builtin_memcpy(p, t, 16);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < valid) p[i] = t[i];
  }
}

}  // namespace kern
}  // namespace segpoly
