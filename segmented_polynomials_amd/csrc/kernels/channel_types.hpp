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
  using Bits = uint16_t;
};
template <>
struct Chunk<float> {
  static constexpr int kN = 4;
  using Bits = uint32_t;
};

using u32x4 = uint32_t __attribute__((ext_vector_type(4)));

// The chunk at column c of a row of `width` elements, by one 16-byte load
// from an address that is only element aligned (global accesses of this
// target may be unaligned).  A chunk that crosses the row's end is loaded
// from further left, so that it ends with the row; settle_chunk moves its
// elements down and fills up with zeros, after the load has landed: several
// chunks can be in flight.  Rows narrower than a chunk are read by elements.
template <typename T>
__device__ __forceinline__ u32x4 load_raw(const T* row, int c, int width) {
  constexpr int N = Chunk<T>::kN;
  u32x4 r = {0, 0, 0, 0};
  if (c < width) {
    if (width >= N) {
      __builtin_memcpy(&r, row + (c + N <= width ? c : width - N), 16);
    } else {
      uint64_t lo = 0, hi = 0;
#pragma clang loop unroll(disable)
      for (int i = width - 1; i >= 0; --i) {
        constexpr int kBits = 8 * sizeof(T);
        using Bits = typename Chunk<T>::Bits;
        hi = hi << kBits | lo >> (64 - kBits);
        lo = lo << kBits | __builtin_bit_cast(Bits, row[i]);
      }
      r = u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                static_cast<uint32_t>(hi >> 32)};
    }
  }
  return r;
}

template <typename T>
__device__ __forceinline__ u32x4 settle_chunk(u32x4 r, int c, int width) {
  constexpr int N = Chunk<T>::kN;
  if (c < width && c + N > width && width >= N) {
    const int bits = (c + N - width) * (128 / N);  // 1 .. N - 1 elements
    uint64_t lo = r[0] | static_cast<uint64_t>(r[1]) << 32, hi = r[2] | static_cast<uint64_t>(r[3]) << 32;
    if (bits >= 64) {
      lo = hi >> (bits - 64);
      hi = 0;
    } else {
      lo = lo >> bits | hi << (64 - bits);
      hi >>= bits;
    }
    r = u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
              static_cast<uint32_t>(hi >> 32)};
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void unpack_chunk(u32x4 r, int c, int width, float* v) {
  constexpr int N = Chunk<T>::kN;
  r = settle_chunk<T>(r, c, width);
  T t[N];
  __builtin_memcpy(t, &r, 16);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = static_cast<float>(t[i]);
}

template <typename T>
__device__ __forceinline__ void load_chunk(const T* row, int c, int width, float* v) {
  unpack_chunk<T>(load_raw(row, c, width), c, width, v);
}

// the part of a chunk within the row: 16 bytes, or the halves its count names
template <typename T>
__device__ __forceinline__ void store_chunk(T* row, int c, int width, const float* v) {
  constexpr int N = Chunk<T>::kN;
  if (c >= width) return;
  T t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = static_cast<T>(v[i]);
  T* p = row + c;
  if (c + N <= width) {
    __builtin_memcpy(p, t, 16);
    return;
  }
  const int n = width - c;
  if constexpr (N == 8) {
    if (n & 4) {
      __builtin_memcpy(p, t, 8);
      p += 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = t[i + 4];
    }
  }
  if (n & 2) {
    __builtin_memcpy(p, t, 2 * sizeof(T));
    p += 2;
    t[0] = t[2];
  }
  if (n & 1) p[0] = t[0];
}

// ------------------------------------------------------------ sums over lanes

// Two copies of a value exchange rows of 16 (halves of 32) lanes, so that their
// sum is that of both.  In assembly: the compiler takes both results of the
// builtin for the same value.  Two wait states keep the exchange off a write
// just before it.
__device__ __forceinline__ float swap_add16(float v) {
  float w = v;
  asm("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(v), "+v"(w));
  return v + w;
}
__device__ __forceinline__ float swap_add32(float v) {
  float w = v;
  asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(v), "+v"(w));
  return v + w;
}
template <int Ctrl>
__device__ __forceinline__ float dpp_add(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), Ctrl, 0xf, 0xf, true);
  return v + __builtin_bit_cast(float, o);
}
// Sum over aligned groups of W = 2 .. 64 lanes, the same bits in every lane;
// exchanges within the vector unit, none through LDS.
template <int W>
__device__ __forceinline__ float lane_sum(float v) {
  v = dpp_add<0xb1>(v);                          // lane ^ 1
  if constexpr (W >= 4) v = dpp_add<0x4e>(v);    // lane ^ 2
  if constexpr (W >= 8) v = dpp_add<0x141>(v);   // mirrored in 8
  if constexpr (W >= 16) v = dpp_add<0x140>(v);  // mirrored in 16
  if constexpr (W >= 32) v = swap_add16(v);
  if constexpr (W >= 64) v = swap_add32(v);
  return v;
}

// The largest over aligned groups of W = 16 or 64 lanes, in every lane.
template <int Ctrl>
__device__ __forceinline__ float dpp_max(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), Ctrl, 0xf, 0xf, true);
  return __builtin_fmaxf(v, __builtin_bit_cast(float, o));
}
// over the lanes l, l ^ 16, l ^ 32 and l ^ 48
__device__ __forceinline__ float max_over_rows(float v) {
  float w = v;
  asm("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(v), "+v"(w));
  v = __builtin_fmaxf(v, w);
  w = v;
  asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(v), "+v"(w));
  return __builtin_fmaxf(v, w);
}
template <int W>
__device__ __forceinline__ float lane_max(float v) {
  v = dpp_max<0x140>(dpp_max<0x141>(dpp_max<0x4e>(dpp_max<0xb1>(v))));
  if constexpr (W == 64) v = max_over_rows(v);
  return v;
}

// 1 / (1 + e^-v); the reciprocal is the hardware's, within one unit of the last place
__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.f + __expf(-v)); }

}  // namespace kern
}  // namespace segpoly
