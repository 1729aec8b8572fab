// Matrix-core tile kernel of the gated feed-forward and the dense operators:
//   C[m, n] = sum over phases p and k of A_p[m, k] B_p[n, k]
// for 16-bit operands, float32 accumulation, and an epilogue on the
// accumulators.  Either operand is stored along k ([rows][k]) or across it
// ([k][rows]): the second form goes through the transposing LDS read, so no
// gradient product needs a transposed copy.  float32 operands come as three
// bf16 planes x = x1 + x2 + x3 (each the bf16 rounding of what is left: 24
// bits, the whole significand), and a product is the six plane pairs down to
// 2^-16 of the first, the smallest first; what is left out is at most 2^-23
// of it.  A step loads the three planes once for its six products.
//
// One workgroup computes a BM x BN tile in steps of KS k.  The operand tiles
// go from global memory to LDS directly (16 bytes a lane) into S buffers in
// turn, S - 1 steps ahead of the matrix instructions and with one barrier a
// step: the loads of a step have the time of S - 1 steps to land, which a
// small tile's step alone is too short for.  Such a load writes its wave's 64
// lanes in order, so the swizzle that keeps the fragment reads free of bank
// conflicts is applied to the global address: 16-byte slot s of row r holds
// chunk s ^ swizzle(r).  Rows, columns and k past the operand's end read as
// zero (the buffer descriptor's range check).  The matrix instruction gets
// the operands swapped, so a lane holds four neighbouring n of one m and
// stores them together.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../channel_ops.hpp"
#include "channel_types.hpp"
#include "mfma.hpp"

namespace segpoly {
namespace kern {

constexpr int kMaxBatch = 3;

struct GemmArgs {
  // plane k of phase p of batch z at [(z * phases + p) * planes + k]
  const uint16_t* a[kMaxBatch * 3];
  const uint16_t* b[kMaxBatch * 3];
  const uint16_t* b2[3];  // second B of a paired product (rows n of both belong together)
  int phases, batch;
  int64_t k;              // the sum over k of every phase
  // of each batch; lda, ldb in elements, multiples of 8
  int64_t m[kMaxBatch], n[kMaxBatch], lda[kMaxBatch], ldb[kMaxBatch], ldc[kMaxBatch];
  void* c[kMaxBatch];
  int64_t tiles_m[kMaxBatch], tiles_n[kMaxBatch];
  // workgroups (x, y) take the y-th share of the steps of a tile and store their
  // float32 sums split_stride elements apart
  int splits;
  int64_t split_stride;
  // epilogue of paired products
  uint16_t *h, *dg, *du;  // planes of [m][ldh], plane_stride apart
  const float* dh;        // [m][ldh]
  int64_t ldh, plane_stride;
  int act;
  // float16: exponents of blocks (scaled, below), [m / 64][e_ld] by n / 32; the
  // paired product's outputs, and of A and B at [z * phases + p], null: not scaled
  int *e_h, *e_dg, *e_du;
  const int *ea[kMaxBatch], *eb[kMaxBatch];
  int64_t e_ld;
  // epilogue of the dense operator, all of the io type: [n], [m][ld_res], either
  // null.  Forward: c = act(product + bias) + res.  Backward: res is the gradient
  // of the output; dg (of float32 operands [m][ldh] float32) and e_dg as above, and
  // the sums of dg's columns over each wave's rows, [column_rows][n up to a multiple
  // of four], or null.
  const void *bias, *res;
  int64_t ld_res, column_rows;  // tiles_m times the tile's waves along m, at most 2 ceil(m / 64) + 2
  float* column_sums;
};

enum { kEpiStore = 0, kEpiStoreF32 = 1, kEpiGated = 2, kEpiGatedBwd = 3, kEpiDense = 4, kEpiDenseBwd = 5 };

// io type T, matrix type E, planes per operand, products held in scaled blocks;
// staged: operands are read as they are (gemm_staged.hpp)
struct DtBF16 { using T = bf16; using E = bf16; static constexpr int kPlanes = 1; static constexpr bool kScaled = false; };
struct DtF16 { using T = f16; using E = f16; static constexpr int kPlanes = 1; static constexpr bool kScaled = true; };
// without scaled blocks: of products whose operands are the caller's
struct DtF16Plain { using T = f16; using E = f16; static constexpr int kPlanes = 1; static constexpr bool kScaled = false; };
struct DtF32 { using T = float; using E = bf16; static constexpr int kPlanes = 3; static constexpr bool kScaled = false; };
struct DtF32Staged : DtF32 {};
template <typename Dt>
constexpr bool kStaged = std::is_same_v<Dt, DtF32Staged>;

// float16 reaches from 2^-24 to 2^16.  A value that is held in it between two
// products can pass both ends where the inputs and the result do not, so its
// block is held times 2^-E: E = 0 while the block's largest finite value is
// between 2^-9 and 2^15, else a multiple of 8 that brings it between 2^7 and
// 2^15.  What a block's small values lose is then below 2^-16 of its largest, a
// sixteenth of what the largest loses in its own rounding.
constexpr int kReach = 64;      // below the largest exponent of a sum, values no longer count
constexpr int kNoValue = -128;  // the exponent of a block of zeros, infinities and NaN
__device__ __forceinline__ int block_exponent(float largest) {
  if (largest == 0.f) return kNoValue;
  const int e = static_cast<int>(__builtin_bit_cast(uint32_t, largest) >> 23) - 127;
  if (e >= -9 && e <= 14) return 0;
  const int scaled = (e - 14 + 7) >> 3 << 3;
  return scaled > -112 ? scaled : -112;
}
__device__ __forceinline__ float power_of_two(int e) {  // -126 .. 127
  return __builtin_bit_cast(float, (127 + e) << 23);
}
__device__ __forceinline__ float block_scale(int e) { return e == kNoValue ? 1.f : power_of_two(-e); }
__device__ __forceinline__ float finite_abs(float v) {
  v = __builtin_fabsf(v);
  return v < __builtin_inff() ? v : 0.f;
}

// Plane pairs of a float32 product, the smallest first.
constexpr int kPairs3[6][2] = {{2, 0}, {1, 1}, {0, 2}, {1, 0}, {0, 1}, {0, 0}};

using u16x8 = uint16_t __attribute__((ext_vector_type(8)));
using s16x4 = short __attribute__((ext_vector_type(4)));
using LdsS16x4 = __attribute__((address_space(3))) s16x4;
using LdsVoid = __attribute__((address_space(3))) void;

__device__ __forceinline__ v4f mma16(bf16, u16x8 a, u16x8 b, v4f c) {
  using V = bf16 __attribute__((ext_vector_type(8)));
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, 0, 0, 0);
}
__device__ __forceinline__ v4f mma16(f16, u16x8 a, u16x8 b, v4f c) {
  using V = f16 __attribute__((ext_vector_type(8)));
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, 0, 0, 0);
}

// x = sum of its three bf16 planes.  A value past the largest bf16 is cut
// instead of rounded up to infinity; infinities and NaN stay in plane 0.
__device__ __forceinline__ void split3(float x, bf16 (&p)[3]) {
  p[0] = static_cast<bf16>(x);
  float r = x - static_cast<float>(p[0]);
  if (!(__builtin_fabsf(static_cast<float>(p[0])) < __builtin_inff())) {
    const bool finite = __builtin_fabsf(x) < __builtin_inff();
    if (finite) p[0] = __builtin_bit_cast(bf16, static_cast<uint16_t>(__builtin_bit_cast(uint32_t, x) >> 16));
    r = finite ? x - static_cast<float>(p[0]) : 0.f;
  }
  p[1] = static_cast<bf16>(r);
  r -= static_cast<float>(p[1]);
  p[2] = static_cast<bf16>(r);
}

// The sum of the large products of planes and of the small ones.  An infinite
// or NaN operand is in a first plane, whose large products carry it; in the
// small ones it meets the zeros and either signs of other planes, which make
// NaN of an infinity, so they do not count then.
__device__ __forceinline__ v4f add_small(v4f large, v4f small) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (__builtin_fabsf(large[q]) < __builtin_inff()) large[q] += small[q];
  return large;
}

// The normal distribution function: half the complementary error function of
// |g| / sqrt(2), by the Chebyshev fit t exp(-x^2 + p(t)), t = 1 / (1 + x / 2), of
// Press et al., Numerical Recipes, whose relative error is below 1.2e-7 on the
// whole line.  The C library's form has two branches that a wave takes both of,
// several times the work.
__device__ __forceinline__ float normal_cdf(float g) {
  const float x = __builtin_fabsf(g) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(1.f + 0.5f * x);
  float p = 0.17087277f;
  p = p * t - 0.82215223f;
  p = p * t + 1.48851587f;
  p = p * t - 1.13520398f;
  p = p * t + 0.27886807f;
  p = p * t - 0.18628806f;
  p = p * t + 0.09678418f;
  p = p * t + 0.37409196f;
  p = p * t + 1.00002368f;
  p = p * t - 1.26551223f;
  const float c = 0.5f * t * __expf(p - x * x);
  return g < 0.f ? c : 1.f - c;
}

__device__ __forceinline__ float act_value(float g, int act) {
  if (act == kActSilu) return g * sigmoid(g);
  if (act == kActGelu) return g * normal_cdf(g);
  if (act == kActRelu) return g > 0.f ? g : (g != g ? g : 0.f);
  return sigmoid(g);
}
__device__ __forceinline__ void act_both(float g, int act, float& a, float& da) {
  if (act == kActSilu) {
    const float s = sigmoid(g);
    a = g * s;
    da = s * (1.f + g * (1.f - s));
  } else if (act == kActGelu) {
    const float p = normal_cdf(g);
    a = g * p;
    da = p + g * __expf(-0.5f * g * g) * 0.39894228040143268f;
  } else if (act == kActRelu) {
    a = act_value(g, act);
    da = g > 0.f ? 1.f : 0.f;
  } else {
    a = sigmoid(g);
    da = a * (1.f - a);
  }
}

// `body` with the activation as a compile-time constant: a branch per value costs
// more than the value (200000 x 64 x 200 bf16 forward 129 us with it, 72 without)
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& body) {
  if (act == kActNone) return body(std::integral_constant<int, kActNone>{});
  if (act == kActSilu) return body(std::integral_constant<int, kActSilu>{});
  if (act == kActGelu) return body(std::integral_constant<int, kActGelu>{});
  if (act == kActRelu) return body(std::integral_constant<int, kActRelu>{});
  return body(std::integral_constant<int, kActSigmoid>{});
}
template <typename Act>
__device__ __forceinline__ float dense_act(Act, float z) {
  if constexpr (Act::value == kActNone)
    return z;
  else
    return act_value(z, Act::value);
}
// the slope alone
template <typename Act>
__device__ __forceinline__ float dense_slope(Act, float z) {
  float value, slope = 1.f;
  if constexpr (Act::value != kActNone) act_both(z, Act::value, value, slope);
  return slope;
}

// four columns of a row from n on, zeros past its width
template <typename T>
__device__ __forceinline__ v4f load_four(const T* row, int64_t n, int64_t width) {
  T t[4] = {T(0.f), T(0.f), T(0.f), T(0.f)};
  if (n + 4 <= width) {
    __builtin_memcpy(t, row + n, sizeof(t));
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (n + q < width) t[q] = row[n + q];
  }
  return v4f{static_cast<float>(t[0]), static_cast<float>(t[1]), static_cast<float>(t[2]), static_cast<float>(t[3])};
}

// a fragment times 2^d, d <= 0: in two steps, for one that takes all of float16's
// values to zero is itself below it, and would make NaN of an infinity
__device__ __forceinline__ u16x8 lower(u16x8 v, int d) {
  using F8 = f16 __attribute__((ext_vector_type(8)));
  const int d1 = d > -24 ? d : -24, d2 = d - d1 > -24 ? d - d1 : -24;
  const F8 f = __builtin_bit_cast(F8, v) * static_cast<f16>(power_of_two(d1));
  return __builtin_bit_cast(u16x8, f * static_cast<f16>(power_of_two(d2)));
}

// ------------------------------------------------------------ operand tiles

// A tile of R rows and KS k in LDS; Across: stored [k][R], else [R][k].
template <int R, int KS, int Waves, bool Across>
struct TileLoad {
  static constexpr int kInstr = R * KS / 512 / Waves;  // 1 KB each
  static constexpr int kRowChunks = (Across ? R : KS) / 8;
  static_assert(kInstr >= 1, "every wave loads");
  // Swizzle of a row.  Stored along k: the 16 rows of a fragment read are 128
  // (64) bytes apart.  A 16-byte read goes out in groups of 16 lanes such as
  // 0-3, 12-15, 20-23, 24-27, that is rows 0-3 and 12-15 of one chunk with rows
  // 4-11 of the next: those get different 16-byte columns of the 256 bytes
  // that the banks span.  Across: the 16 k that one transposing read of a
  // wave touches get 16 (fewer: as many as fit) different 32-byte columns.
  __device__ __forceinline__ static int fold(int row) {
    if constexpr (Across) return (2 * (row % 4 + 4 * (row / 8))) % kRowChunks;
    if constexpr (KS == 64) return row % 8;
    const int x = row / 4 % 4;  // 0, 2, 3, 1
    return ((x ^ x / 2) & 1) * 2 + x / 2;
  }
  // which chunk of its row a lane loads: the same for every instruction of a tile stored along k
  __device__ __forceinline__ static int lane_chunk(int lane) {
    return KS == 64 ? (lane % 8) ^ fold(lane / 8) : (lane % 4) ^ fold(lane / 4);
  }

  uint32_t off[kInstr];  // byte offset of the lane's chunk from the tile's corner (paired: its half's)
  template <bool Pair>
  __device__ __forceinline__ void init(int64_t ld, int wave, int lane) {
#pragma unroll
    for (int j = 0; j < kInstr; ++j) {
      const int unit = (j * Waves + wave) * 64 + lane;
      const int row = unit / kRowChunks, slot = unit % kRowChunks;
      off[j] = static_cast<uint32_t>((Pair ? row % (R / 2) : row) * ld * 2 + (slot ^ fold(row)) * 16);
    }
  }
  // an instruction of the second half of a paired tile (whole rows: the same for a wave's lanes)
  __device__ __forceinline__ static bool second(int j, int wave) {
    return (j * Waves + wave) * 64 / kRowChunks >= R / 2;
  }
  template <typename F>
  __device__ __forceinline__ void issue(uint16_t* lds, int wave, bool past, F&& rsrc) const {
#pragma unroll
    for (int j = 0; j < kInstr; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(j), (LdsVoid*)(lds + (j * Waves + wave) * 512), 16,
                                               past ? 0x80000000u : off[j], 0, 0, 0);
  }
};

template <int R, int KS, bool Across>
__device__ __forceinline__ u16x8 read_fragment(const uint16_t* lds, int row0, int kk, int lane) {
  using Tile = TileLoad<R, KS, 1, Across>;
  if constexpr (!Across) {
    const int r = row0 + lane % 16, chunk = kk * 4 + lane / 16;
    return *reinterpret_cast<const u16x8*>(lds + r * KS + ((chunk ^ Tile::fold(r)) * 8));
  } else {
    const int i = lane % 16, k = kk * 32 + lane / 16 * 8 + i / 4;
    const int chunk = row0 / 8 + i % 4 / 2;
    const uint16_t* p = lds + k * R + ((chunk ^ Tile::fold(k)) * 8) + i % 2 * 4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4*)(p + 4 * R));
    using S8 = short __attribute__((ext_vector_type(8)));
    const S8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(u16x8, v);
  }
}

// `left` bytes from p on; nothing past 2^31 bytes is addressed from one tile corner
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const char* p, int64_t left) {
  const int bytes = left < 0x7fffffff ? (left > 0 ? static_cast<int>(left) : 0) : 0x7fffffff;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), 0, bytes, 0x00020000);
}

// ------------------------------------------------------------ the kernel

// at most N vector memory accesses outstanding, none of LDS, then the barrier;
// nothing moves across it
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | N / 16 << 14);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The buffers of a tile, declared by the kernel: one object per operand and
// buffer, so that the compiler has a fragment read wait for direct loads into
// its own object only.
template <typename Dt, int BM, int BN, int KS, int S>
struct TileLds {
  static constexpr int kA = Dt::kPlanes * BM * KS, kB = Dt::kPlanes * BN * KS;
  static constexpr int kA2 = S > 2 ? kA : 8, kB2 = S > 2 ? kB : 8, kA3 = S > 3 ? kA : 8, kB3 = S > 3 ? kB : 8;
};
#define SEGPOLY_TILE_LDS(L)                                        \
  __shared__ __attribute__((aligned(16))) uint16_t a0[L::kA];      \
  __shared__ __attribute__((aligned(16))) uint16_t b0[L::kB];      \
  __shared__ __attribute__((aligned(16))) uint16_t a1[L::kA];      \
  __shared__ __attribute__((aligned(16))) uint16_t b1[L::kB];      \
  __shared__ __attribute__((aligned(16))) uint16_t a2[L::kA2];     \
  __shared__ __attribute__((aligned(16))) uint16_t b2[L::kB2];     \
  __shared__ __attribute__((aligned(16))) uint16_t a3[L::kA3];     \
  __shared__ __attribute__((aligned(16))) uint16_t b3[L::kB3]

// Workgroups go round the eight dies, each with its own L2: give each die
// a run of neighbouring tiles, in bands of eight tile rows.
template <int BM, int BN>
__device__ __forceinline__ void tile_corner(int64_t id, int64_t tiles_m, int64_t tiles_n, int64_t& m0, int64_t& n0) {
  const int64_t die = id % 8, tiles = tiles_m * tiles_n, q = tiles / 8, r = tiles % 8;
  const int64_t t = die * q + (die < r ? die : r) + id / 8;
  const int64_t band = t / (8 * tiles_n), in_band = t % (8 * tiles_n);
  const int64_t band_rows = tiles_m - band * 8 < 8 ? tiles_m - band * 8 : 8;
  m0 = (band * 8 + in_band % band_rows) * BM;
  n0 = in_band / band_rows * BN;
}

// The results of a BM x BN tile, 16 bits each, to rows m < gm, columns n < width of
// `to`.  A fragment's lanes hold four columns of sixteen rows, 32 bytes of a line:
// they go through LDS, 64 rows to a buffer, and leave in whole lines.  16-byte slot
// s of row r holds chunk s ^ r, so that sixteen rows of a column fall into different
// banks.  value(i, j, q): element q of the wave's fragment (i, j).
template <int BM, int BN, int WM, int WN, typename V, typename F>
__device__ __forceinline__ void store_lines(uint16_t* q0, uint16_t* q1, V* to, int64_t ld, int64_t m0, int64_t n0,
                                            int64_t gm, int64_t width, F&& value) {
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16, kThreads = WM * WN * 64, kChunks = BN / 8;
  static_assert(sizeof(V) == 2 && BM <= 128 && kThreads / kChunks <= 64, "a pass of the threads is within a buffer");
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wm = wave / WN, wn = wave % WN;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int first = wm * (BM / WM) + i * 16, r = first % 64 + lane % 16;
    uint16_t* at = (first < 64 ? q0 : q1) + r * BN;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int c = wn * (BN / WN) + j * 16 + lane / 16 * 4;
      const V v[4] = {value(i, j, 0), value(i, j, 1), value(i, j, 2), value(i, j, 3)};
      __builtin_memcpy(at + ((c / 8 ^ r % kChunks) * 8) + c % 8, v, 8);
    }
  }
  wait_and_meet<63>();
#pragma unroll
  for (int t = 0; t < BM * kChunks / kThreads; ++t) {
    const int u = t * kThreads + static_cast<int>(threadIdx.x), r = u / kChunks, c = u % kChunks;
    const uint16_t* from = (t * kThreads / kChunks < 64 ? q0 : q1) + r % 64 * BN + (c ^ r % kChunks) * 8;
    const int64_t m = m0 + r, n = n0 + c * 8;
    if (m >= gm || n >= width) continue;
    const u16x8 v = *reinterpret_cast<const u16x8*>(from);
    V* row = to + m * ld + n;
    if (n + 8 <= width) {
      __builtin_memcpy(row, &v, 16);
    } else {
#pragma unroll
      for (int q = 0; q < 7; ++q)
        if (n + q < width) row[q] = __builtin_bit_cast(V, static_cast<uint16_t>(v[q]));
    }
  }
}

// The epilogue of a product with one output: a tile's sums, batch z, corner (m0, n0).
template <typename Dt, int BM, int BN, int WM, int WN, int KS, int Epi>
__device__ __forceinline__ void finish_tile(const GemmArgs& g, int z, int64_t m0, int64_t n0, int share,
                                            v4f (&acc)[BM / WM / 16][BN / WN / 16], uint16_t* a0, uint16_t* b0) {
  using E = typename Dt::E;
  constexpr bool kDense = Epi == kEpiDense || Epi == kEpiDenseBwd;
  constexpr int P = Dt::kPlanes, FM = BM / WM / 16, FN = BN / WN / 16;
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wm = wave / WN, wn = wave % WN;
  const int64_t gm = g.m[z], gn = g.n[z];
  using T = std::conditional_t<Epi == kEpiStoreF32, float, typename Dt::T>;
  const int64_t row0 = m0 + wm * (BM / WM) + lane % 16, col0 = n0 + wn * (BN / WN) + lane / 16 * 4;
  if constexpr (kDense) {
    v4f bias[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j)
      bias[j] = g.bias ? load_four(static_cast<const T*>(g.bias), col0 + j * 16, gn) : v4f{0.f, 0.f, 0.f, 0.f};
    with_act(g.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int64_t m = row0 + i * 16;
        const T* row = static_cast<const T*>(g.res) + (m < gm ? m : 0) * g.ld_res;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          v4f r = {0.f, 0.f, 0.f, 0.f};
          if (g.res && m < gm) r = load_four(row, col0 + j * 16, gn);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float z = acc[i][j][q] + bias[j][q];
            acc[i][j][q] = Epi == kEpiDense ? dense_act(act, z) + r[q] : r[q] * dense_slope(act, z);
          }
        }
      }
    });
    // d past the last row and column is zero whatever its slope, which an infinity times the operands' zeros there
    // makes NaN: the column sums take the rows, the next product the columns up to a multiple of eight
    if (Epi == kEpiDenseBwd && (m0 + BM > gm || n0 + BN > gn)) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (row0 + i * 16 >= gm || col0 + j * 16 + q >= gn) acc[i][j][q] = 0.f;
    }
  }
  // float32 rows: 16 bytes a lane, 64 of a row together
  auto store_rows = [&](T* to, int64_t ld) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t m = row0 + i * 16;
      if (m >= gm) continue;
      T* row = to + m * ld;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int64_t n = col0 + j * 16;
        T v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = static_cast<T>(acc[i][j][q]);
        if (n + 4 <= gn) {
          __builtin_memcpy(row + n, v, sizeof(v));
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (n + q < gn) row[n + q] = v[q];
        }
      }
    }
  };
  static_assert(!kDense || P > 1 || (64 * BN <= BM * KS && 64 * BN <= BN * KS), "64 rows fit in a buffer");
  if constexpr (Epi == kEpiDense && P == 1) {
    wait_and_meet<0>();  // every wave has read its last fragments
    store_lines<BM, BN, WM, WN>(a0, b0, static_cast<T*>(g.c[z]), g.ldc[z], m0, n0, gm, gn,
                                [&](int i, int j, int q) { return static_cast<T>(acc[i][j][q]); });
  } else if constexpr (Epi != kEpiDenseBwd) {
    store_rows(static_cast<T*>(g.c[z]) + (Epi == kEpiStoreF32 ? g.split_stride * share : 0), g.ldc[z]);
  } else {
    if (g.column_sums) {
      float* sums = g.column_sums + (m0 / BM * WM + wm) * ((gn + 3) / 4 * 4);
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float s = 0.f;
#pragma unroll
          for (int i = 0; i < FM; ++i) s += acc[i][j][q];
          s = lane_sum<16>(s);
          const int64_t n = col0 + j * 16 + q;
          if (lane % 16 == 0 && n < gn) sums[n] = s;
        }
    }
    if constexpr (P > 1) return store_rows(reinterpret_cast<float*>(g.dg), g.ldh);
    wait_and_meet<0>();  // every wave has read its last fragments
    if constexpr (Dt::kScaled) {
      constexpr int kRows = BM / WM > 64 ? BM / WM / 64 : 1, kCols = BN / WN / 32, kPer = FM / kRows;
      static_assert(BM == 64 ? WM == 2 && BN / WN == 32 : BM / WM % 64 == 0 && BN / WN % 32 == 0,
                    "a wave holds whole blocks, or half of one");
#pragma unroll
      for (int b = 0; b < kRows; ++b)
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          float top = 0.f;
#pragma unroll
          for (int i = b * kPer; i < (b + 1) * kPer; ++i)
#pragma unroll
            for (int j = c * 2; j < c * 2 + 2; ++j)
#pragma unroll
              for (int q = 0; q < 4; ++q) top = __builtin_fmaxf(top, finite_abs(acc[i][j][q]));
          top = lane_max<64>(top);
          if constexpr (BM == 64) {
            float* shared = reinterpret_cast<float*>(b0);
            if (lane == 0) shared[wave] = top;
            wait_and_meet<63>();
            top = __builtin_fmaxf(shared[wn], shared[WN + wn]);
          }
          const int e = block_exponent(top);
          const float scale = block_scale(e);
#pragma unroll
          for (int i = b * kPer; i < (b + 1) * kPer; ++i)
#pragma unroll
            for (int j = c * 2; j < c * 2 + 2; ++j) acc[i][j] *= scale;
          const int64_t m = m0 + wm * (BM / WM) + b * 64, n = n0 + wn * (BN / WN) + c * 32;
          if (lane == 0 && (BM > 64 || wm == 0) && m < gm && n < gn) g.e_dg[m / 64 * g.e_ld + n / 32] = e;
        }
    }
    if constexpr (P == 1)  // rows of the products' operands are read in 16-byte chunks
      store_lines<BM, BN, WM, WN>(a0, b0, reinterpret_cast<E*>(g.dg), g.ldh, m0, n0, gm, (gn + 7) / 8 * 8,
                                  [&](int i, int j, int q) { return static_cast<E>(acc[i][j][q]); });
  }
}

// Tile `id` of the batches' tiles, share `share` of its steps.
template <typename Dt, int BM, int BN, int WM, int WN, int KS, int S, bool AAcross, bool BAcross, int Epi>
__device__ __forceinline__ void gemm_tile(const GemmArgs& g, int64_t id, int share, uint16_t* a0, uint16_t* b0,
                                          uint16_t* a1, uint16_t* b1, uint16_t* a2, uint16_t* b2, uint16_t* a3,
                                          uint16_t* b3) {
  using E = typename Dt::E;
  constexpr bool kPair = Epi == kEpiGated || Epi == kEpiGatedBwd, kDense = Epi == kEpiDense || Epi == kEpiDenseBwd;
  constexpr bool kUnits = Dt::kScaled && !kPair && !kDense;  // operands may come in scaled blocks
  constexpr int kWaves = WM * WN, P = Dt::kPlanes;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // fragments per wave
  constexpr int kStageA = P * BM * KS, kStageB = P * BN * KS;
  static_assert(S >= 2 && S <= 4, "buffers");
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wm = wave / WN, wn = wave % WN;

  int z = 0;
  if constexpr (!kPair) {
    while (z + 1 < g.batch && id >= g.tiles_m[z] * g.tiles_n[z]) id -= g.tiles_m[z] * g.tiles_n[z], ++z;
  }
  const int64_t gm = g.m[z], gn = g.n[z], lda = g.lda[z], ldb = g.ldb[z], tiles_m = g.tiles_m[z], tiles_n = g.tiles_n[z];

  int64_t m0, n0;
  tile_corner<BM, kPair ? BN / 2 : BN>(id, tiles_m, tiles_n, m0, n0);

  TileLoad<BM, KS, kWaves, AAcross> la;
  TileLoad<BN, KS, kWaves, BAcross> lb;
  la.template init<false>(lda, wave, lane);
  lb.template init<kPair>(ldb, wave, lane);
  // rows are held (along k: with zeros) up to a multiple of eight elements, and
  // the range check drops a whole chunk that crosses the end
  const int64_t k8 = (g.k + 7) / 8 * 8, m8 = (gm + 7) / 8 * 8, n8 = (gn + 7) / 8 * 8;
  const int64_t fa = AAcross ? m0 : m0 * lda, fb = BAcross ? n0 : n0 * ldb;  // the tile's corners
  const int64_t left_a0 = ((AAcross ? (g.k - 1) * lda + m8 : (gm - 1) * lda + k8) - fa) * 2;
  const int64_t left_b0 = ((BAcross ? (g.k - 1) * ldb + n8 : (gn - 1) * ldb + k8) - fb) * 2;
  const int step_a = static_cast<int>(AAcross ? KS * lda * 2 : KS * 2);  // bytes
  const int step_b = static_cast<int>(BAcross ? KS * ldb * 2 : KS * 2);

  // this workgroup's share of the steps of all phases, one at least
  const int64_t steps = (g.k + KS - 1) / KS;
  const int64_t s0 = kPair ? 0 : steps * g.phases * share / g.splits;
  int left = static_cast<int>((kPair ? steps : steps * g.phases * (share + 1) / g.splits) - s0);
  int to_load = left;

  // the next step to load: its k left, its corners and the bytes from there to the operands' ends
  int phase = 0, k_left = 0;
  int64_t left_a = 0, left_b = 0;
  const char *pa[P], *pb[P], *pb2[P];
  auto matrices = [&] {
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const int at = (z * g.phases + phase) * P + q;
      pa[q] = reinterpret_cast<const char*>(g.a[at] + fa);
      pb[q] = reinterpret_cast<const char*>(g.b[at] + fb);
      if constexpr (kPair) pb2[q] = reinterpret_cast<const char*>(g.b2[at] + fb);
    }
    k_left = static_cast<int>(g.k);
    left_a = left_a0;
    left_b = left_b0;
  };
  phase = static_cast<int>(s0 / steps);
  matrices();
  const int64_t skip = s0 % steps;
#pragma unroll
  for (int q = 0; q < P; ++q) {
    pa[q] += skip * step_a;
    pb[q] += skip * step_b;
  }
  left_a -= skip * step_a;
  left_b -= skip * step_b;
  k_left -= static_cast<int>(skip * KS);
  // Loads are issued for exactly S - 1 steps past the last one too (of nothing:
  // the range is empty), so that the count of those outstanding is the same in
  // every step, for the wait below and for the compiler's own.
  auto issue = [&](uint16_t* to_a, uint16_t* to_b) {
    // the last step ends inside a row stored along k: chunks at or past k read out of range, that is zero
    const bool a_past = !AAcross && la.lane_chunk(lane) * 8 >= k_left;
    const bool b_past = !BAcross && lb.lane_chunk(lane) * 8 >= k_left;
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const __amdgpu_buffer_rsrc_t ra = make_rsrc(pa[q], left_a);
      la.issue(to_a + q * BM * KS, wave, a_past, [&](int) { return ra; });
      pa[q] += step_a;
    }
#pragma unroll
    for (int q = 0; q < P; ++q) {
      uint16_t* to = to_b + q * BN * KS;
      if constexpr (kPair) {
        lb.issue(to, wave, b_past, [&](int j) { return make_rsrc(lb.second(j, wave) ? pb2[q] : pb[q], left_b); });
        pb2[q] += step_b;
      } else {
        const __amdgpu_buffer_rsrc_t rb = make_rsrc(pb[q], left_b);
        lb.issue(to, wave, b_past, [&](int) { return rb; });
      }
      pb[q] += step_b;
    }
    left_a -= step_a;
    left_b -= step_b;
    k_left -= KS;
    if (--to_load <= 0) {
      left_a = left_b = 0;
    } else if (k_left <= 0) {
      ++phase;
      matrices();
    }
  };

  v4f acc[FM][FN];
  // the five small products of float32 planes are summed apart: added to the
  // large sum one by one they would round it six times as often
  v4f small[P > 1 ? FM : 1][P > 1 ? FN : 1];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
      if constexpr (P > 1) small[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    }

  // Scaled blocks of this wave's rows of A, or B: a group of fragments per block
  // across the sum.  A group's sum is in units of its present block's exponent
  // and changes them with it (but not by more than kReach from the largest, for
  // float32's range).  Ordinary values have exponents of zero everywhere, which
  // one look over them before the first step shows, while its loads are on their
  // way.
  constexpr int GA = (BM / WM) / (AAcross ? 32 : 64) > 1 ? (BM / WM) / (AAcross ? 32 : 64) : 1;
  constexpr int GB = BN / WN / 32 > 1 ? BN / WN / 32 : 1;
  constexpr bool kScaledB = AAcross && BAcross;  // the other products' B is a weight
  int unit_a[GA] = {}, unit_b[GB] = {}, least_a[GA] = {}, least_b[GB] = {};
  bool mixed = false, in_units = false;
  int64_t now = s0;  // the step that compute works on
  // exponents of one group along the sum: first, distance and number; the last
  // step's second half can be past the last, and a group past the last row (not
  // stored) has the last one's
  struct Along {
    const int* e;
    int64_t step;
    int count;
    __device__ __forceinline__ int at(int t) const { return e[(t < count ? t : count - 1) * step]; }
  };
  auto along = [&](const int* e, int64_t r, int64_t rows, bool across) {
    r = r < rows ? r : rows - 1;
    return across ? Along{e + r / 32, g.e_ld, static_cast<int>((g.k + 63) / 64)}
                  : Along{e + r / 64 * g.e_ld, 1, static_cast<int>((g.k + 31) / 32)};
  };
  auto along_a = [&](int p, int q) {
    return along(g.ea[z * g.phases + p], m0 + wm * (BM / WM) + q * (AAcross ? 32 : 64), gm, AAcross);
  };
  auto along_b = [&](int p, int q) {
    return along(g.eb[z * g.phases + p], n0 + wn * (BN / WN) + q * 32, gn, true);
  };
  // the first look: 256 exponents of each group and phase (one or two), loaded
  // before the first step's operands and waited for after them
  int seen_a[2][GA][4] = {}, seen_b[2][GB][4] = {};
  auto load_seen = [&](auto&& group, auto& seen) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int q = 0; q < static_cast<int>(sizeof(seen[0]) / 16); ++q)
#pragma unroll
        for (int u = 0; u < 4; ++u) seen[p][q][u] = group(p < g.phases ? p : 0, q).at(u * 64 + lane);
  };
  auto look = [&](auto&& group, auto& seen, auto& unit, auto& least) {
    constexpr int G = sizeof(unit) / sizeof(int);
    bool other = false;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int q = 0; q < G; ++q)
#pragma unroll
        for (int u = 0; u < 4; ++u) other |= seen[p][q][u] != 0 && seen[p][q][u] != kNoValue;
    for (int p = 0; p < g.phases; ++p)
      for (int t = 256 + lane; t < group(p, 0).count; t += 64)
#pragma unroll
        for (int q = 0; q < G; ++q) {
          const int e = group(p, q).at(t);
          other |= e != 0 && e != kNoValue;
        }
    if (__ballot(other) == 0) return;
#pragma unroll
    for (int q = 0; q < G; ++q) {
      float hi = kNoValue, lo = -kNoValue;
      for (int p = 0; p < g.phases; ++p)
        for (int t = lane; t < group(p, q).count; t += 64) {
          const int e = group(p, q).at(t);
          if (e == kNoValue) continue;
          hi = __builtin_fmaxf(hi, static_cast<float>(e));
          lo = __builtin_fminf(lo, static_cast<float>(e));
        }
      const int top = __builtin_amdgcn_readfirstlane(static_cast<int>(lane_max<64>(hi + 128.f))) - 128;
      const int low = 128 - __builtin_amdgcn_readfirstlane(static_cast<int>(lane_max<64>(128.f - lo)));
      if (top == kNoValue) continue;
      unit[q] = top;
      least[q] = top - kReach;
      mixed |= low != top;
      in_units |= mixed || top != 0;
    }
  };
  // exponent e comes next in a group: its sum changes units, or its fragments are
  // lowered to them where the exponent is out of reach
  auto enter = [&](int e, int& unit, int least, auto&& sums, auto&& fragments) {
    if (e == kNoValue) return;
    const int to = e > least ? e : least;
    if (to != unit) sums(power_of_two(unit - to));
    unit = to;
    if (e < to) fragments(e - to);
  };

  // paired: the wave's first FN/2 fragments are of B, the others of B2
  auto b_row = [&](int j) {
    if constexpr (kPair)
      return (j < FN / 2 ? 0 : BN / 2) + wn * (BN / 2 / WN) + (j % (FN / 2)) * 16;
    else
      return wn * (BN / WN) + j * 16;
  };
  auto compute = [&](auto units, const uint16_t* at_a, const uint16_t* at_b) {
#pragma unroll
    for (int kk = 0; kk < KS / 32; ++kk) {
      // the transposing reads of two halves at once do not fit in the registers beside a large tile
      if (AAcross && BAcross && FM * FN >= 32 && kk > 0) asm volatile("" ::: "memory");
      u16x8 fa[P][FM], fb[P][FN];
#pragma unroll
      for (int q = 0; q < P; ++q) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
          fb[q][j] = read_fragment<BN, KS, BAcross>(at_b + q * BN * KS, b_row(j), kk, lane);
#pragma unroll
        for (int i = 0; i < FM; ++i)
          fa[q][i] = read_fragment<BM, KS, AAcross>(at_a + q * BM * KS, wm * (BM / WM) + i * 16, kk, lane);
      }
      if constexpr (units) {
        const int p = static_cast<int>(now / steps);
        const int at = static_cast<int>(now % steps) * KS + kk * 32;
        constexpr int NA = FM / GA, NB = FN / GB;
#pragma unroll
        for (int q = 0; q < GA; ++q) {
          if (!g.ea[z * g.phases]) continue;
          auto sums = [&](float f) {
#pragma unroll
            for (int i = q * NA; i < (q + 1) * NA; ++i)
#pragma unroll
              for (int j = 0; j < FN; ++j) acc[i][j] *= f;
          };
          auto fragments = [&](int d) {
#pragma unroll
            for (int i = q * NA; i < (q + 1) * NA; ++i) fa[0][i] = lower(fa[0][i], d);
          };
          enter(along_a(p, q).at(at / (AAcross ? 64 : 32)), unit_a[q], least_a[q], sums, fragments);
        }
#pragma unroll
        for (int q = 0; q < (kScaledB ? GB : 0); ++q) {
          if (!g.eb[z * g.phases]) continue;
          auto sums = [&](float f) {
#pragma unroll
            for (int j = q * NB; j < (q + 1) * NB; ++j)
#pragma unroll
              for (int i = 0; i < FM; ++i) acc[i][j] *= f;
          };
          auto fragments = [&](int d) {
#pragma unroll
            for (int j = q * NB; j < (q + 1) * NB; ++j) fb[0][j] = lower(fb[0][j], d);
          };
          enter(along_b(p, q).at(at / 64), unit_b[q], least_b[q], sums, fragments);
        }
      }
      constexpr int kProducts = P == 1 ? 1 : 6;
#pragma unroll
      for (int t = 0; t < kProducts; ++t)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            if constexpr (P == 1) {
              acc[i][j] = mma16(E{}, fb[0][j], fa[0][i], acc[i][j]);
            } else {
              v4f& c = t < kProducts - 1 ? small[i][j] : acc[i][j];
              c = mma16(E{}, fb[kPairs3[t][1]][j], fa[kPairs3[t][0]][i], c);
            }
          }
    }
  };

  constexpr int kLoads = P * (la.kInstr + lb.kInstr);  // of a wave in a step
  // One step: its own loads have landed (those of the S - 2 steps after it may
  // not have) and the buffer read a step ago is free for the one S - 1 ahead.
  auto step = [&](auto units, uint16_t* now_a, uint16_t* now_b, uint16_t* ahead_a, uint16_t* ahead_b) {
    wait_and_meet<(S - 2) * kLoads>();
    issue(ahead_a, ahead_b);
    compute(units, now_a, now_b);
    if constexpr (units) ++now;
  };
  auto first = [&](auto units) {
    if constexpr (S == 2)
      step(units, a0, b0, a1, b1);
    else if constexpr (S == 3)
      step(units, a0, b0, a2, b2);
    else
      step(units, a0, b0, a3, b3);
  };
  // whole turns of the buffers, then what is left: a loop with exits between
  // the steps would have the compiler wait for loads that are not due
  auto run = [&](auto units) {
    for (; left >= S; left -= S) {
      first(units);
      step(units, a1, b1, a0, b0);
      if constexpr (S > 2) step(units, a2, b2, a1, b1);
      if constexpr (S > 3) step(units, a3, b3, a2, b2);
    }
    if (left > 0) {
      first(units);
      if (S > 2 && left > 1) {
        step(units, a1, b1, a0, b0);
        if (S > 3 && left > 2) step(units, a2, b2, a1, b1);
      }
    }
  };
  if constexpr (kUnits) {
    if (g.ea[z * g.phases]) load_seen(along_a, seen_a);
    if constexpr (kScaledB)
      if (g.eb[z * g.phases]) load_seen(along_b, seen_b);
  }
  issue(a0, b0);
  if constexpr (S > 2) issue(a1, b1);
  if constexpr (S > 3) issue(a2, b2);
  if constexpr (kUnits) {
    if (g.ea[z * g.phases]) look(along_a, seen_a, unit_a, least_a);
    if constexpr (kScaledB)
      if (g.eb[z * g.phases]) look(along_b, seen_b, unit_b, least_b);
    // a loop of its own where units change: waves of a workgroup in either meet at the same barriers
    if (mixed)
      run(std::true_type{});
    else
      run(std::false_type{});
  } else {
    run(std::false_type{});
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);  // no load into LDS outlives the workgroup
  if constexpr (P > 1) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = add_small(acc[i][j], small[i][j]);
  }

  // ---------------------------------------------------------- epilogue
  if constexpr (!kPair) {
    if constexpr (kUnits) {
      if (in_units) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] *= power_of_two(unit_a[i / (FM / GA)]) * power_of_two(unit_b[j / (FN / GB)]);
      }
    }
    finish_tile<Dt, BM, BN, WM, WN, KS, Epi>(g, z, m0, n0, share, acc, a0, b0);
  } else {
    // A fragment's lanes hold four columns of sixteen rows, 32 bytes of a line:
    // the results go through LDS, one 16-bit plane after another in two buffers,
    // and leave in whole lines.  16-byte slot s of row r holds chunk s ^ r, so
    // that sixteen rows of a column fall into different banks.
    constexpr int kChunks = BN / 16;  // of a row
    constexpr bool kSplit = BM * BN / 2 > kStageA;  // the second half of the rows beside the first
    static_assert(!kSplit || (WM == 2 && BM * BN / 4 <= kStageA && BM * BN / 4 <= kStageB), "a plane fits in a buffer");
    const int64_t width = (gn + 7) / 8 * 8;  // rows of the products' operands are read in 16-byte chunks
    const int row0 = wm * (BM / WM) + lane % 16, col0 = wn * (BN / 2 / WN) + lane / 16 * 4;
    auto place = [&](uint16_t* lo, uint16_t* hi, int i, int j, const E(&e)[4]) {
      const int r = row0 + i * 16, c = col0 + j * 16, at = r * (BN / 2) + ((c / 8 ^ r % kChunks) * 8) + c % 8;
      if (kSplit && wm == 1)
        __builtin_memcpy(hi + (at - BM * BN / 4), e, 8);
      else
        __builtin_memcpy(lo + at, e, 8);
    };
    auto leave = [&](const uint16_t* lo, const uint16_t* hi, uint16_t* to) {
      wait_and_meet<63>();
#pragma unroll
      for (int t = 0; t < BM * kChunks / (kWaves * 64); ++t) {
        const int u = t * kWaves * 64 + static_cast<int>(threadIdx.x), r = u / kChunks, c = u % kChunks;
        const int at = r * (BN / 2) + (c ^ r % kChunks) * 8;
        const bool second = kSplit && t >= BM * kChunks / (kWaves * 128);
        const int64_t m = m0 + r, n = n0 + c * 8;
        if (m < gm && n < width)
          *reinterpret_cast<u16x8*>(to + m * g.ldh + n) =
              *reinterpret_cast<const u16x8*>(second ? hi + (at - BM * BN / 4) : lo + at);
      }
    };
    int turn = 0;
    // value(i, j, q): element q of a fragment, as a plane's type
    auto store = [&](uint16_t* to, auto value) {
      uint16_t *lo = turn % 2 ? a1 : a0, *hi = turn % 2 ? b1 : b0;
      ++turn;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN / 2; ++j) {
          const E e[4] = {value(i, j, 0), value(i, j, 1), value(i, j, 2), value(i, j, 3)};
          place(lo, hi, i, j, e);
        }
      leave(lo, hi, to);
    };
    auto plane = [&](float v, int p) {
      if constexpr (P == 1) {
        return static_cast<E>(v);
      } else {
        bf16 s[3];
        split3(v, s);
        return s[p];
      }
    };
    wait_and_meet<0>();  // every wave has read its last fragments
    // hidden columns past the last, which the next products read up to a multiple of eight, are zero: an infinity in a
    // row makes NaN of it and the weights' zeros there
    if (n0 + BN / 2 > gn) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN / 2; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (n0 + col0 + j * 16 + q >= gn) acc[i][j][q] = acc[i][j + FN / 2][q] = 0.f;
    }
    // dh of the wave's fragments
    constexpr int kD = Epi == kEpiGatedBwd ? 1 : 0;
    v4f d[kD ? FM : 1][kD ? FN / 2 : 1];
    auto load_dh = [&](int i, int j) {
      const int64_t m = m0 + row0 + i * 16, n = n0 + col0 + j * 16;
      v4f v = {0.f, 0.f, 0.f, 0.f};
      if (m < gm && n < width) __builtin_memcpy(&v, g.dh + m * g.ldh + n, sizeof(v));
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = n + q < gn ? v[q] : 0.f;
      return v;
    };
    // Scaled blocks: the exponents come of bounds of the block's largest values,
    // |h| <= max |g| max |u|, |dg| <= 1.13 max |dh| max |u| (1.13 bounds every
    // activation's derivative), |du| <= max |dh| max |g| (1 for |g| with a
    // sigmoid), a few times the values themselves, which are not known before the
    // activations are.
    constexpr int kBlocks = BM / WM > 64 ? BM / WM / 64 : 1, kPer = FM / kBlocks;
    float scale_h[kBlocks], scale_dg[kBlocks], scale_du[kBlocks];
    if constexpr (Dt::kScaled) {
      static_assert(BM == 64 ? BN == 64 : BM / WM % 64 == 0 && BN / 2 / WN == 32, "a wave holds whole blocks");
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        float top[3];
        auto largest = [&](auto&& magnitude) {
          top[0] = top[1] = top[2] = 0.f;
#pragma unroll
          for (int i = b * kPer; i < (b + 1) * kPer; ++i)
#pragma unroll
            for (int j = 0; j < FN / 2; ++j)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                top[0] = __builtin_fmaxf(top[0], magnitude(acc[i][j][q]));
                top[1] = __builtin_fmaxf(top[1], magnitude(acc[i][j + FN / 2][q]));
                if constexpr (kD) top[2] = __builtin_fmaxf(top[2], magnitude(d[i][j][q]));
              }
#pragma unroll
          for (int t = 0; t < 2 + kD; ++t) top[t] = lane_max<64>(top[t]);
        };
        if constexpr (kD)
#pragma unroll
          for (int i = b * kPer; i < (b + 1) * kPer; ++i)
#pragma unroll
            for (int j = 0; j < FN / 2; ++j) d[i][j] = load_dh(i, j);
        largest([](float v) { return __builtin_fabsf(v); });  // the largest passes over NaN
        if (!(__builtin_fmaxf(top[0], __builtin_fmaxf(top[1], top[2])) < __builtin_inff()))
          largest([](float v) { return finite_abs(v); });
        if constexpr (BM == 64) {  // one block, the workgroup's
          float* shared = reinterpret_cast<float*>(b0);
          if (lane == 0)
#pragma unroll
            for (int t = 0; t < 3; ++t) shared[t * kWaves + wave] = top[t];
          wait_and_meet<63>();
#pragma unroll
          for (int t = 0; t < 3; ++t)
#pragma unroll
            for (int w = 0; w < kWaves; ++w) top[t] = __builtin_fmaxf(top[t], shared[t * kWaves + w]);
        }
        const float value = g.act == kActSigmoid ? 1.f : top[0];
        const int eh = block_exponent(value * top[1]), eg = block_exponent(1.13f * top[2] * top[1]),
                  eu = block_exponent(top[2] * value);
        scale_h[b] = block_scale(eh), scale_dg[b] = block_scale(eg), scale_du[b] = block_scale(eu);
        const int64_t m = m0 + (BM == 64 ? 0 : wm * (BM / WM) + b * 64), n = n0 + (BM == 64 ? 0 : wn * 32);
        if (m < gm && n < gn && (BM == 64 ? threadIdx.x == 0 : lane == 0)) {
          const int64_t at = m / 64 * g.e_ld + n / 32;
          g.e_h[at] = eh;
          if constexpr (kD) g.e_dg[at] = eg, g.e_du[at] = eu;
        }
      }
    }
    // element v of fragment row i, of the values with these scales
    auto held = [&](float v, const float(&scale)[kBlocks], int i) {
      if constexpr (Dt::kScaled)
        return v * scale[i / kPer];
      else
        return v;
    };
    if constexpr (Epi == kEpiGated || P > 1) {
      v4f h[FM][FN / 2];
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN / 2; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) h[i][j][q] = act_value(acc[i][j][q], g.act) * acc[i][j + FN / 2][q];
#pragma unroll
      for (int p = 0; p < P; ++p)
        store(g.h + p * g.plane_stride, [&](int i, int j, int q) { return plane(held(h[i][j][q], scale_h, i), p); });
    }
    if constexpr (Epi == kEpiGatedBwd) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN / 2; ++j) {
          if constexpr (!Dt::kScaled) d[i][j] = load_dh(i, j);
          float h[4];
          // the gradients replace the two products
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float u = acc[i][j + FN / 2][q], dh = d[i][j][q];
            float v, dv;
            act_both(acc[i][j][q], g.act, v, dv);
            h[q] = held(v * u, scale_h, i);
            acc[i][j][q] = held(dh * u * dv, scale_dg, i);
            acc[i][j + FN / 2][q] = held(dh * v, scale_du, i);
          }
          if constexpr (P == 1) {
            const E e[4] = {static_cast<E>(h[0]), static_cast<E>(h[1]), static_cast<E>(h[2]), static_cast<E>(h[3])};
            place(a0, b0, i, j, e);
          }
        }
      if constexpr (P == 1) {  // the float32 form has stored h
        leave(a0, b0, g.h);
        turn = 1;
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        store(g.dg + p * g.plane_stride, [&](int i, int j, int q) { return plane(acc[i][j][q], p); });
        store(g.du + p * g.plane_stride, [&](int i, int j, int q) { return plane(acc[i][j + FN / 2][q], p); });
      }
    }
  }
}

template <typename Dt, int BM, int BN, int WM, int WN, int KS, int S, bool AAcross, bool BAcross, int Epi>
__global__ void __launch_bounds__(WM * WN * 64, 2)
gemm_tile_kernel(GemmArgs g) {
  using L = TileLds<Dt, BM, BN, KS, S>;
  SEGPOLY_TILE_LDS(L);
  gemm_tile<Dt, BM, BN, WM, WN, KS, S, AAcross, BAcross, Epi>(g, blockIdx.x, blockIdx.y, a0, b0, a1, b1, a2, b2, a3, b3);
}

// Two independent products in one launch, of 64 x 64 tiles: x with one operand
// across k, w with both; x has the first x_blocks workgroups, its shares side
// by side.
template <typename Dt, int KS, int S, int EpiX, int EpiW>
__global__ void __launch_bounds__(256, 2)
gemm_two_kernel(GemmArgs x, GemmArgs w, int64_t x_tiles, int64_t w_tiles) {
  using L = TileLds<Dt, 64, 64, KS, S>;
  SEGPOLY_TILE_LDS(L);
  const int64_t x_blocks = x_tiles * x.splits;
  if (blockIdx.x < x_blocks) {
    gemm_tile<Dt, 64, 64, 2, 2, KS, S, false, true, EpiX>(x, blockIdx.x % x_tiles, static_cast<int>(blockIdx.x / x_tiles),
                                                          a0, b0, a1, b1, a2, b2, a3, b3);
  } else {
    const int64_t id = blockIdx.x - x_blocks;
    gemm_tile<Dt, 64, 64, 2, 2, KS, S, true, true, EpiW>(w, id % w_tiles, static_cast<int>(id / w_tiles), a0, b0, a1, b1,
                                                         a2, b2, a3, b3);
  }
}

// The sum of the shares, in order, in the output's type: four columns a lane.
struct SplitSumArgs {
  static constexpr int kMax = kMaxBatch + 1;
  const float* from[kMax];
  void* to[kMax];
  int64_t m[kMax], n[kMax], ld[kMax], ldc[kMax], split_stride[kMax];
  int splits[kMax], batch;
};
template <typename T>
__global__ void __launch_bounds__(256)
split_sum_kernel(SplitSumArgs g) {
  const int z = blockIdx.y;
  const int64_t quads = g.ld[z] / 4, total = g.m[z] * quads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = i / quads;
    const int c = static_cast<int>(i % quads * 4);
    const float* from = g.from[z] + r * g.ld[z] + c;
    v4f s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int k = 0; k < g.splits[z]; ++k) s += *reinterpret_cast<const v4f*>(from + k * g.split_stride[z]);
    T* to = static_cast<T*>(g.to[z]) + r * g.ldc[z] + c;
    const T v[4] = {static_cast<T>(s[0]), static_cast<T>(s[1]), static_cast<T>(s[2]), static_cast<T>(s[3])};
    if (c + 4 <= g.n[z]) {
      __builtin_memcpy(to, v, sizeof(v));
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (c + q < g.n[z]) to[q] = v[q];
    }
  }
}

}  // namespace kern
}  // namespace segpoly
