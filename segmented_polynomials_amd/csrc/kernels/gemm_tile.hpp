// Matrix-core tile kernel of the gated feed-forward operator:
//   C[m, n] = sum over phases p and k of A_p[m, k] B_p[n, k]
// for 16-bit operands, float32 accumulation, and an epilogue on the
// accumulators.  Either operand is stored along k ([rows][k]) or across it
// ([k][rows]): the second form goes through the transposing LDS read, so no
// gradient product needs a transposed copy.  float32 operands come as three
// bf16 planes x = x1 + x2 + x3 (each the bf16 rounding of what is left: 24
// bits, the whole significand), and a product is the six phases of the plane
// pairs down to 2^-16 of the first; what is left out is below 2^-24 of it.
//
// One workgroup computes a BM x BN tile in steps of 64 k.  Both operand
// tiles go from global memory to LDS directly (16 bytes a lane), one step
// ahead of the matrix instructions, in two buffers and with one barrier a
// step.  Such a load writes its wave's 64 lanes in order, so the swizzle that
// keeps the fragment reads free of bank conflicts is applied to the global
// address: 16-byte slot s of row r holds chunk s ^ swizzle(r).  Rows, columns and k
// past the operand's end read as zero (the buffer descriptor's range check).
// The matrix instruction gets the operands swapped, so a lane holds four
// neighbouring n of one m and stores them together.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../channel_ops.hpp"
#include "channel_types.hpp"
#include "mfma.hpp"

namespace segpoly {
namespace kern {

constexpr int kStepK = 64;
constexpr int kMaxPhases = 24;

struct GemmArgs {
  const uint16_t* a[kMaxPhases];  // phase p of batch z at [z * phases + p]
  const uint16_t* b[kMaxPhases];
  const uint16_t* b2[kMaxPhases];  // second B of a paired product (rows n of both belong together)
  int phases, batch;
  int64_t m, n, k;        // k: steps run to round_up(k, 64); the operands end at k
  int64_t lda, ldb;       // elements; multiples of 8
  int64_t tiles_m, tiles_n;
  // epilogue
  void* c[2];             // per batch
  int64_t ldc;
  uint16_t *h, *dg, *du;  // paired products: planes of [m][ldh], plane_stride apart
  const void* dh;         // [m][ldh], the product's 16-bit type or float32
  int64_t ldh, plane_stride;
  int act;
};

enum { kEpiStore = 0, kEpiGated = 1, kEpiGatedBwd = 2 };

// io type T, matrix type E, type DH the hidden gradient is held in between its
// product and the gating, planes per operand
struct DtBF16 { using T = bf16; using E = bf16; using DH = bf16; static constexpr int kPlanes = 1; };
struct DtF16 { using T = f16; using E = f16; using DH = f16; static constexpr int kPlanes = 1; };
struct DtF32 { using T = float; using E = bf16; using DH = float; static constexpr int kPlanes = 3; };

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

__device__ __forceinline__ float act_value(float g, int act) {
  if (act == kActSilu) return g / (1.f + __expf(-g));
  if (act == kActGelu) return 0.5f * g * (1.f + erff(g * 0.70710678118654752f));
  if (act == kActRelu) return g > 0.f ? g : (g != g ? g : 0.f);
  return 1.f / (1.f + __expf(-g));
}
__device__ __forceinline__ void act_both(float g, int act, float& a, float& da) {
  if (act == kActSilu) {
    const float s = 1.f / (1.f + __expf(-g));
    a = g * s;
    da = s * (1.f + g * (1.f - s));
  } else if (act == kActGelu) {
    const float p = 0.5f * (1.f + erff(g * 0.70710678118654752f));
    a = g * p;
    da = p + g * __expf(-0.5f * g * g) * 0.39894228040143268f;
  } else if (act == kActRelu) {
    a = act_value(g, act);
    da = g > 0.f ? 1.f : 0.f;
  } else {
    a = 1.f / (1.f + __expf(-g));
    da = a * (1.f - a);
  }
}

// ------------------------------------------------------------ operand tiles

// A tile of R rows and 64 k in LDS; Across: stored [k][R], else [R][k].
template <int R, int Waves, bool Across>
struct TileLoad {
  static constexpr int kInstr = R / 8 / Waves;  // 1 KB each
  static constexpr int kRowChunks = Across ? R / 8 : 8;
  // swizzle of a [k][R] row: the 16 rows that one transposing read of a wave
  // touches get 16 (fewer: as many as fit) different 32-byte columns
  __device__ __forceinline__ static int fold(int k) { return (2 * (k % 4 + 4 * (k / 8))) % kRowChunks; }

  uint32_t off[kInstr];  // byte offset of the lane's chunk from the tile's corner
  __device__ __forceinline__ void init(int64_t ld, int wave, int lane) {
#pragma unroll
    for (int j = 0; j < kInstr; ++j) {
      const int unit = (j * Waves + wave) * 64 + lane;
      const int row = unit / kRowChunks, slot = unit % kRowChunks;
      const int chunk = Across ? slot ^ fold(row) : slot ^ (row % 8);
      off[j] = static_cast<uint32_t>(row * ld * 2 + chunk * 16);
    }
  }
  // k0: first k of the step; row0 may differ per instruction for paired B
  template <typename F>
  __device__ __forceinline__ void issue(uint16_t* lds, int wave, F&& rsrc) const {
#pragma unroll
    for (int j = 0; j < kInstr; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(j), (LdsVoid*)(lds + (j * Waves + wave) * 512), 16, off[j], 0, 0,
                                               0);
  }
};

template <int R, bool Across>
__device__ __forceinline__ u16x8 read_fragment(const uint16_t* lds, int row0, int kk, int lane) {
  if constexpr (!Across) {
    const int r = row0 + lane % 16, chunk = kk * 4 + lane / 16;
    return *reinterpret_cast<const u16x8*>(lds + r * 64 + ((chunk ^ (r % 8)) * 8));
  } else {
    using Tile = TileLoad<R, 1, true>;
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

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const uint16_t* base, int64_t first, int64_t end) {
  // elements [first, end) of base; nothing past 2^31 bytes is addressed from one tile corner
  const int64_t bytes = first < end ? (end - first) * 2 : 0;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base + (first < end ? first : 0)), 0,
                                           static_cast<int>(bytes < 0x7fffffff ? bytes : 0x7fffffff), 0x00020000);
}

// ------------------------------------------------------------ the kernel

template <typename Dt, int BM, int BN, int WM, int WN, bool AAcross, bool BAcross, int Epi>
__global__ void __launch_bounds__(WM * WN * 64)
gemm_tile_kernel(GemmArgs g) {
  using E = typename Dt::E;
  constexpr bool kPair = Epi != kEpiStore;
  constexpr int kWaves = WM * WN;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // fragments per wave
  __shared__ __attribute__((aligned(16))) uint16_t a0[BM * kStepK];
  __shared__ __attribute__((aligned(16))) uint16_t a1[BM * kStepK];
  __shared__ __attribute__((aligned(16))) uint16_t b0[BN * kStepK];
  __shared__ __attribute__((aligned(16))) uint16_t b1[BN * kStepK];
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wm = wave / WN, wn = wave % WN;

  // Workgroups go round the eight dies, each with its own L2: give each die
  // a run of neighbouring tiles, in bands of eight tile rows.
  const int64_t tiles = g.tiles_m * g.tiles_n;
  int64_t t;
  {
    const int64_t id = blockIdx.x, die = id % 8, q = tiles / 8, r = tiles % 8;
    t = die * q + (die < r ? die : r) + id / 8;
  }
  const int64_t band = t / (8 * g.tiles_n), in_band = t % (8 * g.tiles_n);
  const int64_t band_rows = g.tiles_m - band * 8 < 8 ? g.tiles_m - band * 8 : 8;
  const int64_t m0 = (band * 8 + in_band % band_rows) * BM;
  const int64_t n0 = in_band / band_rows * (kPair ? BN / 2 : BN);
  const int z = blockIdx.z;

  TileLoad<BM, kWaves, AAcross> la;
  TileLoad<BN, kWaves, BAcross> lb;
  la.init(g.lda, wave, lane);
  lb.init(g.ldb, wave, lane);
  if constexpr (kPair) {  // the upper half of the tile's rows is the second matrix's, from its own corner
#pragma unroll
    for (int j = lb.kInstr / 2; j < lb.kInstr; ++j) lb.off[j] = lb.off[j - lb.kInstr / 2];
  }
  const int64_t steps = (g.k + kStepK - 1) / kStepK;
  // rows are held (along k: with zeros) up to a multiple of eight elements, and
  // the range check drops a whole chunk that crosses the end
  const int64_t k8 = (g.k + 7) / 8 * 8, m8 = (g.m + 7) / 8 * 8, n8 = (g.n + 7) / 8 * 8;
  const int64_t a_end = AAcross ? (g.k - 1) * g.lda + m8 : (g.m - 1) * g.lda + k8;
  const int64_t b_end = BAcross ? (g.k - 1) * g.ldb + n8 : (g.n - 1) * g.ldb + k8;

  int phase = 0;
  int64_t ks = 0;  // step within the phase, of the next load
  auto issue = [&](uint16_t* la_lds, uint16_t* lb_lds) {
    const int p = z * g.phases + phase;
    const int64_t k0 = ks * kStepK;
    const int64_t left = g.k - k0;  // the last step ends inside a row stored along k
    const int64_t fa = AAcross ? k0 * g.lda + m0 : m0 * g.lda + k0;
    const int64_t fb = BAcross ? k0 * g.ldb + n0 : n0 * g.ldb + k0;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(g.a[p], fa, a_end);
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(g.b[p], fb, b_end);
    if (left >= kStepK || (AAcross && BAcross)) {
      la.issue(la_lds, wave, [&](int) { return ra; });
      if constexpr (kPair) {
        const __amdgpu_buffer_rsrc_t rb2 = make_rsrc(g.b2[p], fb, b_end);
        lb.issue(lb_lds, wave, [&](int j) { return j < lb.kInstr / 2 ? rb : rb2; });
      } else {
        lb.issue(lb_lds, wave, [&](int) { return rb; });
      }
    } else {
      // chunks at or past k read out of range, that is zero
      TileLoad<BM, kWaves, AAcross> ta = la;
      TileLoad<BN, kWaves, BAcross> tb = lb;
      const int chunk = (lane % 8) ^ (lane / 8);
      const bool past = chunk * 8 >= left;
      if constexpr (!AAcross)
#pragma unroll
        for (int j = 0; j < ta.kInstr; ++j) ta.off[j] = past ? 0x80000000u : ta.off[j];
      if constexpr (!BAcross)
#pragma unroll
        for (int j = 0; j < tb.kInstr; ++j) tb.off[j] = past ? 0x80000000u : tb.off[j];
      ta.issue(la_lds, wave, [&](int) { return ra; });
      if constexpr (kPair) {
        const __amdgpu_buffer_rsrc_t rb2 = make_rsrc(g.b2[p], fb, b_end);
        tb.issue(lb_lds, wave, [&](int j) { return j < tb.kInstr / 2 ? rb : rb2; });
      } else {
        tb.issue(lb_lds, wave, [&](int) { return rb; });
      }
    }
    if (++ks == steps) ks = 0, ++phase;
  };

  v4f acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  // paired: the wave's first FN/2 fragments are of B, the others of B2
  auto b_row = [&](int j) {
    if constexpr (kPair)
      return (j < FN / 2 ? 0 : BN / 2) + wn * (BN / 2 / WN) + (j % (FN / 2)) * 16;
    else
      return wn * (BN / WN) + j * 16;
  };
  auto compute = [&](const uint16_t* pa, const uint16_t* pb) {
#pragma unroll
    for (int kk = 0; kk < kStepK / 32; ++kk) {
      u16x8 fa[FM], fb[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[j] = read_fragment<BN, BAcross>(pb, b_row(j), kk, lane);
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[i] = read_fragment<BM, AAcross>(pa, wm * (BM / WM) + i * 16, kk, lane);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mma16(E{}, fb[j], fa[i], acc[i][j]);
    }
  };
  auto landed = [] {
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    __syncthreads();
  };

  const int64_t total = steps * g.phases;
  if (total > 0) issue(a0, b0);  // none: a gradient over no rows is zero
  for (int64_t s = 0; s < total; s += 2) {
    landed();  // this step's tiles; the other buffers have been read
    if (s + 1 < total) issue(a1, b1);
    compute(a0, b0);
    if (s + 1 >= total) break;
    landed();
    if (s + 2 < total) issue(a0, b0);
    compute(a1, b1);
  }

  // ---------------------------------------------------------- epilogue
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = m0 + wm * (BM / WM) + i * 16 + lane % 16;
    if (m >= g.m) continue;
    if constexpr (Epi == kEpiStore) {
      using T = typename Dt::T;
      T* row = static_cast<T*>(g.c[z]) + m * g.ldc;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int64_t n = n0 + wn * (BN / WN) + j * 16 + lane / 16 * 4;
        T v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = static_cast<T>(acc[i][j][q]);
        if (n + 4 <= g.n) {
          __builtin_memcpy(row + n, v, sizeof(v));
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (n + q < g.n) row[n + q] = v[q];
        }
      }
    } else {
      const int64_t width = (g.n + 7) / 8 * 8;  // rows of the products' operands are read in 16-byte chunks
#pragma unroll
      for (int j = 0; j < FN / 2; ++j) {
        const int64_t n = n0 + wn * (BN / 2 / WN) + j * 16 + lane / 16 * 4;
        if (n >= width) continue;
        const int64_t at = m * g.ldh + n;
        float h[4], dg[4], du[4];
        if constexpr (Epi == kEpiGated) {
#pragma unroll
          for (int q = 0; q < 4; ++q) h[q] = act_value(acc[i][j][q], g.act) * acc[i][j + FN / 2][q];
        } else {
          typename Dt::DH d[4];
          __builtin_memcpy(d, static_cast<const typename Dt::DH*>(g.dh) + at, sizeof(d));
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float u = acc[i][j + FN / 2][q], dh = n + q < g.n ? static_cast<float>(d[q]) : 0.f;
            float a, da;
            act_both(acc[i][j][q], g.act, a, da);
            h[q] = a * u;
            dg[q] = dh * u * da;
            du[q] = dh * a;
          }
        }
        auto put = [&](uint16_t* to, const float(&v)[4]) {
          if constexpr (Dt::kPlanes == 1) {
            E e[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) e[q] = static_cast<E>(v[q]);
            __builtin_memcpy(to + at, e, 8);
          } else {
            bf16 p[4][3];
#pragma unroll
            for (int q = 0; q < 4; ++q) split3(v[q], p[q]);
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              bf16 e[4] = {p[0][k], p[1][k], p[2][k], p[3][k]};
              __builtin_memcpy(to + k * g.plane_stride + at, e, 8);
            }
          }
        };
        put(g.h, h);
        if constexpr (Epi == kEpiGatedBwd) {
          put(g.dg, dg);
          put(g.du, du);
        }
      }
    }
  }
}

}  // namespace kern
}  // namespace segpoly
