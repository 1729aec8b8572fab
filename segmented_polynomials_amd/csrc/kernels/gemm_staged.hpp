// Matrix-core tiles of float32 operands as they are in memory, of any stride and
// alignment: the products of gemm_tile.hpp (three bf16 planes, six products) with
// the planes made on the way to LDS instead of by a pass of its own.  That pass
// reads 4 bytes of an element and writes 6, which every tile then reads: more than
// the product itself where one side is a few hundred wide.
// A thread loads eight neighbours of a row two steps ahead, splits them a step
// ahead and writes their planes to the LDS buffer that the next step reads; one
// barrier a step, two buffers.  The splitting (some 7 vector instructions an
// element) runs beside the other waves' matrix instructions.
#pragma once
#include "gemm_rows.hpp"

namespace segpoly {
namespace kern {

// Eight float32 as planes; true where a value may round up to infinity: the planes
// are split3's then.  The planes behind an infinity's first or a NaN's are NaN here,
// zero there: they are of small products, which do not count beside a large one that
// is not finite (add_small).
__device__ __forceinline__ bool split_fast(const float (&v)[8], u16x8 (&p)[3]) {
  float r[8], top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r[i] = v[i];
    top = __builtin_fmaxf(top, __builtin_fabsf(v[i]));
  }
#pragma unroll
  for (int q = 0; q < 3; ++q)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bf16 s = static_cast<bf16>(r[i]);
      p[q][i] = __builtin_bit_cast(uint16_t, s);
      if (q < 2) r[i] -= static_cast<float>(s);
    }
  return top >= 0x1.ffp127f;
}
__device__ __forceinline__ void split_slow(const float (&v)[8], u16x8 (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    bf16 s[3];
    split3(v[i], s);
#pragma unroll
    for (int q = 0; q < 3; ++q) p[q][i] = __builtin_bit_cast(uint16_t, s[q]);
  }
}
__device__ __forceinline__ void split_eight(const float (&v)[8], u16x8 (&p)[3]) {
  if (__ballot(split_fast(v, p))) split_slow(v, p);
}

// Eight elements of a row from column `at` on, those from `limit` on zeros: the width,
// or 0 for a row that does not count, whose address is another's.  Whole: of rows whose
// width is a multiple of 16 bytes, no load crosses the end.  Else one that would is from
// further left, and a wave with any moves its elements after they have landed
// (settle_eight); no branches around the loads.  What that costs, float32 forward, us of whole, even and odd
// widths: 100000 x 128 x 128 33, of 126 and of 125 to 127 36 and 38; 20000 x 512 x 512 101, 117, 119; 2000 x 2000 x 2000
// 105, 157, 156, where it also takes the smooth loop (StagedOperand).
template <typename Dt, bool Whole>
__device__ __forceinline__ void load_eight(RowChunk<Dt>& c, const typename Dt::T* row, int at, int width, int limit) {
  constexpr int N = Chunk<typename Dt::T>::kN;
#pragma unroll
  for (int i = 0; i < RowChunk<Dt>::kLoads; ++i) {
    const int col = at + i * N;
    if constexpr (Whole) {
      c.raw[i] = u32x4{0, 0, 0, 0};
      if (col < limit) __builtin_memcpy(&c.raw[i], row + col, 16);
    } else if (width >= N) {
      __builtin_memcpy(&c.raw[i], row + (col + N <= width ? col : width - N), 16);
    } else {
      c.raw[i] = load_raw(row, limit ? col : width, width);
    }
  }
}
template <typename Dt>
__device__ __forceinline__ void settle_eight(RowChunk<Dt>& c, int at, int width, int limit) {
  using T = typename Dt::T;
  constexpr int N = Chunk<T>::kN;
  if (width < N || !__ballot(at + 8 > limit)) return;
#pragma unroll
  for (int i = 0; i < RowChunk<Dt>::kLoads; ++i) {
    const int col = at + i * N;
    c.raw[i] = settle_chunk<T>(c.raw[i], col, width);
    if (col >= limit) c.raw[i] = u32x4{0, 0, 0, 0};
  }
}
// the eight values
template <typename Dt, bool Whole>
__device__ __forceinline__ void eight_values(RowChunk<Dt> c, int at, int width, int limit, float (&v)[8]) {
  if constexpr (!Whole) settle_eight<Dt>(c, at, width, limit);
  typename Dt::T t[8];
  __builtin_memcpy(t, c.raw, sizeof(t));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(t[i]);
}
// and as matrix operands
template <typename Dt, bool Whole>
__device__ __forceinline__ void chunk_planes(RowChunk<Dt> c, int at, int width, int limit, u16x8 (&p)[Dt::kPlanes]) {
  if constexpr (Dt::kPlanes == 1) {
    if constexpr (!Whole) settle_eight<Dt>(c, at, width, limit);
    p[0] = __builtin_bit_cast(u16x8, c.raw[0]);
  } else {
    float v[8];
    eight_values<Dt, Whole>(c, at, width, limit, v);
    split_eight(v, p);
  }
}

constexpr int kStagedK = 32;  // k of a step

// The eight neighbours that this thread brings to each step's tile of an operand of
// R rows (along k: of one row; across: of one k).  Smooth: no branches, so that the
// step's work can go between the matrix instructions, at the price of some more
// of it: for the large tile, whose workgroup has a compute unit to itself.  One
// MI355X, us of forward passes with and without: 2000 x 2000 x 2000 103, 107; in
// the small tile 50000 x 256 x 256 76, 61.
template <int R, int Threads, bool Across, bool Whole>
struct StagedOperand {
  static constexpr bool kSmooth = Whole && Threads == 512;
  static_assert(R * kStagedK / 8 == Threads, "eight elements a thread");
  static constexpr int kRowChunks = (Across ? R : kStagedK) / 8;
  const float* base;
  int64_t ld;
  int row, chunk, width, k;  // along: width is k; across: the operand's rows from the tile's on
  __device__ __forceinline__ StagedOperand(const void* p, int64_t ld_, int64_t corner, int64_t rows, int64_t k_) : ld(ld_) {
    row = threadIdx.x / kRowChunks;
    chunk = threadIdx.x % kRowChunks;
    k = static_cast<int>(k_);
    if constexpr (Across) {
      base = static_cast<const float*>(p) + corner;
      width = static_cast<int>(rows - corner < R ? rows - corner : R);
    } else {  // rows past the last repeat it, and are not stored
      base = static_cast<const float*>(p) + (corner + row < rows ? corner + row : rows - 1) * ld;
      width = k;
    }
  }
  // Smooth: what lies past the ends is loaded from within; past the last k it counts
  // as zero, past the last row or column it is not stored.
  __device__ __forceinline__ int first(int64_t step) const {  // along: the k of the first
    return Across ? chunk * 8 : static_cast<int>(step) * kStagedK + chunk * 8;
  }
  __device__ __forceinline__ int columns(int64_t step) const {  // none past the last k
    return Across && step * kStagedK + row >= k ? 0 : width;
  }
  __device__ __forceinline__ void load(RowChunk<DtF32>& c, int64_t step) const {
    if constexpr (kSmooth) {
      const int kk = static_cast<int>(step) * kStagedK + row;
      const float* at = Across ? base + (kk < k ? kk : k - 1) * ld : base;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = first(step) + i * 4;
        __builtin_memcpy(&c.raw[i], at + (col < width ? col : width - 4), 16);
      }
    } else {
      load_eight<DtF32, Whole>(c, Across ? base + (step * kStagedK + (columns(step) ? row : 0)) * ld : base, first(step),
                               width, columns(step));
    }
  }
  __device__ __forceinline__ void values(const RowChunk<DtF32>& c, int64_t step, float (&v)[8]) const {
    if constexpr (kSmooth) {
      const int kk = static_cast<int>(step) * kStagedK + row;
      __builtin_memcpy(v, c.raw, sizeof(v));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (Across ? kk < k : first(step) + i / 4 * 4 < k) ? v[i] : 0.f;
    } else {
      eight_values<DtF32, Whole>(c, first(step), width, columns(step), v);
    }
  }
  __device__ __forceinline__ void place(const u16x8 (&p)[3], uint16_t* lds) const {
    const int slot = row * (kRowChunks * 8) + (chunk ^ TileLoad<R, kStagedK, 1, Across>::fold(row)) * 8;
#pragma unroll
    for (int q = 0; q < 3; ++q) *reinterpret_cast<u16x8*>(lds + q * R * kStagedK + slot) = p[q];
  }
  // true where the planes are not yet right
  __device__ __forceinline__ bool write(const RowChunk<DtF32>& c, int64_t step, uint16_t* lds) const {
    float v[8];
    u16x8 p[3];
    values(c, step, v);
    bool again = split_fast(v, p);
    if constexpr (!kSmooth) {
      if (__ballot(again)) split_slow(v, p);
      again = false;
    }
    place(p, lds);
    return again;
  }
  __device__ __forceinline__ void write_again(const RowChunk<DtF32>& c, int64_t step, uint16_t* lds) const {
    float v[8];
    u16x8 p[3];
    values(c, step, v);
    split_slow(v, p);
    place(p, lds);
  }
};

// Tile `id`, share `share` of its steps; one phase and one batch.
template <int BM, int BN, int WM, int WN, bool AAcross, bool BAcross, int Epi, bool Whole>
__device__ __forceinline__ void gemm_staged(const GemmArgs& g, int64_t id, int share, uint16_t* a0, uint16_t* b0,
                                            uint16_t* a1, uint16_t* b1) {
  constexpr int kThreads = WM * WN * 64, KS = kStagedK;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wm = wave / WN, wn = wave % WN;
  const int64_t gm = g.m[0], gn = g.n[0], tiles_m = g.tiles_m[0], tiles_n = g.tiles_n[0];
  int64_t m0, n0;
  tile_corner<BM, BN>(id, tiles_m, tiles_n, m0, n0);
  const StagedOperand<BM, kThreads, AAcross, Whole> la(g.a[0], g.lda[0], m0, gm, g.k);
  const StagedOperand<BN, kThreads, BAcross, Whole> lb(g.b[0], g.ldb[0], n0, gn, g.k);
  const int64_t steps = (g.k + KS - 1) / KS;
  const int64_t s0 = steps * share / g.splits, s1 = steps * (share + 1) / g.splits;

  v4f acc[FM][FN], small[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = small[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const uint16_t* at_a, const uint16_t* at_b) __attribute__((always_inline)) {
    u16x8 fa[3][FM], fb[3][FN];
#pragma unroll
    for (int q = 0; q < 3; ++q) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
        fb[q][j] = read_fragment<BN, KS, BAcross>(at_b + q * BN * KS, wn * (BN / WN) + j * 16, 0, lane);
#pragma unroll
      for (int i = 0; i < FM; ++i)
        fa[q][i] = read_fragment<BM, KS, AAcross>(at_a + q * BM * KS, wm * (BM / WM) + i * 16, 0, lane);
    }
#pragma unroll
    for (int t = 0; t < 6; ++t)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          v4f& c = t < 5 ? small[i][j] : acc[i][j];
          c = mma16(bf16{}, fb[kPairs3[t][1]][j], fa[kPairs3[t][0]][i], c);
        }
  };
  RowChunk<DtF32> ra[2], rb[2];
  // past the last step: the last again, which is not used
  auto within = [&](int64_t s) { return s < s1 ? s : s1 - 1; };
  constexpr bool kSmooth = decltype(la)::kSmooth;
  auto fetch = [&](int r, int64_t s) __attribute__((always_inline)) {
    if (!kSmooth && s >= s1) return;
    la.load(ra[r], within(s));
    lb.load(rb[r], within(s));
  };
  // the planes of values that split_fast does not split, behind the matrix
  // instructions; a wave's writes to LDS are in order
  auto repair = [&](bool again_a, bool again_b, const RowChunk<DtF32>& a, const RowChunk<DtF32>& b, int64_t s,
                    uint16_t* to_a, uint16_t* to_b) __attribute__((always_inline)) {
    if constexpr (kSmooth) {
      if (__ballot(again_a)) la.write_again(a, s, to_a);
      if (__ballot(again_b)) lb.write_again(b, s, to_b);
    }
  };
  // step s computes from its buffer while the next step's planes go to the other,
  // which was last read a barrier ago
  auto step = [&](int next, int64_t s, const uint16_t* now_a, const uint16_t* now_b, uint16_t* next_a, uint16_t* next_b)
                  __attribute__((always_inline)) {
    const RowChunk<DtF32> a = ra[next], b = rb[next];
    bool again_a = false, again_b = false;
    if (kSmooth || s + 1 < s1) {
      again_a = la.write(a, within(s + 1), next_a);
      again_b = lb.write(b, within(s + 1), next_b);
    }
    fetch(next, s + 3);
    compute(now_a, now_b);
    repair(again_a, again_b, a, b, within(s + 1), next_a, next_b);
    wait_and_meet<63>();
  };
  if (s0 < s1) {
    fetch(0, s0);
    fetch(1, s0 + 1);
    const bool again_a = la.write(ra[0], s0, a0), again_b = lb.write(rb[0], s0, b0);
    repair(again_a, again_b, ra[0], rb[0], s0, a0, b0);
    fetch(0, s0 + 2);
    wait_and_meet<63>();
    for (int64_t s = s0; s < s1; s += 2) {
      step(1, s, a0, b0, a1, b1);
      if (s + 1 < s1) step(0, s + 1, a1, b1, a0, b0);
    }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = add_small(acc[i][j], small[i][j]);
  finish_tile<DtF32Staged, BM, BN, WM, WN, KS, Epi>(g, 0, m0, n0, share, acc, a0, b0);
}

#define SEGPOLY_STAGED_LDS(BM, BN)                                        \
  __shared__ __attribute__((aligned(16))) uint16_t a0[3 * BM * kStagedK]; \
  __shared__ __attribute__((aligned(16))) uint16_t b0[3 * BN * kStagedK]; \
  __shared__ __attribute__((aligned(16))) uint16_t a1[3 * BM * kStagedK]; \
  __shared__ __attribute__((aligned(16))) uint16_t b1[3 * BN * kStagedK]

template <int BM, int BN, int WM, int WN, bool AAcross, bool BAcross, int Epi, bool Whole>
__global__ void __launch_bounds__(WM * WN * 64, 2)
gemm_staged_kernel(GemmArgs g) {
  SEGPOLY_STAGED_LDS(BM, BN);
  gemm_staged<BM, BN, WM, WN, AAcross, BAcross, Epi, Whole>(g, blockIdx.x, blockIdx.y, a0, b0, a1, b1);
}

// Two independent products in one launch, as gemm_two_kernel.
template <int EpiX, int EpiW, bool Whole>
__global__ void __launch_bounds__(256, 2)
gemm_staged_two_kernel(GemmArgs x, GemmArgs w, int64_t x_tiles, int64_t w_tiles) {
  SEGPOLY_STAGED_LDS(64, 64);
  const int64_t x_blocks = x_tiles * x.splits;
  if (blockIdx.x < x_blocks) {
    gemm_staged<64, 64, 2, 2, false, true, EpiX, Whole>(x, blockIdx.x % x_tiles, static_cast<int>(blockIdx.x / x_tiles), a0,
                                                        b0, a1, b1);
  } else {
    const int64_t id = blockIdx.x - x_blocks;
    gemm_staged<64, 64, 2, 2, true, true, EpiW, Whole>(w, id % w_tiles, static_cast<int>(id / w_tiles), a0, b0, a1, b1);
  }
}

}  // namespace kern
}  // namespace segpoly
