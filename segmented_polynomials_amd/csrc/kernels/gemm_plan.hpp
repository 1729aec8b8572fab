// Matrix products in tiles (gemm_tile.hpp) from the host's side: operands in the
// form that the tile loads take, the choice of tiles, long sums shared out over
// workgroups, and the workspace.
#pragma once
#include <algorithm>
#include <cmath>

#include "../launch.hpp"
#include "gemm_staged.hpp"
#include "gemm_tile.hpp"

namespace segpoly {
namespace kern {

// A matrix in the form the tile loads take: planes, row stride a multiple
// of 8, 16-byte aligned, rows zero up to a multiple of 8 columns.
struct Operand {
  const uint16_t* plane[3];
  int64_t ld;
  int* exponents = nullptr;  // of scaled blocks of 64 rows and 32 columns
  int64_t exponents_ld = 0;
};

constexpr int kMaxPack = 5;
struct PackArgs {
  const void* src[kMaxPack];
  uint16_t* dst[kMaxPack];
  int64_t rows[kMaxPack], width[kMaxPack], src_ld[kMaxPack], dst_ld[kMaxPack], plane_stride[kMaxPack];
};

// 8 columns a lane: copied (16-bit) or split into three planes (float32),
// zeros past the width
template <typename Dt>
__global__ void __launch_bounds__(256)
pack_kernel(PackArgs g) {
  using T = typename Dt::T;
  using E = typename Dt::E;
  const int o = blockIdx.y;
  const int64_t chunks = g.dst_ld[o] / 8, total = g.rows[o] * chunks;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = i / chunks, c = i % chunks * 8;
    const T* src = static_cast<const T*>(g.src[o]) + r * g.src_ld[o] + c;
    T v[8];
    if (c + 8 <= g.width[o]) {
      __builtin_memcpy(v, src, sizeof(v));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = c + j < g.width[o] ? src[j] : T(0.f);
    }
    uint16_t* dst = g.dst[o] + r * g.dst_ld[o] + c;
    if constexpr (Dt::kPlanes == 1) {
      __builtin_memcpy(dst, v, 16);
    } else {
      E p[8][3];
#pragma unroll
      for (int j = 0; j < 8; ++j) split3(static_cast<float>(v[j]), p[j]);
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        E e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = p[j][k];
        __builtin_memcpy(dst + k * g.plane_stride[o], e, 16);
      }
    }
  }
}

template <typename Dt>
void add_phase(GemmArgs& g, int& at, const Operand& a, const Operand& b, const Operand* b2 = nullptr) {
  for (int p = 0; p < Dt::kPlanes; ++p) {
    const int i = at * Dt::kPlanes + p;
    g.a[i] = a.plane[p];
    g.b[i] = b.plane[p];
    if (b2) g.b2[i] = b2->plane[p];
  }
  g.ea[at] = a.exponents;
  g.eb[at] = b.exponents;
  g.e_ld = std::max(a.exponents_ld, b.exponents_ld);
  ++at;
}

// rows of both staged operands in multiples of 16 bytes
template <bool AAcross, bool BAcross>
bool staged_whole(const GemmArgs& g) {
  return (AAcross ? g.m[0] : g.k) % 4 == 0 && (BAcross ? g.n[0] : g.k) % 4 == 0;
}

template <typename Dt, int BM, int BN, int WM, int WN, int KS, int S, bool AAcross, bool BAcross, int Epi>
int gemm_launch_tile(GemmArgs& g, hipStream_t st) {
  const int64_t bn = Epi == kEpiGated || Epi == kEpiGatedBwd ? BN / 2 : BN;
  int64_t tiles = 0;
  for (int z = 0; z < g.batch; ++z) {
    g.tiles_m[z] = (g.m[z] + BM - 1) / BM;
    g.tiles_n[z] = (g.n[z] + bn - 1) / bn;
    tiles += g.tiles_m[z] * g.tiles_n[z];
  }
  if (tiles == 0) return 0;  // no rows
  if (g.splits < 1) g.splits = 1;
  g.column_rows = g.tiles_m[0] * WM;
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(g.splits));
  if constexpr (kStaged<Dt>) {
    auto* kernel = staged_whole<AAcross, BAcross>(g) ? gemm_staged_kernel<BM, BN, WM, WN, AAcross, BAcross, Epi, true>
                                                     : gemm_staged_kernel<BM, BN, WM, WN, AAcross, BAcross, Epi, false>;
    hipLaunchKernelGGL(kernel, grid, dim3(WM * WN * 64), 0, st, g);
  } else {
    hipLaunchKernelGGL((gemm_tile_kernel<Dt, BM, BN, WM, WN, KS, S, AAcross, BAcross, Epi>), grid, dim3(WM * WN * 64), 0, st,
                       g);
  }
  return static_cast<int>(hipGetLastError());
}

// Shares of the sum over k of a product with few tiles.  A card holds 768
// workgroups of the 64 x 64 tile; a product that fills less than half of them
// and has a long sum gives each tile several, of at least sixteen steps, whose
// float32 sums a second kernel adds.  One MI355X, 63 rows of 1352 x 5603 x 272
// float32, backward: 158 us, 385 us without.  With at least 8, 16 and 32 steps a
// share, us of backward passes in bf16 | f32: 1357 x 322 x 853 x 257 46, 43, 42 | 95, 96,
// 96; 500 x 256 x 512 x 256 20, 19, 19 | 43, 46, 53; 64 x 1024 x 4096 x 1024 46, 45, 49 |
// 105, 111, 129; 300 x 128 x 8000 x 128 43, 40, 42 | 87, 80, 81.
struct Split {
  int splits = 1;
  int64_t elements = 0;  // of one share
};
template <typename Dt>
Split plan_split(const GemmArgs& g) {
  constexpr int64_t kStep = Dt::kPlanes == 1 ? 64 : 32;
  Split p;
  int64_t tiles = 0;
  for (int z = 0; z < g.batch; ++z) {
    tiles += round_up(g.m[z], 64) / 64 * (round_up(g.n[z], 64) / 64);
    p.elements += g.m[z] * round_up(g.n[z], 4);
  }
  const int64_t steps = (g.k + kStep - 1) / kStep * g.phases;
  if (tiles > 0 && tiles < 384)
    p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(768 / tiles, steps / 16)));
  // A step of staged operands takes a microsecond where a unit has one workgroup: shares of five steps until most
  // units have one.  One MI355X, us with five and sixteen at least, float32: 40 x 700 x 700 forward 12, 25, gradient
  // 27, 53; 700 x 1500 x 96 13, 29 and 31, 61; 1357 x 322 x 853 gradient 68, 75.
  if (kStaged<Dt> && tiles > 0 && tiles * p.splits < 192)
    p.splits = static_cast<int>(std::max<int64_t>(p.splits, std::min<int64_t>((256 + tiles - 1) / tiles, steps / 5)));
  return p;
}

// The same in tiles of 128 x 128, each element read and split or moved by half as
// many tiles, where their shares fill the card: a compute unit holds one workgroup of
// staged operands, two of others.  One MI355X, us of the gradients with these and in tiles of 64 x 64:
// 20000 x 512 x 512 float32 257, 288; 60000 x 256 x 1000 796, 898, bf16 262, 293; 8192 x 1024 x
// 1024 float32 325, 376; of a product that half fills the card: 2000 x 2000 x 2000 bf16 73, 66.
template <typename Dt>
Split plan_split_wide(const GemmArgs& g) {
  constexpr int64_t kStep = Dt::kPlanes == 1 ? 64 : 32, kHeld = Dt::kPlanes == 1 ? 512 : 256;
  Split p;
  if (g.batch != 1 || g.phases != 1 || g.m[0] <= 64 || g.n[0] <= 64) return p;
  const int64_t tiles = (g.m[0] + 127) / 128 * ((g.n[0] + 127) / 128), steps = (g.k + kStep - 1) / kStep;
  const int64_t splits = std::min(kHeld / tiles, steps / 16);
  if (splits < 2 || tiles * 4 > kHeld || tiles * splits * 4 < kHeld * 3) return p;
  p.splits = static_cast<int>(splits);
  p.elements = g.m[0] * round_up(g.n[0], 4);
  return p;
}

// Directs the product's shares into `sums` and notes what adds them up; the
// elements of `sums` that it takes.
inline int64_t split_into(GemmArgs& g, const Split& p, float* sums, SplitSumArgs& q) {
  int64_t at = 0;
  for (int z = 0; z < g.batch; ++z) {
    const int k = q.batch++;
    q.m[k] = g.m[z], q.n[k] = g.n[z], q.ld[k] = round_up(g.n[z], 4), q.ldc[k] = g.ldc[z], q.to[k] = g.c[z];
    q.from[k] = sums + at, q.split_stride[k] = p.elements, q.splits[k] = p.splits;
    g.c[z] = sums + at, g.ldc[z] = q.ld[k];
    at += q.m[k] * q.ld[k];
  }
  g.split_stride = p.elements;
  g.splits = p.splits;
  return p.splits * p.elements;
}

template <typename T>
int split_sum_launch(const SplitSumArgs& q, hipStream_t st) {
  int64_t most = 0;
  for (int k = 0; k < q.batch; ++k) most = std::max(most, q.m[k] * q.ld[k] / 4);
  if (most == 0) return 0;
  hipLaunchKernelGGL(split_sum_kernel<T>, dim3(static_cast<unsigned>(std::min<int64_t>((most + 255) / 256, 2048)), q.batch),
                     dim3(256), 0, st, q);
  return static_cast<int>(hipGetLastError());
}

template <typename Dt, bool AAcross, bool BAcross, int Epi>
int gemm_launch(GemmArgs& g, hipStream_t st);

// A step of 64 x 64 tiles, and the buffers: three workgroups share a compute unit.
template <typename Dt>
constexpr int kSmallK = Dt::kPlanes == 1 ? 64 : 32;
template <typename Dt>
constexpr int kSmallS = Dt::kPlanes == 1 ? 3 : 2;

// A product with a plain epilogue, split if that pays; `sums` is the space that
// SplitSpace found for it.  q: sums of others to be added up with its shares.
template <typename Dt, bool AAcross, bool BAcross, int Epi, bool Wide = false>
int gemm_launch_split(GemmArgs& g, float* sums, hipStream_t st, SplitSumArgs q = {}) {
  using T = std::conditional_t<Epi == kEpiStoreF32, float, typename Dt::T>;
  int rc;
  const Split wide = Wide ? plan_split_wide<Dt>(g) : Split{};
  if (wide.splits > 1) {
    if constexpr (Wide) {
      split_into(g, wide, sums, q);
      if constexpr (Dt::kPlanes == 1)
        rc = gemm_launch_tile<Dt, 128, 128, 2, 2, 64, 2, AAcross, BAcross, kEpiStoreF32>(g, st);
      else
        rc = gemm_launch_tile<Dt, 128, 128, 2, 4, 32, 2, AAcross, BAcross, kEpiStoreF32>(g, st);
    }
  } else {
    const Split p = plan_split<Dt>(g);
    if (p.splits == 1) {
      rc = gemm_launch<Dt, AAcross, BAcross, Epi>(g, st);
    } else {
      split_into(g, p, sums, q);
      rc = gemm_launch_tile<Dt, 64, 64, 2, 2, kSmallK<Dt>, kSmallS<Dt>, AAcross, BAcross, kEpiStoreF32>(g, st);
    }
  }
  return rc ? rc : split_sum_launch<T>(q, st);
}

template <typename Dt, int EpiX, int EpiW>
int gemm_launch_two(GemmArgs& x, GemmArgs& w, hipStream_t st) {
  int64_t tiles[2] = {0, 0};
  GemmArgs* g[2] = {&x, &w};
  for (int k = 0; k < 2; ++k) {
    if (g[k]->splits < 1) g[k]->splits = 1;
    for (int z = 0; z < g[k]->batch; ++z) {
      g[k]->tiles_m[z] = (g[k]->m[z] + 63) / 64;
      g[k]->tiles_n[z] = (g[k]->n[z] + 63) / 64;
      tiles[k] += g[k]->tiles_m[z] * g[k]->tiles_n[z];
    }
  }
  const int64_t blocks = tiles[0] * x.splits + tiles[1] * w.splits;
  if (blocks == 0) return 0;
  const dim3 grid(static_cast<unsigned>(blocks));
  if constexpr (kStaged<Dt>) {
    auto* kernel = staged_whole<false, true>(x) && staged_whole<true, true>(w) ? gemm_staged_two_kernel<EpiX, EpiW, true>
                                                                               : gemm_staged_two_kernel<EpiX, EpiW, false>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, x, w, tiles[0], tiles[1]);
  } else {
    hipLaunchKernelGGL((gemm_two_kernel<Dt, kSmallK<Dt>, kSmallS<Dt>, EpiX, EpiW>), grid, dim3(256), 0, st, x, w, tiles[0],
                       tiles[1]);
  }
  return static_cast<int>(hipGetLastError());
}

// The two together, each split if that pays.
template <typename Dt>
int gemm_launch_two_split(GemmArgs& x, GemmArgs& w, float* sums, hipStream_t st, SplitSumArgs q = {}) {
  const Split px = plan_split<Dt>(x), pw = plan_split<Dt>(w);
  int64_t at = 0;
  if (px.splits > 1) at += split_into(x, px, sums, q);
  if (pw.splits > 1) split_into(w, pw, sums + at, q);
  int rc;
  if (px.splits > 1)
    rc = pw.splits > 1 ? gemm_launch_two<Dt, kEpiStoreF32, kEpiStoreF32>(x, w, st)
                       : gemm_launch_two<Dt, kEpiStoreF32, kEpiStore>(x, w, st);
  else
    rc = pw.splits > 1 ? gemm_launch_two<Dt, kEpiStore, kEpiStoreF32>(x, w, st)
                       : gemm_launch_two<Dt, kEpiStore, kEpiStore>(x, w, st);
  return rc ? rc : split_sum_launch<typename Dt::T>(q, st);
}

// The tile with the least estimated time.  `each` workgroups of a tile share a
// compute unit; a round of 256 x each tiles takes their area over the share of
// the matrix rate that the tile reaches.  A last round that is not full counts
// half way between a whole one and its share (whole with one workgroup a unit).
// One MI355X, 8192 rows, widths 2048 and 5632, bf16, TFLOP/s: the paired
// product 1090 with 256 x 256 tiles, 1020 with 128 x 128; its backward form,
// whose epilogue moves 460 MB, 885 with 256 x 128 in three buffers, 722 with
// 256 x 256, 831 with 128 x 128; one operand across k 1060 and 1395 with
// 256 x 256, 970 and 1085 with 128 x 128; both across 1150 and 952 with
// 256 x 128 in steps of 32, two workgroups a unit, 1086 and 997 with 256 x 256.
template <typename Dt, bool AAcross, bool BAcross, int Epi>
int gemm_launch(GemmArgs& g, hipStream_t st) {
  const int64_t pair = Epi == kEpiGated || Epi == kEpiGatedBwd ? 2 : 1;
  auto cost = [&](int64_t bm, int64_t bn, int each, double rate) {
    int64_t t = 0;
    for (int z = 0; z < g.batch; ++z) t += (g.m[z] + bm - 1) / bm * ((g.n[z] * pair + bn - 1) / bn);
    const double rounds = static_cast<double>(t) / (256 * each), whole = std::ceil(rounds);
    return (each > 1 && rounds > 1 ? 0.5 * (rounds + whole) : whole) * static_cast<double>(bm * bn * each) / rate;
  };
  if constexpr (Dt::kPlanes == 1) {
    constexpr bool kTwoAcross = AAcross && BAcross, kBwd = Epi == kEpiGatedBwd;
    // the dense epilogues' activations and slopes take a tile as long as a few hundred k: beside a second workgroup's
    // products (8192 x 2048 x 5632 bf16, gradient with gelu: 5 % less than with 256 x 128 tiles on the same card;
    // 20000 x 512 x 512 forward 28 us, 34)
    constexpr bool kDense = Epi == kEpiDense || Epi == kEpiDenseBwd;
    const double large = kTwoAcross || kBwd ? cost(256, 128, kBwd ? 1 : 2, 1.0) : cost(256, 256, 1, 1.0);
    const double c128 = cost(128, 128, 2, 0.8), c64 = cost(64, 64, 3, 0.45);
    if constexpr (!kDense) {
      if (large <= c128 && large <= c64) {
        if constexpr (kTwoAcross)
          return gemm_launch_tile<Dt, 256, 128, 2, 2, 32, 3, AAcross, BAcross, Epi>(g, st);
        else if constexpr (kBwd)
          return gemm_launch_tile<Dt, 256, 128, 4, 2, 64, 3, AAcross, BAcross, Epi>(g, st);
        else
          return gemm_launch_tile<Dt, 256, 256, 2, 4, 64, 2, AAcross, BAcross, Epi>(g, st);
      }
    }
    if (c128 <= c64) return gemm_launch_tile<Dt, 128, 128, 2, 2, 64, 2, AAcross, BAcross, Epi>(g, st);
    return gemm_launch_tile<Dt, 64, 64, 2, 2, kSmallK<Dt>, kSmallS<Dt>, AAcross, BAcross, Epi>(g, st);
  } else {
    // 20000 rows of 128 x 512: paired 52 us with 128 x 128 tiles, 48 us with 64 x 64, three workgroups a unit
    if (cost(128, 128, 1, 0.9) <= cost(64, 64, 3, 0.9))
      return gemm_launch_tile<Dt, 128, 128, 2, 4, 32, 2, AAcross, BAcross, Epi>(g, st);
    return gemm_launch_tile<Dt, 64, 64, 2, 2, kSmallK<Dt>, kSmallS<Dt>, AAcross, BAcross, Epi>(g, st);
  }
}

// Hands out the workspace; with a null base only counts.
struct Arena {
  char* base;
  size_t at = 0;
  template <typename T>
  T* take(int64_t count) {
    const size_t o = at;
    at += (static_cast<size_t>(count) * sizeof(T) + 255) / 256 * 256;
    return base ? reinterpret_cast<T*>(base + o) : nullptr;
  }
};

template <typename Dt>
struct MatrixPlan {
  using T = typename Dt::T;
  static constexpr int P = Dt::kPlanes;
  Arena arena;
  PackArgs pack{};
  int packs = 0;
  int64_t pack_chunks = 0;

  explicit MatrixPlan(void* ws) : arena{static_cast<char*>(ws)} {}

  // worst: as if the matrix had to be packed (the size query).  summed: over its
  // rows, in some product, whose loads of the last step would read rows past the
  // last where rows overlap (each starts within the one before).
  Operand use(const void* src, int64_t rows, int64_t width, int64_t ld, bool worst, bool summed = false) {
    Operand o{};
    if (kStaged<Dt> || (!worst && P == 1 && !(summed && ld < width) && width % 8 == 0 && ld % 8 == 0 && reinterpret_cast<uintptr_t>(src) % 16 == 0)) {
      o.plane[0] = static_cast<const uint16_t*>(src);
      o.ld = ld;
      return o;
    }
    o.ld = round_up(width, 8);
    uint16_t* dst = arena.take<uint16_t>(P * rows * o.ld);
    if (dst)
      for (int k = 0; k < P; ++k) o.plane[k] = dst + k * rows * o.ld;
    pack.src[packs] = src, pack.dst[packs] = dst, pack.rows[packs] = rows, pack.width[packs] = width;
    pack.src_ld[packs] = ld, pack.dst_ld[packs] = o.ld, pack.plane_stride[packs] = rows * o.ld;
    pack_chunks = std::max(pack_chunks, rows * (o.ld / 8));
    ++packs;
    return o;
  }
  Operand hidden(int64_t n, int64_t hidden) {
    Operand o{};
    if constexpr (kStaged<Dt>) {  // float32 rows
      o.ld = round_up(hidden, 4);
      o.plane[0] = reinterpret_cast<const uint16_t*>(arena.take<float>(n * o.ld));
      return o;
    }
    o.ld = round_up(hidden, 64);
    uint16_t* p = arena.take<uint16_t>(P * n * o.ld);
    if (p)
      for (int k = 0; k < P; ++k) o.plane[k] = p + k * n * o.ld;
    if constexpr (Dt::kScaled) {
      o.exponents_ld = (hidden + 31) / 32;
      o.exponents = arena.take<int>((n + 63) / 64 * o.exponents_ld);
    }
    return o;
  }
  int run_pack(hipStream_t st) {
    if (!packs) return 0;
    const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((pack_chunks + 255) / 256, 2048));
    hipLaunchKernelGGL(pack_kernel<Dt>, dim3(static_cast<unsigned>(blocks), packs), dim3(256), 0, st, pack);
    return static_cast<int>(hipGetLastError());
  }
};

// the sums' space of the largest of a call's split products
template <typename Dt>
struct SplitSpace {
  int64_t most = 0;
  static int64_t of(const GemmArgs& g) { return of(plan_split<Dt>(g)); }
  static int64_t of(const Split& p) { return p.splits > 1 ? p.splits * p.elements : 0; }
  void add(int64_t elements) { most = std::max(most, elements); }
};

template <typename Dt>
GemmArgs product(int64_t m, int64_t n, int64_t k, const Operand& a, const Operand& b, void* c, int64_t ldc) {
  GemmArgs g{};
  add_phase<Dt>(g, g.phases, a, b);
  g.batch = 1, g.m[0] = m, g.n[0] = n, g.k = k, g.lda[0] = a.ld, g.ldb[0] = b.ld, g.c[0] = c, g.ldc[0] = ldc;
  return g;
}

}  // namespace kern
}  // namespace segpoly
