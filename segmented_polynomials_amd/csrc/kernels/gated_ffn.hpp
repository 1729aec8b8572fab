// The gated feed-forward block and its backward as tile products
// (gemm_tile.hpp), for one element type per translation unit:
//   forward   h = act(x Wg^T) * (x Wu^T)     one paired product, the
//                                            activation and gating its epilogue
//             out = h Wd^T                   (few rows: gemm_rows.hpp)
//   backward  dh = g Wd
//             h, dg, du from x, Wg, Wu, dh   the paired product again
//             dx = dg Wg + du Wu             one product of two phases
//             dWg = dg^T x, dWu = du^T x, dWd = g^T h     one launch of the three
// Between the products h, dg and du are held in the operands' type: they are
// operands of matrix instructions, each rounding is at most a relative 2^-8
// (bf16) or 2^-11 (f16) of one term of a long sum, the size of the inputs' own
// rounding; outputs are off by about 1.4 times what their one rounding alone
// would leave.  As two planes they would cost every product of theirs a second
// matrix instruction, a third more of a forward's and five eighths more of a
// backward's (few rows, measured: 13.5 -> 15 us for 3 rows, 34 -> 49 us for 64, of
// 1024 x 4096 x 1024 bf16).  float16's range does not hold what lies between
// inputs and results, so it holds them in scaled blocks (gemm_tile.hpp,
// gemm_rows.hpp); that costs 2 % of large calls and 1 to 4 us of small ones
// (8192 x 2048 x 5632 backward 1505 -> 1530 us, 100 x 1024 x 4096 x 1024 48.7 -> 52.7).
// float32 keeps three bf16 planes (24 bits).  dh is no operand and stays float32: rounded as
// well, it would add half again to the error of dx, dWg and dWu.
#pragma once
#include <algorithm>
#include <cmath>

#include "../launch.hpp"
#include "gemm_rows.hpp"
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
  hipLaunchKernelGGL((gemm_tile_kernel<Dt, BM, BN, WM, WN, KS, S, AAcross, BAcross, Epi>),
                     dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(g.splits)), dim3(WM * WN * 64), 0, st, g);
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
// SplitSpace found for it.
template <typename Dt, bool AAcross, bool BAcross, int Epi>
int gemm_launch_split(GemmArgs& g, float* sums, hipStream_t st) {
  using T = std::conditional_t<Epi == kEpiStoreF32, float, typename Dt::T>;
  const Split p = plan_split<Dt>(g);
  if (p.splits == 1) return gemm_launch<Dt, AAcross, BAcross, Epi>(g, st);
  SplitSumArgs q{};
  split_into(g, p, sums, q);
  const int rc =
      gemm_launch_tile<Dt, 64, 64, 2, 2, kSmallK<Dt>, kSmallS<Dt>, AAcross, BAcross, kEpiStoreF32>(g, st);
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
  hipLaunchKernelGGL((gemm_two_kernel<Dt, kSmallK<Dt>, kSmallS<Dt>, EpiX, EpiW>), dim3(static_cast<unsigned>(blocks)),
                     dim3(256), 0, st, x, w, tiles[0], tiles[1]);
  return static_cast<int>(hipGetLastError());
}

// The two together, each split if that pays.
template <typename Dt>
int gemm_launch_two_split(GemmArgs& x, GemmArgs& w, float* sums, hipStream_t st) {
  const Split px = plan_split<Dt>(x), pw = plan_split<Dt>(w);
  SplitSumArgs q{};
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
    const double large = kTwoAcross || kBwd ? cost(256, 128, kBwd ? 1 : 2, 1.0) : cost(256, 256, 1, 1.0);
    const double c128 = cost(128, 128, 2, 0.8), c64 = cost(64, 64, 3, 0.45);
    if (large <= c128 && large <= c64) {
      if constexpr (kTwoAcross)
        return gemm_launch_tile<Dt, 256, 128, 2, 2, 32, 3, AAcross, BAcross, Epi>(g, st);
      else if constexpr (kBwd)
        return gemm_launch_tile<Dt, 256, 128, 4, 2, 64, 3, AAcross, BAcross, Epi>(g, st);
      else
        return gemm_launch_tile<Dt, 256, 256, 2, 4, 64, 2, AAcross, BAcross, Epi>(g, st);
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
struct FfnPlan {
  using T = typename Dt::T;
  static constexpr int P = Dt::kPlanes;
  Arena arena;
  PackArgs pack{};
  int packs = 0;
  int64_t pack_chunks = 0;

  explicit FfnPlan(void* ws) : arena{static_cast<char*>(ws)} {}

  // worst: as if the matrix had to be packed (the size query).  summed: over its
  // rows, in some product, whose loads of the last step would read rows past the
  // last where rows overlap (each starts within the one before).
  Operand use(const void* src, int64_t rows, int64_t width, int64_t ld, bool worst, bool summed = false) {
    Operand o{};
    if (!worst && P == 1 && !(summed && ld < width) && width % 8 == 0 && ld % 8 == 0 && reinterpret_cast<uintptr_t>(src) % 16 == 0) {
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
  static int64_t of(const GemmArgs& g) {
    const Split p = plan_split<Dt>(g);
    return p.splits > 1 ? p.splits * p.elements : 0;
  }
  void add(int64_t elements) { most = std::max(most, elements); }
};

template <typename Dt>
GemmArgs product(int64_t m, int64_t n, int64_t k, const Operand& a, const Operand& b, void* c, int64_t ldc) {
  GemmArgs g{};
  add_phase<Dt>(g, g.phases, a, b);
  g.batch = 1, g.m[0] = m, g.n[0] = n, g.k = k, g.lda[0] = a.ld, g.ldb[0] = b.ld, g.c[0] = c, g.ldc[0] = ldc;
  return g;
}

// x Wg^T and x Wu^T; the caller adds what the epilogue writes
template <typename Dt>
GemmArgs paired_product(const GatedFfnArgs& a, const Operand& x, const Operand& wg, const Operand& wu,
                        const Operand& h) {
  GemmArgs g{};
  // the two weights share a row stride: packing decides for both alike but for their alignment
  add_phase<Dt>(g, g.phases, x, wg, &wu);
  g.batch = 1, g.m[0] = a.n, g.n[0] = a.hidden, g.k = a.d_in, g.lda[0] = x.ld, g.ldb[0] = wg.ld;
  g.h = const_cast<uint16_t*>(h.plane[0]), g.ldh = h.ld, g.plane_stride = a.n * h.ld, g.act = a.act;
  g.e_h = h.exponents, g.e_ld = h.exponents_ld;
  return g;
}

template <typename Dt>
int ffn_fwd(const GatedFfnArgs& a, size_t* bytes) {
  const bool worst = bytes != nullptr;
  const hipStream_t st = static_cast<hipStream_t>(a.stream);
  if (takes_few_rows<Dt>(a.n, a.hidden, a.d_out)) {
    Arena arena{static_cast<char*>(a.workspace)};
    const int64_t ldh = round_up(a.hidden, 8);
    void* h = arena.take<typename Dt::T>(a.n * ldh);
    int8_t* e = nullptr;
    uint32_t* odd = nullptr;
    if constexpr (Dt::kScaled) {
      const int64_t groups = (a.hidden + 15) / 16;
      e = arena.take<int8_t>(a.n * groups);
      odd = arena.take<uint32_t>(round_up(groups, 4));
    }
    if (worst) {
      *bytes = arena.at;
      return 0;
    }
    const int rc =
        gemm_rows<Dt, true>({a.x, a.w_gate, a.w_up, h, e, odd, a.n, a.hidden, a.d_in, a.x_stride, ldh, a.act}, st);
    return rc ? rc
              : gemm_rows<Dt, false>({h, a.w_down, nullptr, a.out, e, odd, a.n, a.d_out, a.hidden, ldh, a.out_stride, 0},
                                     st);
  }
  FfnPlan<Dt> plan(a.workspace);
  const Operand x = plan.use(a.x, a.n, a.d_in, a.x_stride, worst);
  const Operand wg = plan.use(a.w_gate, a.hidden, a.d_in, a.d_in, worst);
  const Operand wu = plan.use(a.w_up, a.hidden, a.d_in, a.d_in, worst);
  const Operand wd = plan.use(a.w_down, a.d_out, a.hidden, a.hidden, worst);
  const Operand h = plan.hidden(a.n, a.hidden);
  GemmArgs g = paired_product<Dt>(a, x, wg, wu, h);
  GemmArgs d = product<Dt>(a.n, a.d_out, a.hidden, h, wd, a.out, a.out_stride);
  SplitSpace<Dt> space;
  space.add(space.of(d));
  float* sums = plan.arena.template take<float>(space.most);
  if (worst) {
    *bytes = plan.arena.at;
    return 0;
  }
  int rc = plan.run_pack(st);
  if (!rc) rc = gemm_launch<Dt, false, false, kEpiGated>(g, st);
  if (!rc) rc = gemm_launch_split<Dt, false, false, kEpiStore>(d, sums, st);
  return rc;
}

template <typename Dt>
int ffn_bwd(const GatedFfnArgs& a, size_t* bytes) {
  const bool worst = bytes != nullptr;
  const hipStream_t st = static_cast<hipStream_t>(a.stream);
  FfnPlan<Dt> plan(a.workspace);
  const Operand x = plan.use(a.x, a.n, a.d_in, a.x_stride, worst, true);
  const Operand wg = plan.use(a.w_gate, a.hidden, a.d_in, a.d_in, worst);
  const Operand wu = plan.use(a.w_up, a.hidden, a.d_in, a.d_in, worst);
  const Operand wd = plan.use(a.w_down, a.d_out, a.hidden, a.hidden, worst);
  const Operand go = plan.use(a.gout, a.n, a.d_out, a.gout_stride, worst, true);
  const Operand h = plan.hidden(a.n, a.hidden), dg = plan.hidden(a.n, a.hidden), du = plan.hidden(a.n, a.hidden);
  float* dh = plan.arena.template take<float>(a.n * h.ld);
  GemmArgs first = product<Dt>(a.n, a.hidden, a.d_out, go, wd, dh, h.ld);
  GemmArgs pair = paired_product<Dt>(a, x, wg, wu, h);
  pair.e_dg = dg.exponents, pair.e_du = du.exponents;
  pair.dg = const_cast<uint16_t*>(dg.plane[0]), pair.du = const_cast<uint16_t*>(du.plane[0]), pair.dh = dh;
  GemmArgs dx = product<Dt>(a.n, a.d_in, a.hidden, dg, wg, a.gx, a.d_in);
  add_phase<Dt>(dx, dx.phases, du, wu);
  GemmArgs dw = product<Dt>(a.hidden, a.d_in, a.n, dg, x, a.gw_gate, a.d_in);
  GemmArgs down = product<Dt>(a.d_out, a.hidden, a.n, go, h, a.gw_down, a.hidden);
  int at = 1;
  add_phase<Dt>(dw, at, du, x);
  dw.batch = 2;
  dw.m[1] = dw.m[0], dw.n[1] = dw.n[0], dw.lda[1] = dw.lda[0], dw.ldb[1] = dw.ldb[0], dw.ldc[1] = dw.ldc[0];
  dw.c[1] = a.gw_up;
  // The three products share a launch unless they fill many rounds of the card, where each is better chosen
  // a tile of its own.  One MI355X, us together and apart, by 64 x 64 tiles, bf16 | f32:
  //   238 (1357 x 322 x 853 x 257)        48,  58   |   101,  122
  //   1296 (4096 x 768 x 2304 x 768)     196, 207   |   768,  778
  //   2112 (8192 x 1024 x 2816 x 1024)   504, 525   |  2306, 2360
  //   8448 (4096 x 2048 x 5632 x 2048)   792, 806   |  4794, 4643
  // and of 8192 rows of the last 578 and 521 for these products alone.
  const int64_t tiles = round_up(a.hidden, 64) / 64 * (round_up(a.d_in, 64) / 64 * 2 + round_up(a.d_out, 64) / 64);
  const bool apart = tiles > 4096;
  if (!apart) {
    add_phase<Dt>(dw, at, go, h);
    dw.batch = 3;
    dw.m[2] = down.m[0], dw.n[2] = down.n[0], dw.lda[2] = down.lda[0], dw.ldb[2] = down.ldb[0];
    dw.ldc[2] = down.ldc[0], dw.c[2] = down.c[0];
  }
  SplitSpace<Dt> space;  // sized for every gradient, asked for or not
  space.add(space.of(first));
  space.add(space.of(dx) + space.of(dw));
  space.add(space.of(down));
  float* sums = plan.arena.template take<float>(space.most);
  if (worst) {
    *bytes = plan.arena.at;
    return 0;
  }
  int rc = plan.run_pack(st);
  if (!rc) rc = gemm_launch_split<Dt, false, true, kEpiStoreF32>(first, sums, st);
  if (!rc) rc = gemm_launch<Dt, false, false, kEpiGatedBwd>(pair, st);
  // Nor do dx and the weights' gradients wait for each other: up to two rounds of the card they share a launch too,
  // in 64 x 64 tiles.  One MI355X, us in one launch and in two, by tiles, bf16 | f32:
  //   370 (the first above)               42,  48   |    97,  100
  //   1024 (2000 x 512 x 2048 x 512)      75,  80   |   236,  238
  //   1240 (4096 x 640 x 1280 x 640)     115, 123   |   385,  393
  //   2064 (the second above)            198, 186   |   758,  774
  //   4160 (the third)                   681, 492   |  2566, 2309
  if (!rc && a.gx && a.gw_gate && tiles + round_up(a.n, 64) / 64 * (round_up(a.d_in, 64) / 64) <= 2 * 768)
    return gemm_launch_two_split<Dt>(dx, dw, sums, st);
  if (!rc && a.gx) rc = gemm_launch_split<Dt, false, true, kEpiStore>(dx, sums, st);
  if (!rc && a.gw_gate) {
    rc = gemm_launch_split<Dt, true, true, kEpiStore>(dw, sums, st);
    if (!rc && apart) rc = gemm_launch_split<Dt, true, true, kEpiStore>(down, sums, st);
  }
  return rc;
}

}  // namespace kern
}  // namespace segpoly
