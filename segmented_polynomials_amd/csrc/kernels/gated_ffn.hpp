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

#include "gemm_plan.hpp"
#include "gemm_rows.hpp"

namespace segpoly {
namespace kern {

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
        gemm_rows<Dt, kRowsPaired>({a.x, a.w_gate, a.w_up, h, e, odd, a.n, a.hidden, a.d_in, a.x_stride, ldh, a.act}, st);
    return rc ? rc
              : gemm_rows<Dt, kRowsPlain>({h, a.w_down, nullptr, a.out, e, odd, a.n, a.d_out, a.hidden, ldh, a.out_stride, 0},
                                          st);
  }
  MatrixPlan<Dt> plan(a.workspace);
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
  MatrixPlan<Dt> plan(a.workspace);
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
