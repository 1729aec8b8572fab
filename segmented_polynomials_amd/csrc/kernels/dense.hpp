// The dense layer, out = act(x W^T + bias) + residual, and its gradient as tile
// products (gemm_tile.hpp), for one element type per translation unit:
//   forward   one product, bias, activation and residual its epilogue
//             (few rows: gemm_rows.hpp; many under a small weight: dense_stream.hpp)
//   backward  d = g act'(x W^T + bias)      the product again, the slope and the
//                                           gradient its epilogue; without an
//                                           activation d is g itself
//             dx = d W, dW = d^T x, dbias = sums of d's columns
//             (at most four rows: dense_few.hpp; up to 64 x 64 columns, many rows:
//             dense_fused.hpp)
// Between the products d is held in the operands' type, as it is an operand of
// matrix instructions: one rounding of a term of a long sum, the size of the
// inputs' own (float16 in scaled blocks, gemm_tile.hpp; float32 as it is,
// gemm_staged.hpp).
// The column sums are of d before that rounding: each wave of the product leaves
// its rows' in float32, a second launch adds them in order.
// Bound by the matrix units and, at sums of a few hundred, by the epilogue, which runs
// beside a second workgroup's products.  One MI355X, 8192 x 2048 x 5632 bf16 with gelu:
// gradients 609 to 655 us by card (865 to 930 TFLOP/s), the product with the slope 259 of them.
#pragma once
#include <algorithm>

#include "column_sums.hpp"
#include "dense_few.hpp"
#include "dense_fused.hpp"
#include "dense_stream.hpp"
#include "gemm_plan.hpp"
#include "gemm_rows.hpp"

namespace segpoly {
namespace kern {

// The shares of a long sum, in order, then the epilogue: four columns a lane.
struct DenseSumArgs {
  const float* from;
  int64_t split_stride, m, n, ld;
  int splits, act;
  const void *bias, *res;
  int64_t ld_res;
  void* to;
  int64_t ldc;
};
template <typename T>
__global__ void __launch_bounds__(256)
dense_sum_kernel(DenseSumArgs g) {
  const int64_t quads = g.ld / 4, total = g.m * quads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = i / quads, c = i % quads * 4;
    const float* from = g.from + r * g.ld + c;
    v4f s = {0.f, 0.f, 0.f, 0.f}, res = s;
    if (g.bias) s = load_four(static_cast<const T*>(g.bias), c, g.n);
    if (g.res) res = load_four(static_cast<const T*>(g.res) + r * g.ld_res, c, g.n);
    v4f p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int k = 0; k < g.splits; ++k) p += *reinterpret_cast<const v4f*>(from + k * g.split_stride);
    T v[4];
    with_act(g.act, [&](auto act) {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = static_cast<T>(dense_act(act, p[q] + s[q]) + res[q]);
    });
    T* to = static_cast<T*>(g.to) + r * g.ldc + c;
    if (c + 4 <= g.n) {
      __builtin_memcpy(to, v, sizeof(v));
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (c + q < g.n) to[q] = v[q];
    }
  }
}

template <typename T>
int dense_sum(const DenseSumArgs& g, hipStream_t st) {
  const int64_t blocks = std::min<int64_t>((g.m * (g.ld / 4) + 255) / 256, 2048);
  hipLaunchKernelGGL(dense_sum_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, g);
  return static_cast<int>(hipGetLastError());
}

// The shares of x w^T of few rows, [shares][n][ld].
template <typename Dt>
int few_sums(RowsArgs r, float* sums, int64_t ld, hipStream_t st) {
  r.out = sums, r.ldo = ld, r.k_share = few_share(r.k, r.n), r.share_stride = r.m * ld;
  return gemm_rows<Dt, kRowsSums>(r, st);
}

// Column sums of a segment of the rows: 32 chunks of 16 bytes by 8 rows at a
// time, whose sums are added in order.
constexpr int64_t kSegmentRows = 64;  // 500 x 256 bf16 gradient without activation 11 us, 14 with 256; 20000 x 128 21, 24
template <typename T>
__global__ void __launch_bounds__(256)
dense_columns_kernel(const void* __restrict__ src, int64_t n, int64_t stride, int64_t width, int64_t rows, float* sums,
                     int64_t ld_sums) {
  constexpr int V = Chunk<T>::kN;
  __shared__ float lds[8][32 * V];
  const int c = static_cast<int>((blockIdx.x * 32 + threadIdx.x % 32) * V), set = threadIdx.x / 32;
  const int64_t from = blockIdx.y * rows, to = from + rows < n ? from + rows : n;
  float s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = 0.f;
#pragma unroll 8
  for (int64_t r = from + set; r < to; r += 8) {
    float v[V];
    load_chunk(static_cast<const T*>(src) + r * stride, c, static_cast<int>(width), v);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] += v[i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) lds[set][threadIdx.x % 32 * V + i] = s[i];
  __syncthreads();
  for (int k = threadIdx.x; k < 32 * V; k += 256) {
    const int64_t col = static_cast<int64_t>(blockIdx.x) * (32 * V) + k;
    if (col >= width) continue;
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) t += lds[q][k];
    sums[blockIdx.y * ld_sums + col] = t;
  }
}
// to[m][c] = sum over p of sums[p][m][c]; `ld` between rows, a multiple of four from the
// width on.  Row `rows` is the bias's, of partial rows of its own.
struct FoldArgs {
  const float *sums, *bias_sums;
  int64_t parts, rows, width, bias_parts, bias_width;
  void *to, *to_bias;
};
template <typename T>
__global__ void __launch_bounds__(1024)
dense_fold_kernel(FoldArgs g) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x % 32, m = blockIdx.y;
  const bool bias = m == g.rows;
  const int64_t width = bias ? g.bias_width : g.width, ld = (width + 3) / 4 * 4;
  if (static_cast<int64_t>(blockIdx.x) * 32 >= width) return;
  const float t = bias ? column_sum(g.bias_sums, g.bias_parts, ld, width, c)
                       : column_sum(g.sums + m * ld, g.parts, g.rows * ld, width, c);
  T* to = static_cast<T*>(bias ? g.to_bias : g.to) + (bias ? 0 : m * width);
  if (threadIdx.x < 32 && c < width) to[c] = static_cast<T>(t);
}
// what of the two is asked for, and not null
template <typename T>
int dense_fold(FoldArgs g, hipStream_t st) {
  if (!g.to) g.rows = g.width = 0;
  if (!g.to_bias) g.bias_width = 0;
  const int64_t wide = std::max(g.width, g.bias_width), rows = g.rows + (g.bias_width ? 1 : 0);
  if (wide == 0 || rows == 0) return 0;
  hipLaunchKernelGGL(dense_fold_kernel<T>, dim3(static_cast<unsigned>((wide + 31) / 32), static_cast<unsigned>(rows)),
                     dim3(1024), 0, st, g);
  return static_cast<int>(hipGetLastError());
}

// rows of a segment: at most 2048 segments, whose sums are added up again
inline int64_t segment_rows(int64_t n) { return std::max(kSegmentRows, round_up((n + 2047) / 2048, 8)); }
inline int64_t segments(int64_t n) { return (n + segment_rows(n) - 1) / segment_rows(n); }

constexpr int64_t kFewRows = 16, kFewRowsBwd = 4;

// The rows' form of the product against tiles (or the streaming form).  One MI355X, us, silu, rows' form first:
//                 16 x 64 x 64    16 x 1024 x 1024   16 x 4096 x 4096   32 x 256 x 256   32 x 1024 x 4096
//   forward bf16      3.1, 3.6          6.4, 8.1            11, 12          3.9, 4.1          6.3, 7.9
//           f32       4.6, 5.3          9.1, 13             23, 29          6.9, 11           13, 15
//   gradient's: 16 rows of 64 x 64 bf16 9.2, 8.1, f32 12, 10; of 256 x 256 10.5, 9.7 and 19, 22; of 1024 x 1024
//   15, 16 and 23, 27; of 4096 x 4096 41, 39 and 83, 87 (its slope takes a launch more)
// and where 17 to 32 rows end, 17 and 32 rows (f16 as bf16):
//   bf16  64 x 64 3.3, 3.4 and 3.4, 3.6; 2048 x 512 7.0, 9.6 and 7.5, 9.6; 2048 x 4096 8.5, 10.8 and 9.7, 11.0; 8192 x
//         512 7.9, 9.5 and 8.6, 9.6; 4096 x 1024 8.5, 10.1 and 9.3, 10.3; 1024 x 8192 7.8, 8.8 and 9.2, 8.9; 7920 x
//         791 (28 rows) 10.5, 12.9; past these 4096 x 2048 12.3, 11.2 and 15.1, 11.4; 8192 x 1024 11.2, 10.8 and 12.6,
//         10.9; 512 x 16384 7.8, 7.1 and 9.3, 7.2.
//         Weights of even width that the tiles need copied: 510 x 512 4.2, 8.4 and 4.5, 8.4; 2046 x 4096 8.5, 22 and
//         9.4, 22; 8190 x 8192 38, 78 and 49, 83; odd ones, whose loads cost more, as those of whole chunks
//   f32   136 x 64 6.1, 8.1 and 6.0, 8.2; 512 x 512 7.8, 11.4 and 8.5, 11.7; 1024 x 8192 18, 23 and 20, 23; 2048 x 512
//         10.8, 12.3 and 11.3, 12.6; 4096 x 512 10.1, 12.4 and 10.7, 12.8; past these 128 x 1024 6.1, 5.4 and 6.2, 5.4;
//         2048 x 2048 20.4, 14.4 and 21.6, 14.5; 4096 x 4096 37, 27 and 39, 27; 256 x 32768 18.9, 14.8 and 20.9, 15.3;
//         and of widths that the tiles load in pieces, 125 x 5920 (19 rows) 7.1, 10.2; 1897 x 2959 (31) 19.7, 24.7; 1669 x
//         5377 (22) 24.8, 37.4; but 2046 x 2048 6 to 10 % behind
template <typename Dt>
bool takes_few_fwd(int64_t n, int64_t d_in, int64_t d_out) {
  if (n <= kFewRows || n > 2 * kFewRows) return n <= kFewRows;
  const int64_t size = d_in * d_out;
  if (kStaged<Dt>) {
    if (d_in % 4 != 0 && d_in > 1024 && d_in <= 2048) return d_out <= 8192;
    return d_in > (d_out <= 4096 ? 128 : 64) && d_out <= 8192 && (d_in <= 1024 || size <= 1 << 21);
  }
  if (d_in % 8 != 0 && d_in % 2 == 0) return true;
  return d_out <= (d_in <= 1024 ? 8192 : 4096) && size <= (d_in <= 2048 ? 1 << 23 : 3 << 21);
}
template <typename Dt>
bool takes_few_bwd(int64_t n, int64_t d_in) { return n <= kFewRows && d_in >= (kStaged<Dt> ? 128 : 512); }

// Float32: the gradients of x and the weight apart, each in tiles of 128 x 128, where x's fill rounds of a workgroup
// a unit and the weight's are shared out; else together in tiles of 64 x 64.  One MI355X, us apart, together: 8000 x
// 512 x 512 110, 123 (252 tiles of x); 4000 x 1024 x 512 121, 134 (256); 20000 x 256 x 256 107, 98 (314); 3000 x 512 x
// 512 86, 68 (96).  bf16 the same calls 53, 49; 46, 43; 52, 50; 37, 31.
template <typename Dt>
bool takes_apart(const DenseArgs& a, const GemmArgs& dw) {
  if (!kStaged<Dt> || plan_split_wide<Dt>(dw).splits < 2) return false;
  const int64_t tiles = (a.n + 127) / 128 * ((a.d_in + 127) / 128);
  return tiles * 4 >= round_up(tiles, 256) * 3;
}

template <typename Dt>
int dense_fwd(const DenseArgs& a, size_t* bytes) {
  using T = typename Dt::T;
  const bool worst = bytes != nullptr;
  const hipStream_t st = static_cast<hipStream_t>(a.stream);
  if (takes_few_fwd<Dt>(a.n, a.d_in, a.d_out)) {
    const int64_t shares = few_shares(a.d_in, a.d_out);
    Arena arena{static_cast<char*>(a.workspace)};
    const int64_t ld = round_up(a.d_out, 4);
    float* sums = arena.take<float>(shares > 1 ? shares * a.n * ld : 0);
    if (worst) {
      *bytes = arena.at;
      return 0;
    }
    RowsArgs r{a.x, a.w, nullptr, a.out, nullptr, nullptr, a.n, a.d_out, a.d_in, a.x_stride, a.out_stride, a.act};
    r.bias = a.bias, r.res = a.residual, r.ld_res = a.residual_stride;
    if (shares == 1) return gemm_rows<Dt, kRowsDense>(r, st);
    const int rc = few_sums<Dt>(r, sums, ld, st);
    return rc ? rc
              : dense_sum<T>({sums, a.n * ld, a.n, a.d_out, ld, static_cast<int>(shares), a.act, a.bias, a.residual,
                              a.residual_stride, a.out, a.out_stride}, st);
  }
  if (takes_stream<Dt>(a.n, a.d_in, a.d_out)) {
    if (worst) {
      *bytes = 0;
      return 0;
    }
    return dense_stream<Dt>({a.x, a.w, a.bias, a.residual, a.out, a.n, a.x_stride, a.residual_stride, a.out_stride,
                             static_cast<int>(a.d_in), static_cast<int>(a.d_out), a.act, 0}, st);
  }
  MatrixPlan<Dt> plan(a.workspace);
  const Operand x = plan.use(a.x, a.n, a.d_in, a.x_stride, worst);
  const Operand w = plan.use(a.w, a.d_out, a.d_in, a.d_in, worst);
  GemmArgs g = product<Dt>(a.n, a.d_out, a.d_in, x, w, a.out, a.out_stride);
  g.act = a.act, g.bias = a.bias, g.res = a.residual, g.ld_res = a.residual_stride;
  SplitSpace<Dt> space;
  space.add(space.of(g));
  float* sums = plan.arena.template take<float>(space.most);
  if (worst) {
    *bytes = plan.arena.at;
    return 0;
  }
  int rc = plan.run_pack(st);
  if (rc) return rc;
  const Split p = plan_split<Dt>(g);
  if (p.splits == 1) return gemm_launch<Dt, false, false, kEpiDense>(g, st);
  SplitSumArgs q{};
  split_into(g, p, sums, q);
  rc = gemm_launch_tile<Dt, 64, 64, 2, 2, kSmallK<Dt>, kSmallS<Dt>, false, false, kEpiStoreF32>(g, st);
  if (rc) return rc;
  return dense_sum<T>({sums, q.split_stride[0], a.n, a.d_out, q.ld[0], p.splits, a.act, a.bias, a.residual,
                       a.residual_stride, a.out, a.out_stride}, st);
}

// At most kFewRowsBwd rows: three or four launches, each about as long as the weight
// takes to cross memory once.
template <typename Dt>
int dense_bwd_few(const DenseArgs& a, size_t* bytes) {
  using T = typename Dt::T;
  const bool again = a.act != kActNone;
  const hipStream_t st = static_cast<hipStream_t>(a.stream);
  Arena arena{static_cast<char*>(a.workspace)};
  const int64_t ld = round_up(a.d_out, 4), ld_dx = round_up(a.d_in, 4), shares = few_shares(a.d_in, a.d_out);
  const FewPlan p = few_plan<T>(a.n, a.d_in, a.d_out);
  float* d = arena.take<float>(a.n * ld);
  float* sums = arena.take<float>(again ? shares * a.n * ld : 0);
  float* dx = arena.take<float>(p.parts * a.n * ld_dx);
  if (bytes) {
    *bytes = arena.at;
    return 0;
  }
  int rc = 0;
  if (again) {
    RowsArgs r{a.x, a.w, nullptr, nullptr, nullptr, nullptr, a.n, a.d_out, a.d_in, a.x_stride, 0, 0};
    rc = few_sums<Dt>(r, sums, ld, st);
    if (rc) return rc;
  }
  SlopeArgs s{};
  s.from = again ? sums : nullptr, s.split_stride = a.n * ld, s.m = a.n, s.n = a.d_out, s.ld = ld;
  s.splits = static_cast<int>(shares), s.act = a.act, s.bias = again ? a.bias : nullptr, s.gout = a.gout;
  s.ld_gout = a.gout_stride, s.d = d, s.ld_d = ld, s.gbias = a.gbias;
  rc = dense_slope<Dt, true>(s, st);
  if (rc || (!a.gx && !a.gw)) return rc;
  FewArgs f{a.x, a.w, d, a.gx ? dx : nullptr, a.gw, a.d_in, a.d_out, a.x_stride, ld, ld_dx, static_cast<int>(a.n),
            static_cast<int>(p.rows), p.lanes};
  rc = dense_few_bwd<T>(f, p, st);
  if (rc || !a.gx) return rc;
  return dense_fold<T>({dx, nullptr, p.parts, a.n, a.d_in, 0, 0, a.gx, nullptr}, st);
}

// Up to 64 by 64 columns: one pass over the rows, then its workgroups' sums.
template <typename Dt>
int dense_bwd_fused(const DenseArgs& a, size_t* bytes) {
  using T = typename Dt::T;
  const hipStream_t st = static_cast<hipStream_t>(a.stream);
  Arena arena{static_cast<char*>(a.workspace)};
  const int64_t blocks = fused_blocks(a.n), ld = round_up(a.d_in, 4), ld_bias = round_up(a.d_out, 4);
  float* dw = arena.take<float>(blocks * a.d_out * ld);
  float* dbias = arena.take<float>(blocks * ld_bias);
  if (bytes) {
    *bytes = arena.at;
    return 0;
  }
  int rc = dense_fused_bwd<Dt>({a.x, a.w, a.act == kActNone ? nullptr : a.bias, a.gout, a.gx, a.gw ? dw : nullptr,
                                a.gbias ? dbias : nullptr, a.n, a.x_stride, a.gout_stride, static_cast<int>(a.d_in),
                                static_cast<int>(a.d_out), a.act}, st);
  return rc ? rc : dense_fold<T>({dw, dbias, blocks, a.d_out, a.d_in, blocks, a.d_out, a.gw, a.gbias}, st);
}

template <typename Dt>
int dense_bwd(const DenseArgs& a, size_t* bytes) {
  using T = typename Dt::T;
  if (takes_fused_bwd<T>(a.n, a.d_in, a.d_out)) return dense_bwd_fused<Dt>(a, bytes);
  if (a.n <= kFewRowsBwd) return dense_bwd_few<Dt>(a, bytes);
  const bool worst = bytes != nullptr, product_again = a.act != kActNone;
  const hipStream_t st = static_cast<hipStream_t>(a.stream);
  MatrixPlan<Dt> plan(a.workspace);
  const Operand x = plan.use(a.x, a.n, a.d_in, a.x_stride, worst, true);
  const Operand w = plan.use(a.w, a.d_out, a.d_in, a.d_in, worst);
  const Operand d = product_again ? plan.hidden(a.n, a.d_out) : plan.use(a.gout, a.n, a.d_out, a.gout_stride, worst, true);
  GemmArgs again = product<Dt>(a.n, a.d_out, a.d_in, x, w, nullptr, 0);
  again.act = a.act, again.bias = a.bias, again.res = a.gout, again.ld_res = a.gout_stride;
  again.dg = const_cast<uint16_t*>(d.plane[0]), again.ldh = d.ld, again.plane_stride = a.n * d.ld;
  again.e_dg = d.exponents, again.e_ld = d.exponents_ld;
  Split shared = product_again ? plan_split<Dt>(again) : Split{};
  const bool few = product_again && takes_few_bwd<Dt>(a.n, a.d_in);
  const int64_t ld_shared = round_up(a.d_out, 4);
  if (few) shared.splits = static_cast<int>(few_shares(a.d_in, a.d_out)), shared.elements = a.n * ld_shared;
  GemmArgs dx = product<Dt>(a.n, a.d_in, a.d_out, d, w, a.gx, a.d_in);
  GemmArgs dw = product<Dt>(a.d_out, a.d_in, a.n, d, x, a.gw, a.d_in);
  SplitSpace<Dt> space;  // sized for every gradient, asked for or not
  space.add(few ? shared.splits * shared.elements : space.of(shared));
  space.add(space.of(dx) + space.of(dw));
  space.add(space.of(plan_split_wide<Dt>(dx)));
  space.add(space.of(plan_split_wide<Dt>(dw)));
  float* sums = plan.arena.template take<float>(space.most);
  const int64_t ld_columns = round_up(a.d_out, 4);
  float* columns =
      plan.arena.template take<float>((product_again ? (a.n + 63) / 64 * 2 + 2 : segments(a.n)) * ld_columns);
  if (worst) {
    *bytes = plan.arena.at;
    return 0;
  }
  int rc = plan.run_pack(st);
  if (rc) return rc;
  int64_t column_rows = 0;
  if (few || shared.splits > 1) {
    if (few) {
      const RowsArgs r{a.x, a.w, nullptr, nullptr, nullptr, nullptr, a.n, a.d_out, a.d_in, a.x_stride, 0, 0};
      rc = few_sums<Dt>(r, sums, ld_shared, st);
    } else {
      SplitSumArgs q{};
      split_into(again, shared, sums, q);
      rc = gemm_launch_tile<Dt, 64, 64, 2, 2, kSmallK<Dt>, kSmallS<Dt>, false, false, kEpiStoreF32>(again, st);
    }
    if (rc) return rc;
    SlopeArgs s{};
    s.from = sums, s.split_stride = shared.elements, s.m = a.n, s.n = a.d_out, s.ld = ld_shared, s.splits = shared.splits;
    s.act = a.act, s.bias = a.bias, s.gout = a.gout, s.ld_gout = a.gout_stride, s.d = again.dg, s.ld_d = d.ld;
    s.exponents = d.exponents, s.e_ld = d.exponents_ld, s.column_sums = a.gbias ? columns : nullptr;
    rc = dense_slope<Dt, kStaged<Dt>>(s, st);
    column_rows = (a.n + 63) / 64;
  } else if (product_again) {
    again.column_sums = a.gbias ? columns : nullptr;
    rc = gemm_launch<Dt, false, false, kEpiDenseBwd>(again, st);
    column_rows = again.column_rows;
  } else if (a.gbias) {
    column_rows = segments(a.n);
    constexpr int kWide = 32 * Chunk<T>::kN;
    hipLaunchKernelGGL(dense_columns_kernel<T>,
                       dim3(static_cast<unsigned>((a.d_out + kWide - 1) / kWide), static_cast<unsigned>(column_rows)),
                       dim3(256), 0, st, a.gout, a.n, a.gout_stride, a.d_out, segment_rows(a.n), columns, ld_columns);
    rc = static_cast<int>(hipGetLastError());
  }
  // the bias's sums: few partial rows join the last launch that adds shares, which reads them one after another (500 x
  // 256 x 256 float32, 14 rows: 27 us, 29 apart; 1357 x 322 x 853 bf16, 42 rows: 30, 28)
  SplitSumArgs last{};
  if (a.gbias && column_rows <= 16 && (a.gx || a.gw)) {
    last.batch = 1, last.from[0] = columns, last.to[0] = a.gbias, last.m[0] = 1, last.n[0] = a.d_out;
    last.ld[0] = ld_columns, last.ldc[0] = a.d_out, last.split_stride[0] = ld_columns;
    last.splits[0] = static_cast<int>(column_rows);
  } else if (!rc) {
    rc = dense_fold<T>({nullptr, columns, 0, 0, 0, column_rows, a.d_out, nullptr, a.gbias}, st);
  }
  if (rc) return rc;
  const int64_t tiles = round_up(a.d_in, 64) / 64 * (round_up(a.d_out, 64) / 64 + round_up(a.n, 64) / 64);
  if (a.gx && a.gw && tiles <= 2 * 768 && !takes_apart<Dt>(a, dw))
    return gemm_launch_two_split<Dt>(dx, dw, sums, st, last);
  if (a.gx) rc = gemm_launch_split<Dt, false, true, kEpiStore, true>(dx, sums, st, a.gw ? SplitSumArgs{} : last);
  if (!rc && a.gw) rc = gemm_launch_split<Dt, true, true, kEpiStore, true>(dw, sums, st, last);
  return rc;
}

}  // namespace kern
}  // namespace segpoly
