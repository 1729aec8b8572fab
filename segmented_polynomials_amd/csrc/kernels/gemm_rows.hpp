// Products of a few rows with a weight matrix, out[m, o] = sum over k of
// x[m, k] w[o, k] for at most 32 rows: bound by reading the weights once.  A workgroup
// takes 16 weight rows (paired: of both matrices) and its waves share out the
// sum over k, 64 k at a time; weights and rows go from memory straight into
// the matrix instructions' registers, with no staging and no barrier before
// the waves' sums are added, in order, through LDS.  Loads are of 16 bytes at any
// alignment, float32 is split into its planes in registers: no operand is
// copied first.  With an output of 1024 columns the second product has 64
// workgroups, a quarter of the card, and takes longer (7 us, 8 MB) than the paired
// one with 256 (6 us, 16 MB; 3 rows of 1024 x 4096 x 1024 bf16): its own loads and
// sums bound it, not the memory.
// float16 hidden rows go from the paired product to the second in scaled blocks
// (gemm_tile.hpp), here of sixteen columns of one row.
#pragma once
#include <algorithm>

#include "gemm_tile.hpp"

namespace segpoly {
namespace kern {

// Which calls take this form: up to 16 rows all, up to 32 those whose second
// product's long sums over few outputs do not keep too few workgroups busy.  One
// MI355X, us here and in tiles (gemm_tile.hpp):
//                          bf16 8-16 rows   17           32          f32 17       32
//   128 x 512 x 128          6.0,  8.4    7.4,  8.6    7.8,  8.6   15,  18    16,  19
//   4096 x 1024 x 512       17.7, 25.7   20.7, 25.9   23.4, 26.0   63,  86    66,  89
//   512 x 2048 x 4096       10.9, 14.6   13.0, 14.7   14.5, 15.1   33,  45    35,  47
//   1024 x 2048 x 1024      11.5, 16.3   13.9, 16.5   15.6, 16.6   38,  45    40,  46
//   512 x 4096 x 512        13.7, 15.0   16.0, 15.1   18.7, 15.4   48,  38    52,  40
//   1024 x 4096 x 1024      15.7, 17.1   18.5, 17.0   21.8, 17.4   57,  53    59,  55
//   2048 x 5632 x 2048      27.6, 23.8   33.3, 23.7   39.1, 24.1  110, 129   112, 129
//   128 x 4096 x 8192       21.5, 20.8   25.0, 20.9   29.2, 21.3   64, 122    68, 124
// One row of the last but one 20.8 and 23.2.  48 rows: 128 x 512 x 128 bf16 10.5, 8.7,
// 1024 x 4096 x 1024 f32 88, 56.
template <typename Dt>
bool takes_few_rows(int64_t n, int64_t hidden, int64_t d_out) {
  return n <= 16 || (n <= 32 && (hidden <= 2048 || (Dt::kPlanes > 1 && hidden <= 3 * d_out)));
}

struct RowsArgs {
  const void *x, *w, *w2;  // [m][k] with row stride ldx, [n][k] dense; w2 of a paired product
  void* out;               // [m][ldo]
  int8_t* exponents;       // float16: of 16 columns of a hidden row, [m][hidden / 16]
  uint32_t* odd;           // and whether any row's is not zero, [hidden / 16], a byte a wave
  int64_t m, n, k, ldx, ldo;
  int act;
};

// eight k of a row from column c on, as the planes of a matrix operand
template <typename Dt>
struct RowChunk {
  using T = typename Dt::T;
  static constexpr int kLoads = sizeof(T) / 2;
  u32x4 raw[kLoads];
  __device__ __forceinline__ void load(const T* row, int c, int width) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) raw[i] = load_raw(row, c + i * 4, width);
  }
  __device__ __forceinline__ void planes(int c, int width, u16x8 (&p)[Dt::kPlanes]) const {
    if constexpr (Dt::kPlanes == 1) {
      p[0] = __builtin_bit_cast(u16x8, settle_chunk<T>(raw[0], c, width));
    } else {
      float v[8];
      unpack_chunk<T>(raw[0], c, width, v);
      unpack_chunk<T>(raw[1], c + 4, width, v + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        bf16 s[3];
        split3(v[i], s);
#pragma unroll
        for (int q = 0; q < 3; ++q) p[q][i] = __builtin_bit_cast(uint16_t, s[q]);
      }
    }
  }
};

// Waves of a workgroup: eight where the planes of more rows take their registers.
template <typename Dt>
constexpr int rows_waves(int m16) {
  return Dt::kPlanes > 1 && m16 > 1 ? 8 : 16;
}

// M16: blocks of 16 rows of x
template <typename Dt, int M16, bool Pair>
__global__ void __launch_bounds__(rows_waves<Dt>(M16) * 64)
gemm_rows_kernel(RowsArgs g) {
  using T = typename Dt::T;
  constexpr int P = Dt::kPlanes, W = Pair ? 2 : 1;
  __shared__ v4f sums[rows_waves<Dt>(M16)][W][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, waves = blockDim.x / 64;
  const int k = static_cast<int>(g.k);
  const int64_t o = static_cast<int64_t>(blockIdx.x) * 16 + lane % 16, last = g.n - 1;
  const T* w[W];  // rows past the last repeat it, and are not stored
  w[0] = static_cast<const T*>(g.w) + (o < last ? o : last) * g.k;
  if constexpr (Pair) w[1] = static_cast<const T*>(g.w2) + (o < last ? o : last) * g.k;
  const T* x[M16];
#pragma unroll
  for (int i = 0; i < M16; ++i) {
    const int64_t m = i * 16 + lane % 16;
    x[i] = static_cast<const T*>(g.x) + (m < g.m ? m : g.m - 1) * g.ldx;
  }
  v4f acc[W][M16];
  // the small products of several planes are summed apart, as in gemm_tile
  v4f small[P > 1 ? W : 1][P > 1 ? M16 : 1];
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int i = 0; i < M16; ++i) {
      acc[j][i] = v4f{0.f, 0.f, 0.f, 0.f};
      if constexpr (P > 1) small[j][i] = v4f{0.f, 0.f, 0.f, 0.f};
    }
  // float16: where any exponent is not zero the sum is made a second time, with
  // them.  Row i's is then in units of the present ones (lane % 16 has it), as in
  // gemm_tile, and the two sixteens of a step are added apart.
  constexpr bool kUnits = Dt::kScaled && !Pair;
  int unit[M16], top[M16];
  const int groups = (k + 15) / 16;
  u32x4 odd = {0, 0, 0, 0};
  if constexpr (kUnits)
    if (lane * 4 < groups) odd = *reinterpret_cast<const u32x4*>(g.odd + lane * 4);
  auto add = [&](auto units, int j, int i, const u16x8(&pw)[P], const u16x8(&px)[P], int e) {
    if constexpr (units) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bool mine = lane / 32 == s;
        const int es = static_cast<int>(max_over_rows(static_cast<float>(mine ? e : kNoValue)));
        top[i] = es > top[i] ? es : top[i];
        const int to = es == kNoValue ? unit[i] : es > top[i] - kReach ? es : top[i] - kReach;
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[j][i][q] = __builtin_ldexpf(acc[j][i][q], unit[i] - to);
        unit[i] = to;
        const u16x8 part = es < to && es != kNoValue ? lower(px[0], es - to) : px[0];
        acc[j][i] = mma16(typename Dt::E{}, mine ? pw[0] : u16x8{}, mine ? part : u16x8{}, acc[j][i]);
      }
    } else if constexpr (P == 1) {
      acc[j][i] = mma16(typename Dt::E{}, pw[0], px[0], acc[j][i]);
    } else {
#pragma unroll
      for (int t = 0; t < 6; ++t) {
        v4f& c = t < 5 ? small[j][i] : acc[j][i];
        c = mma16(typename Dt::E{}, pw[kPairs3[t][1]], px[kPairs3[t][0]], c);
      }
    }
  };
  auto run = [&](auto units) {
    constexpr int kUnroll = units ? 1 : P == 1 && M16 == 1 ? 4 : 2;
#pragma unroll(kUnroll)
    for (int k0 = wave * 64; k0 < k; k0 += waves * 64) {
      RowChunk<Dt> rw[2][W], rx[2][M16];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = k0 + h * 32 + lane / 16 * 8;
#pragma unroll
        for (int j = 0; j < W; ++j) rw[h][j].load(w[j], c, k);
#pragma unroll
        for (int i = 0; i < M16; ++i) rx[h][i].load(x[i], c, k);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = k0 + h * 32 + lane / 16 * 8;
        auto exponent = [&](int i) -> int {
          if constexpr (units) {
            const int64_t m = i * 16 + lane % 16;
            return c < k ? g.exponents[(m < g.m ? m : g.m - 1) * groups + c / 16] : kNoValue;
          }
          return 0;
        };
        if constexpr (M16 == 1) {  // one weight's planes at a time: sixteen waves have 128 registers each
          u16x8 px[P];
          rx[h][0].planes(c, k, px);
#pragma unroll
          for (int j = 0; j < W; ++j) {
            u16x8 pw[P];
            rw[h][j].planes(c, k, pw);
            add(units, j, 0, pw, px, exponent(0));
          }
        } else {
          u16x8 pw[W][P];
#pragma unroll
          for (int j = 0; j < W; ++j) rw[h][j].planes(c, k, pw[j]);
#pragma unroll
          for (int i = 0; i < M16; ++i) {
            u16x8 px[P];
            rx[h][i].planes(c, k, px);
#pragma unroll
            for (int j = 0; j < W; ++j) add(units, j, i, pw[j], px, exponent(i));
          }
        }
      }
    }
  };
  run(std::false_type{});
  if constexpr (kUnits) {
    uint32_t any = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) any |= lane * 4 + q < groups ? odd[q] : 0;
    for (int t = 256 + lane; t < groups; t += 64) any |= g.odd[t];
    if (__ballot(any != 0)) {
#pragma unroll
      for (int i = 0; i < M16; ++i) {
        acc[0][i] = v4f{0.f, 0.f, 0.f, 0.f};
        unit[i] = top[i] = kNoValue;
      }
      run(std::true_type{});
#pragma unroll
      for (int i = 0; i < M16; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[0][i][q] = __builtin_ldexpf(acc[0][i][q], unit[i]);
    }
  }
  bool not_zero = false;  // an exponent of this thread's
  // lane l of a fragment holds weight rows l / 16 * 4 + q of row l % 16
#pragma unroll
  for (int i = 0; i < M16; ++i) {
    if (i) __syncthreads();
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if constexpr (P > 1) acc[j][i] = add_small(acc[j][i], small[j][i]);
      sums[wave][j][lane] = acc[j][i];
    }
    __syncthreads();
    if (threadIdx.x < 256) {
      const int l = threadIdx.x / 16 + threadIdx.x % 16 / 4 * 16, q = threadIdx.x % 4;
      float v[W];
#pragma unroll
      for (int j = 0; j < W; ++j) {
        v[j] = 0.f;
        for (int s = 0; s < waves; ++s) v[j] += sums[s][j][l][q];
      }
      const int64_t m = i * 16 + l % 16, n = static_cast<int64_t>(blockIdx.x) * 16 + l / 16 * 4 + q;
      if constexpr (Pair) v[0] = act_value(v[0], g.act) * v[1];
      if constexpr (Pair && Dt::kScaled) {  // sixteen lanes have a row's sixteen columns
        const int e = block_exponent(lane_max<16>(finite_abs(v[0])));
        v[0] *= block_scale(e);
        not_zero |= e != 0 && e != kNoValue;
        if (m < g.m && l / 16 + q == 0) g.exponents[m * ((g.n + 15) / 16) + blockIdx.x] = static_cast<int8_t>(e);
      }
      if (m < g.m && n < g.n) {
        static_cast<T*>(g.out)[m * g.ldo + n] = static_cast<T>(v[0]);
      }
    }
  }
  if constexpr (Pair && Dt::kScaled) {
    if (threadIdx.x < 256) {
      const bool any = __ballot(not_zero) != 0;
      if (lane == 0) reinterpret_cast<uint8_t*>(g.odd + blockIdx.x)[wave] = any;
    }
  }
}

template <typename Dt, int M16, bool Pair>
int gemm_rows_launch(const RowsArgs& g, hipStream_t st) {
  const int64_t waves = std::min<int64_t>(rows_waves<Dt>(M16), std::max<int64_t>(4, (g.k + 63) / 64));
  hipLaunchKernelGGL((gemm_rows_kernel<Dt, M16, Pair>), dim3(static_cast<unsigned>((g.n + 15) / 16)),
                     dim3(static_cast<unsigned>(waves * 64)), 0, st, g);
  return static_cast<int>(hipGetLastError());
}

template <typename Dt, bool Pair>
int gemm_rows(const RowsArgs& g, hipStream_t st) {
  if (g.m <= 16) return gemm_rows_launch<Dt, 1, Pair>(g, st);
  return gemm_rows_launch<Dt, 2, Pair>(g, st);
}

}  // namespace kern
}  // namespace segpoly
