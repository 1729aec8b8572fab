// The gradient of the dense layer of up to 64 by 64 columns in one pass over the rows:
//   d = g act'(x W^T + bias),   dx = d W,   dW = d^T x,   dbias = sums of d's columns
// Bound by memory: x and g are read once and dx is written once; a product at a time
// would write d and read it twice, x twice and g three times.  A wave takes 16 rows at
// a time (32 at once spill: float32 293 us for 600000 x 64 x 64, 147 with 16).  The
// weight stays in LDS in the two orders that its products take.  The product leaves
// each lane eight neighbouring columns of a row (dense_stream.hpp), and d of these is
// at once an operand of the next.  For dW the 16 rows are the sum: x and d go through
// the wave's own LDS, whose transposing reads bring them back by columns; no barrier.
// A wave holds dW of its rows in registers, a workgroup adds its eight waves', a second
// launch the workgroups'.
// d is not rounded to the rows' type: it is an operand as two bf16 planes (float32:
// three), float16 rows and weights as two.
#pragma once
#include <algorithm>

#include "dense_stream.hpp"

namespace segpoly {
namespace kern {

// planes of x and the weight, and of d
template <typename T>
struct FusedPlanes {
  static constexpr int kX = sizeof(T) == 4 ? 3 : std::is_same_v<T, bf16> ? 1 : 2;
  static constexpr int kD = sizeof(T) == 4 ? 3 : 2;
};

// Eight values as P planes of bf16; the last may round.
template <int P>
__device__ __forceinline__ void split_planes(const float (&v)[8], u16x8 (&p)[P]) {
  if constexpr (P == 3) {
    split_eight(v, p);
  } else {
    float r[8], top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[i], top = __builtin_fmaxf(top, __builtin_fabsf(v[i]));
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bf16 s = static_cast<bf16>(r[i]);
        p[q][i] = __builtin_bit_cast(uint16_t, s);
        if (q < P - 1) r[i] -= static_cast<float>(s);
      }
    if (P > 1 && __ballot(top >= 0x1.ffp127f)) {
      u16x8 s[3];
      split_slow(v, s);
#pragma unroll
      for (int q = 0; q < P; ++q) p[q] = s[q];
    }
  }
}

__device__ __forceinline__ v4f mma16(bf16, s16x4 a, s16x4 b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(a, b, c, 0, 0, 0);
}

// c (large products) and s (small ones) of the planes of two operands with those of b,
// in turn: neither waits for its own last.  Of two planes each, whole float16 values, all
// four products count: the smallest is up to 2^-16 of the largest.
template <int PA, int PB, typename V>
__device__ __forceinline__ void multiply_two(const V (&a)[2][PA], const V (&b)[PB], v4f (&c)[2], v4f (&s)[2]) {
  constexpr int kTop = PA == 2 && PB == 2 ? 2 : (PA > PB ? PA : PB) - 1;  // of the sum of two planes' numbers
#pragma unroll
  for (int t = kTop; t > 0; --t)
#pragma unroll
    for (int i = 0; i < PA; ++i)
      if (t - i >= 0 && t - i < PB)
#pragma unroll
        for (int k = 0; k < 2; ++k) s[k] = mma16(bf16{}, a[k][i], b[t - i], s[k]);
#pragma unroll
  for (int k = 0; k < 2; ++k) c[k] = mma16(bf16{}, a[k][0], b[0], c[k]);
}

struct FusedArgs {
  const void *x, *w, *bias, *gout;
  void* gx;       // [n][k], or null
  float* dw;      // [workgroups][cols][k up to a multiple of four], or null
  float* dbias;   // [workgroups][cols up to a multiple of four], or null
  int64_t n, ldx, ld_gout;
  int k, cols, act;
};

constexpr int kFusedWidth = 64, kFusedWaves = 8;
// 16-bit values of a wave: the planes of sixteen rows of x, then those of d
template <typename T>
constexpr int kFusedStage = 16 * kFusedWidth * (FusedPlanes<T>::kX + FusedPlanes<T>::kD);
template <typename T>
constexpr int kFusedLds = 2 * kFusedWidth * kFusedWidth * 2 * FusedPlanes<T>::kX + kFusedWidth * 4 +
                          kFusedWaves * kFusedStage<T> * 2;

// Whole: both widths are multiples of eight
template <typename Dt, bool Whole>
__global__ void __launch_bounds__(kFusedWaves * 64, 2)
dense_fused_bwd_kernel(FusedArgs g) {
  using T = typename Dt::T;
  constexpr int PX = FusedPlanes<T>::kX, PD = FusedPlanes<T>::kD, KC = kFusedWidth / 32, NC = KC, NF = kFusedWidth / 16;
  extern __shared__ __attribute__((aligned(16))) u16x8 lds[];
  u16x8* wz = lds;                          // [fragment of columns][KC][PX][64]
  u16x8* wx = wz + NF * KC * PX * 64;       // [fragment of k][NC][PX][64]
  float* bias = reinterpret_cast<float*>(wx + NF * NC * PX * 64);
  uint16_t* stage = reinterpret_cast<uint16_t*>(bias + kFusedWidth);
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const T* w = static_cast<const T*>(g.w);
  // fragments of both orders; of the second a lane's eight are a column of the weight
  constexpr int kUnits = 2 * NF * KC / kFusedWaves;  // of a wave, whose loads are in flight together: no branches
  T raw[kUnits][8];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const int u = wave + j * kFusedWaves, f = u % (NF * KC) / KC, i = stream_column(f, lane % 16);
    const int at = u % KC * 32 + lane / 16 * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int n = u >= NF * KC ? at + e : i, k = u >= NF * KC ? i : at + e;
      raw[j][e] = w[(n < g.cols ? n : g.cols - 1) * g.k + (k < g.k ? k : g.k - 1)];
    }
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const int u = wave + j * kFusedWaves, f = u % (NF * KC) / KC, i = stream_column(f, lane % 16);
    const int at = u % KC * 32 + lane / 16 * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int n = u >= NF * KC ? at + e : i, k = u >= NF * KC ? i : at + e;
      v[e] = n < g.cols && k < g.k ? static_cast<float>(raw[j][e]) : 0.f;
    }
    u16x8 p[PX];
    split_planes(v, p);
#pragma unroll
    for (int q = 0; q < PX; ++q) (u >= NF * KC ? wx : wz)[((f * KC + u % KC) * PX + q) * 64 + lane] = p[q];
  }
  if (threadIdx.x < kFusedWidth)
    bias[threadIdx.x] = g.bias && static_cast<int>(threadIdx.x) < g.cols
                            ? static_cast<float>(static_cast<const T*>(g.bias)[threadIdx.x]) : 0.f;
  __syncthreads();
  constexpr int kPlane = 16 * kFusedWidth;
  uint16_t *mine = stage + wave * kFusedStage<T>, *mine_d = mine + PX * kPlane;
  const int64_t tiles = (g.n + 15) / 16, step = static_cast<int64_t>(gridDim.x) * kFusedWaves;
  const int chunk = lane / 16 * 8;
  // rows past the last are zeros
  RowChunk<Dt> rx[KC], rg[NC];
  auto fetch = [&](int64_t t) __attribute__((always_inline)) {
    const int64_t m = t * 16 + lane % 16;
    const bool is = m < g.n;
#pragma unroll
    for (int c = 0; c < KC; ++c)
      load_eight<Dt, Whole>(rx[c], static_cast<const T*>(g.x) + (is ? m : 0) * g.ldx, c * 32 + chunk, g.k, is ? g.k : 0);
#pragma unroll
    for (int c = 0; c < NC; ++c)
      load_eight<Dt, Whole>(rg[c], static_cast<const T*>(g.gout) + (is ? m : 0) * g.ld_gout, c * 32 + chunk, g.cols,
                            is ? g.cols : 0);
  };
  // a plane's eight neighbours of this lane's row, where the transposing reads look for them
  auto put = [&](uint16_t* planes, int plane, int c, const u16x8& p) __attribute__((always_inline)) {
    const int row = lane % 16, slot = (c * 4 + lane / 16) ^ TileLoad<kFusedWidth, 32, 1, true>::fold(row);
    *reinterpret_cast<u16x8*>(planes + plane * kPlane + row * kFusedWidth + slot * 8) = p;
  };
  // sixteen columns of a plane with the rows as their sum
  auto columns = [&](const uint16_t* planes, int plane, int f) __attribute__((always_inline)) {
    const int i = lane % 16, row = lane / 16 * 4 + i / 4, at = f * 2 + i % 4 / 2;
    const uint16_t* p = planes + plane * kPlane + row * kFusedWidth +
                        (at ^ TileLoad<kFusedWidth, 32, 1, true>::fold(row)) * 8 + i % 2 * 4;
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4*)p);
  };
  v4f dw[NF][NF / 2][2];  // [columns][k]
  float db[NC][8];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) dw[i][j / 2][j % 2] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) db[c][i] = 0.f;
  int64_t t = static_cast<int64_t>(wave) * gridDim.x + blockIdx.x;
  if (t < tiles) fetch(t);
  for (; t < tiles; t += step) {
    const int64_t m = t * 16 + lane % 16;
    const bool is = m < g.n;
    u16x8 d[NC][PD];
    {
      u16x8 x[KC][PX];
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        if constexpr (PX == 1 && Whole) {
          x[c][0] = __builtin_bit_cast(u16x8, rx[c].raw[0]);
        } else {
          float v[8];
          eight_values<Dt, Whole>(rx[c], c * 32 + chunk, g.k, is ? g.k : 0, v);
          split_planes(v, x[c]);
        }
#pragma unroll
        for (int q = 0; q < PX; ++q) put(mine, q, c, x[c][q]);
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float v[8];
        eight_values<Dt, Whole>(rg[c], c * 32 + chunk, g.cols, is ? g.cols : 0, v);
        if (g.act != kActNone) {
          v4f z[2] = {}, small[2] = {};
#pragma unroll
          for (int q = 0; q < KC; ++q) {
            u16x8 p[2][PX];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int s = 0; s < PX; ++s) p[j][s] = wz[(((c * 2 + j) * KC + q) * PX + s) * 64 + lane];
            multiply_two(p, x[q], z, small);
          }
          with_act(g.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const v4f b = *reinterpret_cast<const v4f*>(bias + c * 32 + chunk + j * 4);
              if constexpr (PX > 1) z[j] = add_small(z[j], small[j]);
#pragma unroll
              for (int q = 0; q < 4; ++q) v[j * 4 + q] *= dense_slope(act, z[j][q] + b[q]);
            }
          });
        }
        // rows past the last and columns past the width are zeros whatever their slopes: an infinity times the
        // weight's zeros there is NaN, which the next product would spread over the row
        const int real = is ? g.cols - (c * 32 + chunk) : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = (Whole ? 0 : i) < real ? v[i] : 0.f;
          db[c][i] += v[i];
        }
        split_planes(v, d[c]);
      }
    }
    if (g.gx) {
#pragma unroll
      for (int pair = 0; pair < KC; ++pair) {
        v4f a[2] = {}, small[2] = {};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          u16x8 p[2][PX];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int s = 0; s < PX; ++s) p[j][s] = wx[(((pair * 2 + j) * NC + c) * PX + s) * 64 + lane];
          multiply_two(p, d[c], a, small);
        }
        T v[8];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          a[j] = add_small(a[j], small[j]);
#pragma unroll
          for (int q = 0; q < 4; ++q) v[j * 4 + q] = static_cast<T>(a[j][q]);
        }
        const int at = pair * 32 + chunk;
        if (!is || at >= g.k) continue;
        T* to = static_cast<T*>(g.gx) + m * g.k + at;
        if (Whole || at + 8 <= g.k) {
          __builtin_memcpy(to, v, sizeof(v));
        } else {
#pragma unroll
          for (int q = 0; q < 7; ++q)
            if (at + q < g.k) to[q] = v[q];
        }
      }
    }
    if (t + step < tiles) fetch(t + step);
    if (g.dw) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int q = 0; q < PD; ++q) put(mine_d, q, c, d[c][q]);
      asm volatile("" ::: "memory");  // a wave's accesses of LDS are in order
      s16x4 x[NF / 2][2][PX];
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int q = 0; q < PX; ++q) x[f / 2][f % 2][q] = columns(mine, q, f);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        s16x4 p[PD];
#pragma unroll
        for (int q = 0; q < PD; ++q) p[q] = columns(mine_d, q, f);
#pragma unroll
        for (int j = 0; j < NF / 2; ++j) {
          v4f small[2] = {};
          multiply_two(x[j], p, dw[f][j], small);
#pragma unroll
          for (int k = 0; k < 2; ++k) dw[f][j][k] = add_small(dw[f][j][k], small[k]);
        }
      }
      asm volatile("" ::: "memory");
    }
  }
  // the waves' sums: in each turn a wave adds its own to another eighth.  Four columns of a row together, where
  // neither neighbouring rows nor neighbouring columns share a bank (rows one after another: 7 us of turns, now 3).
  auto place = [](int row, int four) { return row * kFusedWidth + (four ^ row % 16) * 4; };
  float* sums = reinterpret_cast<float*>(stage);
  float* bias_sums = sums + kFusedWidth * kFusedWidth;
  const int ld = (g.k + 3) / 4 * 4;
  static_assert(NF * NF == 2 * kFusedWaves && NC * 8 == 2 * kFusedWaves, "two fragments a turn");
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) db[c][i] = lane_sum<16>(db[c][i]);
  for (int turn = 0; turn < kFusedWaves; ++turn) {
    __syncthreads();
    const int eighth = (wave + turn) % kFusedWaves;
#pragma unroll
    for (int e = 0; e < kFusedWaves; ++e) {
      if (e != eighth) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int f = (e * 2 + h) / NF, j = (e * 2 + h) % NF;
        v4f* at = reinterpret_cast<v4f*>(sums + place(f * 16 + lane % 16, j * 4 + lane / 16));
        *at = turn ? *at + dw[f][j / 2][j % 2] : dw[f][j / 2][j % 2];
        float* b = bias_sums + (e * 2 + h) / 8 * 32 + chunk + (e * 2 + h) % 8;
        const float s = db[(e * 2 + h) / 8][(e * 2 + h) % 8];
        if (lane % 16 == 0) *b = turn ? *b + s : s;
      }
    }
  }
  __syncthreads();
  if (g.dw) {
    float* to = g.dw + static_cast<int64_t>(blockIdx.x) * g.cols * ld;
    const int fours = ld / 4;
    for (int i = threadIdx.x; i < g.cols * fours; i += kFusedWaves * 64)
      *reinterpret_cast<v4f*>(to + i * 4) = *reinterpret_cast<const v4f*>(sums + place(i / fours, i % fours));
  }
  if (g.dbias) {
    const int ld_bias = (g.cols + 3) / 4 * 4;
    if (static_cast<int>(threadIdx.x) < g.cols)
      g.dbias[static_cast<int64_t>(blockIdx.x) * ld_bias + threadIdx.x] = bias_sums[threadIdx.x];
  }
}

// Filling the weight in and adding up its gradients takes as long as some rows in
// products of their own.  64 x 64, silu, one MI355X, us here and so:
//           100       300       600      1500      6000      20000      600000
//   f32   15, 16    15, 18    15, 22    16, 21    18, 25    21, 42    147, 331
//   bf16  13, 12    13, 13    13, 14    14, 17    16, 21    17, 24     75, 253
//   f16   14, 13    14, 14    15, 15    16, 19    17, 22    19, 26    102, 319
// and without an activation, whose product in tiles is not done again: f32 100 rows 14,
// 12, 300 rows 14, 14; bf16 600 rows 13, 11, 1500 rows 14, 15.
template <typename T>
bool takes_fused_bwd(int64_t n, int64_t d_in, int64_t d_out) {
  return d_in <= kFusedWidth && d_out <= kFusedWidth && n >= (sizeof(T) == 4 ? 128 : 1024);
}
// one workgroup a unit: its registers take the unit whole
inline int64_t fused_blocks(int64_t n) { return std::min<int64_t>((n + 15) / 16, 256); }

template <typename Dt>
int dense_fused_bwd(const FusedArgs& g, hipStream_t st) {
  using T = typename Dt::T;
  auto* kernel = g.k % 8 == 0 && g.cols % 8 == 0 ? dense_fused_bwd_kernel<Dt, true> : dense_fused_bwd_kernel<Dt, false>;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(fused_blocks(g.n))), dim3(kFusedWaves * 64), kFusedLds<T>, st, g);
  return static_cast<int>(hipGetLastError());
}

}  // namespace kern
}  // namespace segpoly
