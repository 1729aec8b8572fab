// The dense layer of many rows and a small weight, out = act(x W^T + bias) +
// residual: bound by reading x and writing out once.  The weight's planes stay in
// LDS as matrix operands for the kernel's whole time; a wave takes 16 R rows at a
// time, its x from memory straight into the registers of the matrix instructions
// (the next rows' loads in flight meanwhile, float32 split into its planes in
// registers), and goes over the columns 32 at a time.  No barrier after the
// weight has been filled in, where the tiles bring both operands to LDS step by step,
// of which short sums have one to four.  Columns that do not fit in LDS, and those of
// few rows, are shared out over workgroups.
// The times of both forms stand at takes_stream.
// A pair of column fragments holds the columns in an order that leaves a lane
// eight neighbouring ones of its row, 16 or 32 bytes to store together.
#pragma once
#include <algorithm>

#include "gemm_staged.hpp"

namespace segpoly {
namespace kern {

struct StreamArgs {
  const void *x, *w, *bias, *res;
  void* out;
  int64_t n, ldx, ld_res, ldo;
  int k, cols, act;
  int pairs;  // of column fragments, of a workgroup: (x, y) takes the y-th part of the columns
};

// columns of a row of fragments: fragment pair * 2 + j, row i of the instruction
__device__ __forceinline__ int stream_column(int fragment, int i) {
  return fragment / 2 * 32 + i / 4 * 8 + fragment % 2 * 4 + i % 4;
}

// Workgroups that a unit's registers hold: two of at most 128 a lane.
template <typename Dt>
constexpr int stream_held(int chunks, bool res, bool whole) {
  return (Dt::kPlanes > 1 ? chunks == 1 && (whole || !res) : chunks <= 2 || whole) ? 2 : 1;
}

// KC: 32 k each of a row.  Loads return in order: the residual's would wait for the
// next rows' if those were on their way already, so with it they are fetched later.
// Whole: x's width is a multiple of 16 bytes, the output's of eight columns.
template <typename Dt, int KC, int R, bool Res, bool Whole>
__global__ void __launch_bounds__(512, 2 * stream_held<Dt>(KC, Res, Whole))
dense_stream_kernel(StreamArgs g) {
  using T = typename Dt::T;
  constexpr int P = Dt::kPlanes;
  extern __shared__ __attribute__((aligned(16))) u16x8 weight[];  // [fragment][KC][P][64]
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), waves = blockDim.x / 64;
  const int pair0 = blockIdx.y * g.pairs, all = (g.cols + 31) / 32;
  const int pairs = all - pair0 < g.pairs ? all - pair0 : g.pairs, units = pairs * 2 * KC;
  v4f* bias = reinterpret_cast<v4f*>(weight + units * P * 64);  // of four columns each
  constexpr int kFill = 4;  // in flight together
  for (int u0 = wave * kFill; u0 < units; u0 += waves * kFill) {
    RowChunk<Dt> c[kFill];
    int limit[kFill];
#pragma unroll
    for (int i = 0; i < kFill; ++i) {
      const int u = u0 + i, n = pair0 * 32 + stream_column(u / KC, lane % 16);
      limit[i] = u < units && n < g.cols ? g.k : 0;
      load_eight<Dt, false>(c[i], static_cast<const T*>(g.w) + static_cast<int64_t>(limit[i] ? n : 0) * g.k,
                            u % KC * 32 + lane / 16 * 8, g.k, limit[i]);
    }
#pragma unroll
    for (int i = 0; i < kFill; ++i) {
      if (u0 + i >= units) continue;
      u16x8 p[P];
      chunk_planes<Dt, false>(c[i], (u0 + i) % KC * 32 + lane / 16 * 8, g.k, limit[i], p);
#pragma unroll
      for (int q = 0; q < P; ++q) weight[((u0 + i) * P + q) * 64 + lane] = p[q];
    }
  }
  for (int i = threadIdx.x; i < pairs * 8; i += blockDim.x)
    bias[i] = g.bias ? load_four(static_cast<const T*>(g.bias), pair0 * 32 + i * 4, g.cols) : v4f{0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  const int64_t tiles = (g.n + 16 * R - 1) / (16 * R), step = static_cast<int64_t>(gridDim.x) * waves;
  RowChunk<Dt> raw[R][KC];
  auto fetch = [&](int64_t t) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      int64_t m = t * (16 * R) + r * 16 + lane % 16;
      m = m < g.n ? m : g.n - 1;
#pragma unroll
      for (int c = 0; c < KC; ++c)
        load_eight<Dt, Whole>(raw[r][c], static_cast<const T*>(g.x) + m * g.ldx, c * 32 + lane / 16 * 8, g.k, g.k);
    }
  };
  int64_t t = static_cast<int64_t>(wave) * gridDim.x + blockIdx.x;
  if (t < tiles) fetch(t);
  for (; t < tiles; t += step) {
    u16x8 x[R][KC][P];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < KC; ++c) chunk_planes<Dt, Whole>(raw[r][c], c * 32 + lane / 16 * 8, g.k, g.k, x[r][c]);
    if (!Res && t + step < tiles) fetch(t + step);
    for (int pair = 0; pair < pairs; ++pair) {
      const int n = (pair0 + pair) * 32 + lane / 16 * 8;
      v4f res[R][2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          res[r][j] = v4f{0.f, 0.f, 0.f, 0.f};
          if constexpr (Res) {
            int64_t m = t * (16 * R) + r * 16 + lane % 16;
            m = m < g.n ? m : g.n - 1;
            res[r][j] = load_four(static_cast<const T*>(g.res) + m * g.ld_res, n + j * 4, g.cols);
          }
        }
      v4f acc[R][2], small[R][2];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[r][j] = small[r][j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        u16x8 w[2][P];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int q = 0; q < P; ++q) w[j][q] = weight[(((pair * 2 + j) * KC + c) * P + q) * 64 + lane];
        constexpr int kProducts = P == 1 ? 1 : 6;
#pragma unroll
        for (int s = 0; s < kProducts; ++s)
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if constexpr (P == 1) {
                acc[r][j] = mma16(typename Dt::E{}, w[j][0], x[r][c][0], acc[r][j]);
              } else {
                v4f& a = s < kProducts - 1 ? small[r][j] : acc[r][j];
                a = mma16(typename Dt::E{}, w[j][kPairs3[s][1]], x[r][c][kPairs3[s][0]], a);
              }
            }
      }
      with_act(g.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          T v[8];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const v4f b = bias[pair * 8 + lane / 16 * 2 + j];
            if constexpr (P > 1) acc[r][j] = add_small(acc[r][j], small[r][j]);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              v[j * 4 + q] = static_cast<T>(dense_act(act, acc[r][j][q] + b[q]) + res[r][j][q]);
          }
          const int64_t m = t * (16 * R) + r * 16 + lane % 16;
          if (m >= g.n || n >= g.cols) continue;
          T* to = static_cast<T*>(g.out) + m * g.ldo + n;
          if (Whole || n + 8 <= g.cols) {
            __builtin_memcpy(to, v, sizeof(v));
          } else {
#pragma unroll
            for (int q = 0; q < 7; ++q)
              if (n + q < g.cols) to[q] = v[q];
          }
        }
      });
    }
    if (Res && t + step < tiles) fetch(t + step);
  }
}

// 32 k each of a row that stay in registers, or 0 for rows that do not.
template <typename Dt>
int stream_chunks(int64_t d_in) {
  constexpr int kMost = Dt::kPlanes == 1 ? 8 : 4;
  for (int chunks = 1; chunks <= kMost; chunks *= 2)
    if (d_in <= chunks * 32) return chunks;
  return 0;
}

// Which calls of more rows than gemm_rows.hpp's take this form.  One MI355X, us here and in tiles, silu, operands in
// the last-level cache (from memory both take longer, to the same sides):
//   float32                     bf16, whole chunks          bf16, widths of x or out that are none
//   1000 x 64 x 64    5.4, 5.8   1000 x 64 x 64    3.7, 4.4   400 x 255 x 256    5.9, 7.6   20000 x 64 x 250    9.3,  11
//   200 x 128 x 128   5.5, 7.7   200 x 128 x 128   4.0, 4.5   2000 x 255 x 1024   19,  10   100000 x 64 x 1023  109,  81
//   5000 x 64 x 256   7.8, 7.3   2000 x 64 x 1024  5.1, 5.8   20000 x 255 x 64    13,  16   1000 x 192 x 1023   6.6, 5.6
//   20000 x 64 x 64   7.7, 7.2   20000 x 128 x 128 6.9, 6.9   100000 x 255 x 16   26,  37   5000 x 256 x 250    7.6, 6.8
//   20000 x 128 x 128  13,  13   20162 x 64 x 896   15,  21   154122 x 243 x 124  42,  63   20000 x 250 x 1020   31,  39
//   20162 x 64 x 896   28,  38   600000 x 64 x 64   28,  50   2000 x 127 x 1024   12, 8.5   100000 x 62 x 255    32,  38
//   600000 x 64 x 64   64,  90   2000 x 256 x 1024 8.5, 6.9   100000 x 127 x 256  52,  41   100000 x 62 x 1024  130,  89
//   100000 x 127 x 256 58,  84   20000 x 256 x 256  13,  12   100000 x 63 x 1024 139,  89   113893 x 19 x 134    22,  36
//   2000 x 64 x 1022   11, 7.8   50000 x 256 x 256  22,  21
//   100000 x 64 x 63   23,  19   300 x 256 x 1024  5.0, 5.2
//   82491 x 61 x 27    12,  17   200000 x 256 x 256 51,  64
// 16-bit rows of x that are no whole chunks are copied before the tiles take them, 3 us and more; those of odd width, at
// any two bytes, cost the streamed loads and stores more than that where there are many.
template <typename Dt>
bool takes_stream(int64_t n, int64_t d_in, int64_t d_out) {
  const int64_t chunks = stream_chunks<Dt>(d_in), size = n * d_out;
  if (chunks == 0) return false;
  if (Dt::kPlanes > 1) return !(chunks <= 2 && d_out % 8 != 0 && d_out > 32 && size >= 1 << 19 && size < 1 << 24);
  if (d_in % 8 == 0 && d_out % 8 == 0)  // all but whole steps of the tiles' sums
    return !(d_in > 128 && d_in % 64 == 0 && d_out >= 256 && size >= 1 << 20 && size <= 3 << 22);
  if (d_out <= (n >= 1 << 16 ? 192 : 64)) return true;
  if (d_in % 8 != 0 && d_in % 2 == 0) return size < 1 << 25;
  return size < (chunks <= 4 ? 1 << 23 : 1 << 20);
}

// Bytes of LDS of 32 columns of the weight and their bias.
template <typename Dt>
int64_t stream_pair_bytes(int chunks) { return 32 * (chunks * Dt::kPlanes * 64 + 4); }

template <typename Dt, int KC, int R>
int stream_launch(StreamArgs g, hipStream_t st) {
  const int64_t tiles = (g.n + 16 * R - 1) / (16 * R), all = (g.cols + 31) / 32;
  // two workgroups share a unit's LDS, where its registers hold two (where they do not, a second round of them would
  // fill the weight in again: 5000 x 64 x 64 float32 7.5 us, now 5.8; 20000 x 64 x 64 9.6, 7.7); fewer columns each
  // until eight waves a unit have work (20162 x 64 x 896 bf16: 15 us, 19 with four)
  const bool whole = g.k % Chunk<typename Dt::T>::kN == 0 && g.cols % 8 == 0;
  int64_t pairs = std::min(all, std::max<int64_t>(1, 80 * 1024 / stream_pair_bytes<Dt>(KC)));
  while (pairs > 1 && tiles * ((all + pairs - 1) / pairs) < 2048) pairs = (pairs + 1) / 2;
  const int64_t groups = (all + pairs - 1) / pairs;
  g.pairs = static_cast<int>((all + groups - 1) / groups);
  const int64_t blocks = std::min<int64_t>(tiles, std::max<int64_t>(1, 256 * stream_held<Dt>(KC, g.res, whole) / groups));
  auto* kernel = whole ? (g.res ? dense_stream_kernel<Dt, KC, R, true, true> : dense_stream_kernel<Dt, KC, R, false, true>)
                       : (g.res ? dense_stream_kernel<Dt, KC, R, true, false> : dense_stream_kernel<Dt, KC, R, false, false>);
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(groups)), dim3(512),
                     g.pairs * stream_pair_bytes<Dt>(KC), st, g);
  return static_cast<int>(hipGetLastError());
}

template <typename Dt>
int dense_stream(const StreamArgs& g, hipStream_t st) {
  constexpr int kFour = Dt::kPlanes == 1 ? 2 : 1;
  const int chunks = stream_chunks<Dt>(g.k);
  if (chunks == 1) return stream_launch<Dt, 1, 2>(g, st);
  if (chunks == 2) return stream_launch<Dt, 2, 2>(g, st);
  if constexpr (Dt::kPlanes == 1) {
    if (chunks == 8) return stream_launch<Dt, 8, 1>(g, st);
  }
  return stream_launch<Dt, 4, kFour>(g, st);
}

}  // namespace kern
}  // namespace segpoly
