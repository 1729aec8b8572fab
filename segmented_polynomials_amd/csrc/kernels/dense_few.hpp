// The dense layer of few rows, and the slope of products whose long sums are shared
// out.
//   forward   at most sixteen rows (32 of some widths): gemm_rows.hpp; a long sum for few columns is
//             shared out over workgroups
//   backward  the product again in the same form, its slope in a launch of its own that
//             leaves d and the bias's gradient; then, of at most four rows, one pass over
//             the weight for both others: a thread has some neighbouring columns k, goes
//             down rows o of the weight, and has for each w[o][k]
//               dx[m][k] += d[m][o] w[o][k],     dw[o][k] = sum over m of d[m][o] x[m][k]
// Bound by reading the weight twice (the second time from the last-level cache where it
// fits) and writing its gradient once; on the vector units, as a matrix instruction
// would work on empty rows and need the weight transposed.  One MI355X, us here and in
// tiles, silu (floor): 1 x 8192 x 8192 f32 195, 465 (107), bf16 91, 109 (54); 2 x 4096 x
// 4096 f32 58, 180 (27), bf16 37, 49 (13); 3 x 1024 x 4096 bf16 20, 23.  Of eight rows the
// sums do not leave registers for the weight's loads: 4096 x 4096 bf16 120, 49.
#pragma once
#include <algorithm>

#include "gemm_plan.hpp"
#include "gemm_rows.hpp"

namespace segpoly {
namespace kern {

// d = g act'(sum of the shares + bias), 64 rows by 32 columns a workgroup: eight
// neighbours of a row each thread.
struct SlopeArgs {
  const float* from;  // [splits][m][ld], or null: no product (no activation)
  int64_t split_stride, m, n, ld;
  int splits, act;
  const void *bias, *gout;
  int64_t ld_gout;
  void* d;            // [m][ld_d]: float32, or (16-bit rows of products' operands) T
  int64_t ld_d;
  int* exponents;     // float16 operands: of 64 rows and 32 columns
  int64_t e_ld;
  float* column_sums; // [blocks of 64 rows][n up to a multiple of four], or null
  void* gbias;        // with one block of rows: the sums themselves, T, or null
};
template <typename Dt, bool FloatD>
__global__ void __launch_bounds__(256)
dense_slope_kernel(SlopeArgs g) {
  using T = typename Dt::T;
  __shared__ float lds[64][33];
  __shared__ float top[4];
  const int row = threadIdx.x / 4, part = threadIdx.x % 4 * 8;
  const int64_t m = static_cast<int64_t>(blockIdx.y) * 64 + row, n = static_cast<int64_t>(blockIdx.x) * 32 + part;
  float d[8];
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    v4f z = {0.f, 0.f, 0.f, 0.f}, r = z, bias = z;
    if (m < g.m && n + i < g.n) {
      r = load_four(static_cast<const T*>(g.gout) + m * g.ld_gout, n + i, g.n);
      if (g.bias) bias = load_four(static_cast<const T*>(g.bias), n + i, g.n);
      if (g.from) {
        const float* from = g.from + m * g.ld + n + i;
#pragma unroll 8
        for (int k = 0; k < g.splits; ++k) z += *reinterpret_cast<const v4f*>(from + k * g.split_stride);
      }
    }
    with_act(g.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < 4; ++q) d[i + q] = r[q] * dense_slope(act, z[q] + bias[q]);
    });
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      d[i + q] = m < g.m && n + i + q < g.n ? d[i + q] : 0.f;
      lds[row][part + i + q] = d[i + q];
    }
  }
  if constexpr (Dt::kScaled && !FloatD) {
    float largest = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) largest = __builtin_fmaxf(largest, finite_abs(d[i]));
    largest = lane_max<64>(largest);
    if (threadIdx.x % 64 == 0) top[threadIdx.x / 64] = largest;
  }
  __syncthreads();
  if constexpr (Dt::kScaled && !FloatD) {
    const int e = block_exponent(__builtin_fmaxf(__builtin_fmaxf(top[0], top[1]), __builtin_fmaxf(top[2], top[3])));
    const float scale = block_scale(e);
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] *= scale;
    if (threadIdx.x == 0) g.exponents[blockIdx.y * g.e_ld + blockIdx.x] = e;
  }
  // rows of the products' operands are read in 16-byte chunks, up to a multiple of eight
  if (m < g.m && n < g.n) {
    if constexpr (FloatD) {
      float* to = static_cast<float*>(g.d) + m * g.ld_d + n;
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        if (n + i < g.n) __builtin_memcpy(to + i, d + i, 16);  // ld_d is a multiple of four
    } else {
      T v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = static_cast<T>(d[i]);
      __builtin_memcpy(static_cast<T*>(g.d) + m * g.ld_d + n, v, 16);
    }
  }
  if (threadIdx.x < 32) {
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float s = 0.f;
#pragma unroll 16
    for (int r = 0; r < 64; ++r) s += lds[r][threadIdx.x];
    if (c < g.n) {
      if (g.column_sums) g.column_sums[blockIdx.y * ((g.n + 3) / 4 * 4) + c] = s;
      if (g.gbias) static_cast<T*>(g.gbias)[c] = static_cast<T>(s);
    }
  }
}
template <typename Dt, bool FloatD>
int dense_slope(const SlopeArgs& g, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>((g.n + 31) / 32), static_cast<unsigned>((g.m + 63) / 64));
  hipLaunchKernelGGL((dense_slope_kernel<Dt, FloatD>), grid, dim3(256), 0, st, g);
  return static_cast<int>(hipGetLastError());
}

// ------------------------------------------------------------ forward

// k of a workgroup's share: of a sum long enough for several, of columns too few to fill
// the card.  5 rows of 8192 x 64, one MI355X, us shared out and not: f32 8.3, 33; bf16 6.1, 13
inline int64_t few_share(int64_t d_in, int64_t d_out) {
  const int64_t groups = (d_out + 15) / 16, shares = groups > 64 ? 1 : std::min<int64_t>(256 / groups, d_in / 512);
  return shares < 2 ? round_up(d_in, 64) : round_up((d_in + shares - 1) / shares, 64);
}
inline int64_t few_shares(int64_t d_in, int64_t d_out) {
  const int64_t share = few_share(d_in, d_out);
  return (d_in + share - 1) / share;
}

// ------------------------------------------------------------ backward

struct FewArgs {
  const void *x, *w;
  const float* d;         // [n][ld_d]
  float* dx;              // [rows of workgroups][n][ld_dx], or null
  void* dw;               // [d_out][d_in], or null
  int64_t d_in, d_out, ldx, ld_d, ld_dx;
  int n, rows, lanes;     // weight rows of a workgroup; threads along k (a power of two)
};

// M: rows held in registers, at most four; V columns a thread
template <typename T, int M, int V>
__global__ void __launch_bounds__(256, 4)
dense_few_bwd_kernel(FewArgs g) {
  constexpr int kPart = 64;                       // weight rows whose d is in LDS
  constexpr int kFlight = 4;                      // weight rows in flight
  __shared__ __attribute__((aligned(16))) float ld[kPart][M];
  __shared__ float lx[M][256 * V];
  const int lane = threadIdx.x % g.lanes, down = threadIdx.x / g.lanes, step = 256 / g.lanes;
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * g.lanes + lane) * V;
  const int64_t o0 = static_cast<int64_t>(blockIdx.y) * g.rows, o1 = o0 + g.rows < g.d_out ? o0 + g.rows : g.d_out;
  const bool here = c < g.d_in;
  struct Values {
    T t[V];
  };
  // V neighbours, those past the row's end zeros
  auto load = [&](const T* row, Values& v) __attribute__((always_inline)) {
    if (c + V <= g.d_in) {
      __builtin_memcpy(v.t, row + c, sizeof(v.t));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v.t[i] = c + i < g.d_in ? row[c + i] : T(0.f);
    }
  };
  float x[M][V], dx[M][V];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    Values v{};
    if (g.dw && here && m < g.n) load(static_cast<const T*>(g.x) + m * g.ldx, v);
#pragma unroll
    for (int i = 0; i < V; ++i) x[m][i] = static_cast<float>(v.t[i]), dx[m][i] = 0.f;
  }
  for (int64_t part = o0; part < o1; part += kPart) {
    __syncthreads();
    for (int i = threadIdx.x; i < kPart * M; i += 256) {
      const int m = i / kPart, o = i % kPart;
      ld[o][m] = m < g.n && part + o < o1 ? g.d[m * g.ld_d + part + o] : 0.f;
    }
    __syncthreads();
    if (!here) continue;
    const int most = o1 - part < kPart ? static_cast<int>(o1 - part) : kPart;
    for (int first = down; first < most; first += step * kFlight) {
      Values raw[kFlight];
      if (g.dx) {
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
          const int o = first + u * step < most ? first + u * step : first;
          load(static_cast<const T*>(g.w) + (part + o) * g.d_in, raw[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int o = first + u * step;
        if (o >= most) break;
        float s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = 0.f;
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const float d = ld[o][m];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if (g.dx) dx[m][i] += d * static_cast<float>(raw[u].t[i]);
            s[i] += d * x[m][i];
          }
        }
        if (g.dw) {
          T t[V];
#pragma unroll
          for (int i = 0; i < V; ++i) t[i] = static_cast<T>(s[i]);
          T* to = static_cast<T*>(g.dw) + (part + o) * g.d_in + c;
          if (c + V <= g.d_in) {
            __builtin_memcpy(to, t, sizeof(t));
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
              if (c + i < g.d_in) to[i] = t[i];
          }
        }
      }
    }
  }
  if (!g.dx) return;
  // the sums of the threads of a column, in order
  __syncthreads();
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int i = 0; i < V; ++i) lx[m][threadIdx.x * V + i] = dx[m][i];
  __syncthreads();
  const int columns = g.lanes * V;
  for (int k = threadIdx.x; k < g.n * columns; k += 256) {
    const int m = k / columns, i = k % columns;
    float s = 0.f;
    for (int q = 0; q < step; ++q) s += lx[m][q * columns + i];
    const int64_t col = static_cast<int64_t>(blockIdx.x) * columns + i;
    if (col < g.ld_dx) g.dx[(static_cast<int64_t>(blockIdx.y) * g.n + m) * g.ld_dx + col] = s;
  }
}

// Threads along k and workgroups down the weight's rows: four workgroups a unit.
struct FewPlan {
  int lanes;
  int64_t columns, rows, parts;
};
template <typename T>
FewPlan few_plan(int64_t n, int64_t d_in, int64_t d_out) {
  const int64_t v = n > 2 ? 4 : Chunk<T>::kN;  // as below
  FewPlan p{16, 0, 0, 0};
  while (p.lanes < 64 && p.lanes * v < d_in) p.lanes *= 2;
  p.columns = (d_in + p.lanes * v - 1) / (p.lanes * v);
  const int64_t most = std::max<int64_t>(1, 1024 / p.columns);
  p.rows = round_up(std::max<int64_t>((d_out + most - 1) / most, 256 / p.lanes * 4), 4);
  p.parts = (d_out + p.rows - 1) / p.rows;
  return p;
}

template <typename T>
int dense_few_bwd(const FewArgs& g, const FewPlan& p, hipStream_t st) {
  constexpr int V = Chunk<T>::kN;
  auto* kernel = g.n == 1 ? dense_few_bwd_kernel<T, 1, V> : g.n == 2 ? dense_few_bwd_kernel<T, 2, V>
                                                                     : dense_few_bwd_kernel<T, 4, 4>;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(p.columns), static_cast<unsigned>(p.parts)), dim3(256), 0, st, g);
  return static_cast<int>(hipGetLastError());
}

}  // namespace kern
}  // namespace segpoly
