// Rows sorted by expert and back, with weights applied, and the gradients:
//   sort      place[e] of entry e = (row, choice): its slot in the stable order by
//             expert; entries without an expert come last, from slot `total` on
//   dispatch  xs[place[i, j]] = x[i]                        (zero rows from `total` on)
//   its gradient, and combine
//             out[i] = residual[i] + sum over j of w[i, j] ys[place[i, j]]
//   combine's gradient
//             gys[place[i, j]] = w[i, j] g[i],   gw[i, j] = <g[i], ys[place[i, j]]>
// The sort is a counting sort without atomics on memory.  A wave ranks its entries 64 at
// a time: one ballot per bit of the expert's number leaves each lane the mask
// of the lanes with its expert; counts of a wave stay in LDS.  One workgroup
// orders short lists in one launch; longer ones take one launch that counts and one
// that places, between them a third that adds the counts up where many
// workgroups would each read too many of them.
// The row operators run along the rows i, not the slots: a row of x, g or out
// crosses memory once, whatever k is, and only the k rows by slot are scattered.
// All are bound by memory: one MI355X, 16384 rows of 2048 bf16 to eight experts each
// 116 us, 4.9 TB/s (the sort before it 16); the gradient of combining 16384 such rows of
// four choices 129 us, 4.7 TB/s.  Sorts by length stand at expert_sort_plan.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../channel_ops.hpp"
#include "channel_types.hpp"

namespace segpoly {
namespace kern {

// ------------------------------------------------------------ the sort

enum { kSortAll = 0, kSortCount = 1, kSortPlace = 2 };

struct SortLds {
  uint16_t before[kSortWaves][kMaxExperts + 2];  // a wave's count; then the count of the waves before it
  int base[kMaxExperts + 1];
  int mine[kMaxExperts + 1];  // of the workgroups before
  int wave_sum[kSortWaves];
};

// base[e] = sum of base[f] over f < e, for the workgroup's threads
__device__ __forceinline__ void scan_base(SortLds& l, int classes) {
  const int threads = blockDim.x, lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int per = (classes + threads - 1) / threads, from = threadIdx.x * per;
  int sum = 0;
  for (int i = from; i < from + per && i < classes; ++i) sum += l.base[i];
  int up = sum;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(up, d);
    up += lane >= d ? o : 0;
  }
  if (lane == 63) l.wave_sum[wave] = up;
  __syncthreads();
  int run = up - sum;
  for (int w = 0; w < wave; ++w) run += l.wave_sum[w];
  for (int i = from; i < from + per && i < classes; ++i) {
    const int c = l.base[i];
    l.base[i] = run;
    run += c;
  }
}

// C: 64 entries each of a wave's turns.  Counts: [blocks][classes]; `summed`: a
// row holds the counts before its workgroup, and a last row the totals.
template <typename I, int C, int Mode>
__global__ void __launch_bounds__(kSortWaves * 64)
expert_sort_kernel(ExpertSortArgs a, int blocks, int summed) {
  __shared__ SortLds l;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, waves = blockDim.x / 64;
  const int classes = a.num + 1;  // the last: no expert
  for (int i = threadIdx.x; i < waves * classes; i += blockDim.x) l.before[i / classes][i % classes] = 0;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * waves + wave) * (64 * C) + lane;
  int expert[C], rank[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t at = first + c * 64;
    I e = -1;
    if (at < a.entries) e = static_cast<const I*>(a.experts)[at];
    expert[c] = e >= 0 && e < a.num ? static_cast<int>(e) : a.num;
  }
  if constexpr (Mode == kSortPlace) {
    for (int e = threadIdx.x; e < classes; e += blockDim.x) {
      l.base[e] = summed ? a.counts[static_cast<int64_t>(blocks) * classes + e] : 0;
      l.mine[e] = summed ? a.counts[static_cast<int64_t>(blockIdx.x) * classes + e] : 0;
    }
  }
  __syncthreads();
  if constexpr (Mode == kSortPlace) {
    // few workgroups' counts: all threads share them out (whole numbers: any order)
    if (!summed) {
#pragma unroll 4
      for (int i = threadIdx.x; i < blocks * classes; i += blockDim.x) {
        const int e = i % classes, c = a.counts[i];
        if (c == 0) continue;
        atomicAdd(&l.base[e], c);
        if (i / classes < static_cast<int>(blockIdx.x)) atomicAdd(&l.mine[e], c);
      }
    }
  }
  const int bits = 32 - __clz(a.num);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const bool is = first + c * 64 < a.entries;
    uint64_t mask = __ballot(is);
    for (int b = 0; b < bits; ++b) {
      const bool one = expert[c] >> b & 1;
      const uint64_t ones = __ballot(one);
      mask &= one ? ones : ~ones;
    }
    const int below = __popcll(mask & ((uint64_t{1} << lane) - 1)), all = __popcll(mask);
    int before = 0;
    if (is) before = l.before[wave][expert[c]];
    rank[c] = before + below;
    asm volatile("" ::: "memory");  // a wave's accesses of LDS are in order
    if (is && below == all - 1) l.before[wave][expert[c]] = static_cast<uint16_t>(before + all);
    asm volatile("" ::: "memory");
  }
  __syncthreads();
  for (int e = threadIdx.x; e < classes; e += blockDim.x) {
    int run = 0;
    for (int w = 0; w < waves; ++w) {
      const int c = l.before[w][e];
      l.before[w][e] = static_cast<uint16_t>(run);
      run += c;
    }
    if constexpr (Mode == kSortCount) a.counts[static_cast<int64_t>(blockIdx.x) * classes + e] = run;
    if constexpr (Mode == kSortAll) l.base[e] = run;
  }
  if constexpr (Mode == kSortCount) return;
  __syncthreads();
  scan_base(l, classes);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e < classes; e += blockDim.x) a.offsets[e] = l.base[e];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t at = first + c * 64;
    if (at >= a.entries) continue;
    int slot = l.base[expert[c]] + l.before[wave][expert[c]] + rank[c];
    if constexpr (Mode == kSortPlace) slot += l.mine[expert[c]];
    if (slot >= a.entries) continue;  // not reached while the list stays as it was counted
    a.place[at] = slot;
    a.order[slot] = static_cast<int>(at);
    a.ids[slot] = expert[c] < a.num ? expert[c] : -1;
  }
}

// Each class's counts become the counts before; the totals go to a last row.  A
// workgroup of 1024 takes 32 classes by 32 runs of the rows.
__global__ void __launch_bounds__(1024)
expert_counts_kernel(int* counts, int blocks, int classes) {
  __shared__ int sums[32][33];
  const int e = blockIdx.x * 32 + threadIdx.x % 32, run = threadIdx.x / 32;
  const int per = (blocks + 31) / 32, from = run * per, to = from + per < blocks ? from + per : blocks;
  int s = 0;
  if (e < classes) {
#pragma unroll 8
    for (int b = from; b < to; ++b) s += counts[static_cast<int64_t>(b) * classes + e];
  }
  sums[run][threadIdx.x % 32] = s;
  __syncthreads();
  if (e >= classes) return;
  int before = 0;
  for (int r = 0; r < run; ++r) before += sums[r][threadIdx.x % 32];
  for (int b = from; b < to; ++b) {
    int* at = counts + static_cast<int64_t>(b) * classes + e;
    const int c = *at;
    *at = before;
    before += c;
  }
  if (run == 31) counts[static_cast<int64_t>(blocks) * classes + e] = before;
}

template <typename I, int C>
int expert_sort_launch(const ExpertSortArgs& a, const ExpertSortPlan& p) {
  const hipStream_t st = static_cast<hipStream_t>(a.stream);
  const dim3 grid(static_cast<unsigned>(p.blocks)), threads(p.waves * 64);
  const int blocks = static_cast<int>(p.blocks), classes = a.num + 1;
  if (p.blocks == 1) {
    hipLaunchKernelGGL((expert_sort_kernel<I, C, kSortAll>), grid, threads, 0, st, a, 1, 0);
    return static_cast<int>(hipGetLastError());
  }
  hipLaunchKernelGGL((expert_sort_kernel<I, C, kSortCount>), grid, threads, 0, st, a, blocks, 0);
  if (const hipError_t e = hipGetLastError()) return static_cast<int>(e);
  // Unsummed, every workgroup reads all counts.  One MI355X, us so and with the third launch, by counts (blocks x
  // classes): 3835 10.1, 11.5; 8320 12.3, 13.3 and 19.6, 20.6; 16512 15.8, 14.0 and 24.2, 22.4; 65792 36.8, 17.4
  const bool sum = blocks * classes > 10240;
  if (sum) {
    hipLaunchKernelGGL(expert_counts_kernel, dim3(static_cast<unsigned>((classes + 31) / 32)), dim3(1024), 0, st, a.counts,
                       blocks, classes);
    if (const hipError_t e = hipGetLastError()) return static_cast<int>(e);
  }
  hipLaunchKernelGGL((expert_sort_kernel<I, C, kSortPlace>), grid, threads, 0, st, a, blocks, static_cast<int>(sum));
  return static_cast<int>(hipGetLastError());
}

// ------------------------------------------------------------ rows

constexpr int kRowChunks = 2;  // of a thread, in flight together

// The chunks of the rows one after another, kRowChunks a thread, 256 apart.
template <typename F>
__device__ __forceinline__ void for_chunks(int64_t n, uint32_t row_chunks, int64_t blocks, F&& body) {
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t first = b * (256 * kRowChunks), row0 = first / row_chunks;
    const uint32_t chunk0 = static_cast<uint32_t>(first % row_chunks) + threadIdx.x;
    int64_t row[kRowChunks];
    int chunk[kRowChunks];
#pragma unroll
    for (int u = 0; u < kRowChunks; ++u) {
      const uint32_t at = chunk0 + u * 256, r = at / row_chunks;
      row[u] = row0 + r;
      chunk[u] = static_cast<int>(at - r * row_chunks);
      if (row[u] >= n) row[u] = -1;
    }
    body(row, chunk);
  }
}

template <typename T>
__global__ void __launch_bounds__(256)
expert_dispatch_kernel(ExpertRowsArgs a, uint32_t row_chunks, int64_t blocks) {
  constexpr int V = Chunk<T>::kN, U = kRowChunks, J = 4;
  const int dim = static_cast<int>(a.dim), k = static_cast<int>(a.k);
  const uint32_t slots = static_cast<uint32_t>(a.n * a.k);
  const uint32_t total = static_cast<uint32_t>(*a.total);
  for_chunks(a.n, row_chunks, blocks, [&](const int64_t(&row)[U], const int(&chunk)[U]) {
    u32x4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      x[u] = load_raw(static_cast<const T*>(a.x) + (row[u] < 0 ? 0 : row[u]) * a.x_stride, row[u] < 0 ? dim : chunk[u] * V,
                      dim);
    for (int j0 = 0; j0 < k; j0 += J) {
      uint32_t slot[U][J];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < J; ++j)
          slot[u][j] = row[u] >= 0 && j0 + j < k ? static_cast<uint32_t>(a.place[row[u] * k + j0 + j]) : slots;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const u32x4 v = settle_chunk<T>(x[u], row[u] < 0 ? dim : chunk[u] * V, dim), zero = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (slot[u][j] < slots)
            store_raw(static_cast<T*>(a.out) + slot[u][j] * a.dim, chunk[u] * V, dim, slot[u][j] < total ? v : zero);
      }
    }
  });
}

template <typename T, bool Weights>
__global__ void __launch_bounds__(256)
expert_combine_kernel(ExpertRowsArgs a, uint32_t row_chunks, int64_t blocks) {
  constexpr int V = Chunk<T>::kN, U = kRowChunks, J = 4;
  const int dim = static_cast<int>(a.dim), k = static_cast<int>(a.k);
  const uint32_t slots = static_cast<uint32_t>(a.n * a.k);
  uint32_t total = static_cast<uint32_t>(*a.total);
  total = total < slots ? total : slots;
  for_chunks(a.n, row_chunks, blocks, [&](const int64_t(&row)[U], const int(&chunk)[U]) {
    float sum[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < V; ++i) sum[u][i] = 0.f;
    for (int j0 = 0; j0 < k; j0 += J) {
      uint32_t slot[U][J];
      float w[U][J];
      u32x4 y[U][J];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const bool is = row[u] >= 0 && j0 + j < k;
          slot[u][j] = is ? static_cast<uint32_t>(a.place[row[u] * k + j0 + j]) : slots;
          if constexpr (Weights) w[u][j] = is ? a.weights[row[u] * k + j0 + j] : 0.f;
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const bool is = slot[u][j] < total;
          y[u][j] = load_raw(static_cast<const T*>(a.ys) + (is ? slot[u][j] : 0) * a.ys_stride, is ? chunk[u] * V : dim, dim);
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          float v[V];
          unpack_chunk<T>(y[u][j], chunk[u] * V, dim, v);
          if (slot[u][j] < total)
#pragma unroll
            for (int i = 0; i < V; ++i) sum[u][i] += Weights ? w[u][j] * v[i] : v[i];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (row[u] < 0) continue;
      if (a.residual) {
        float r[V];
        load_chunk(static_cast<const T*>(a.residual) + row[u] * a.residual_stride, chunk[u] * V, dim, r);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[u][i] += r[i];
      }
      store_chunk(static_cast<T*>(a.out) + row[u] * a.out_stride, chunk[u] * V, dim, sum[u]);
    }
  });
}

// G lanes hold a row; eight choices at a time, whose sums stay in registers.
template <typename T, int G>
__global__ void __launch_bounds__(256)
expert_combine_bwd_kernel(ExpertRowsArgs a, int64_t blocks) {
  constexpr int V = Chunk<T>::kN, J = 8, kPer = 256 / G;
  __shared__ float lds[2][4][J];
  int half = 0;
  const int dim = static_cast<int>(a.dim), k = static_cast<int>(a.k), lane = threadIdx.x % G;
  const uint32_t slots = static_cast<uint32_t>(a.n * a.k);
  const uint32_t total = static_cast<uint32_t>(*a.total);
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t row = b * kPer + threadIdx.x / G;
    const bool here = row < a.n;
    const T* g = static_cast<const T*>(a.x) + (here ? row : 0) * a.x_stride;
    for (int j0 = 0; j0 < k; j0 += J) {
      uint32_t slot[J];
      float w[J], dot[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const bool is = here && j0 + j < k;
        slot[j] = is ? static_cast<uint32_t>(a.place[row * k + j0 + j]) : slots;
        w[j] = is ? a.weights[row * k + j0 + j] : 0.f;
        dot[j] = 0.f;
      }
      for (int c = lane * V; c < dim; c += G * V) {
        u32x4 y[J];
        const u32x4 raw = load_raw(g, c, dim);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const bool is = slot[j] < slots && slot[j] < total;
          y[j] = load_raw(static_cast<const T*>(a.ys) + (is ? slot[j] : 0) * a.ys_stride, is ? c : dim, dim);
        }
        float gv[V];
        unpack_chunk<T>(raw, c, dim, gv);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (slot[j] >= slots) continue;
          float v[V], out[V];
          unpack_chunk<T>(y[j], c, dim, v);
          const bool is = slot[j] < total;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            dot[j] += is ? gv[i] * v[i] : 0.f;
            out[i] = is ? w[j] * gv[i] : 0.f;
          }
          store_chunk(static_cast<T*>(a.out) + slot[j] * a.dim, c, dim, out);
        }
      }
#pragma unroll
      for (int j = 0; j < J; ++j) dot[j] = lane_sum<(G < 64 ? G : 64)>(dot[j]);
      if constexpr (G > 64) {
        if (threadIdx.x % 64 == 0)
#pragma unroll
          for (int j = 0; j < J; ++j) lds[half][threadIdx.x / 64][j] = dot[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < J; ++j) {
          dot[j] = 0.f;
#pragma unroll
          for (int q = 0; q < G / 64; ++q) dot[j] += lds[half][q][j];
        }
        half ^= 1;
      }
      if (here && lane == 0)
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (j0 + j < k) a.grad_weights[row * k + j0 + j] = dot[j];
    }
  }
}

constexpr int64_t kMostBlocks = 1 << 22;

struct RowGrid {
  uint32_t row_chunks;
  int64_t blocks;
  dim3 grid;
};
template <typename T>
RowGrid row_grid(const ExpertRowsArgs& a) {
  const int64_t chunks = (a.dim + Chunk<T>::kN - 1) / Chunk<T>::kN;
  const int64_t blocks = (a.n * chunks + 256 * kRowChunks - 1) / (256 * kRowChunks);
  return {static_cast<uint32_t>(chunks), blocks, dim3(static_cast<unsigned>(std::min(blocks, kMostBlocks)))};
}

template <typename T>
int dispatch_launch(const ExpertRowsArgs& a) {
  const RowGrid g = row_grid<T>(a);
  hipLaunchKernelGGL(expert_dispatch_kernel<T>, g.grid, dim3(256), 0, static_cast<hipStream_t>(a.stream), a, g.row_chunks,
                     g.blocks);
  return static_cast<int>(hipGetLastError());
}

template <typename T>
int combine_launch(const ExpertRowsArgs& a) {
  const RowGrid g = row_grid<T>(a);
  auto* kernel = a.weights ? expert_combine_kernel<T, true> : expert_combine_kernel<T, false>;
  hipLaunchKernelGGL(kernel, g.grid, dim3(256), 0, static_cast<hipStream_t>(a.stream), a, g.row_chunks, g.blocks);
  return static_cast<int>(hipGetLastError());
}

template <typename T>
int combine_bwd_launch(const ExpertRowsArgs& a) {
  const int64_t chunks = (a.dim + Chunk<T>::kN - 1) / Chunk<T>::kN;
  const hipStream_t st = static_cast<hipStream_t>(a.stream);
  // Rows of a workgroup: 16, 4 or 1.  One MI355X, us of 20000 rows of four choices, by width:
  //               bf16 256     512    1024    2048 (8192 rows)  4096 (8192, k 8)   f32 128 (50000, k 2)  256   512  1024
  //     16              19      33      81      65              301                    27                 32    80   193
  //      4              31      35      75      59              254                    52                 36    78   160
  //      1              90      90     128      68              237                   173                 87   120   148
  // and few rows take more lanes each: 500 rows of 1024 bf16 15, 7.0, 6.5, f32 23, 9.3, 6.6.
  int per = chunks <= 64 ? 16 : chunks <= (sizeof(T) == 2 ? 256 : 128) ? 4 : 1;
  while (per > 1 && (a.n + per - 1) / per < 512 && chunks > 256 / per) per /= 4;
  const int64_t blocks = (a.n + per - 1) / per;
  const dim3 grid(static_cast<unsigned>(std::min(blocks, kMostBlocks)));
  auto* kernel = per == 16 ? expert_combine_bwd_kernel<T, 16>
                           : per == 4 ? expert_combine_bwd_kernel<T, 64> : expert_combine_bwd_kernel<T, 256>;
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, a, blocks);
  return static_cast<int>(hipGetLastError());
}

}  // namespace kern

ExpertSortPlan expert_sort_plan(int64_t entries, int64_t num) {
  ExpertSortPlan p{};
  p.waves = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kSortWaves, (entries + 63) / 64)));
  // 64 entries each of a wave: one where that gives the units work, more where the counts would grow as long as the
  // list.  One MI355X, us with 1, 4 and 16 by entries (experts): 1200 (8) 7.3, 5.8, 10.8; 2048 (64) 8.2, 7.4, 13.7;
  // 8000 (64) 8.7, 13, 18; 131072 (256) 16, 20, 46; 524288 (64) 23, 21, 39; 1048576 (128) 43, 26, 48; 2000000 (16) 58,
  // 32, 38; 4000000 (2048) 387, 184, 139; 16000000 (64) 477, 254, 220.
  constexpr int64_t kTurn = 64 * kSortWaves;
  const bool one = entries <= kTurn, single = entries <= 4 * kTurn;
  p.chunks = one || (!single && entries <= 256 * kTurn) ? 1 : entries <= 2048 * kTurn ? 4 : 16;
  if (!one) p.waves = kSortWaves;
  const int64_t each = int64_t{64} * p.waves * p.chunks;
  p.blocks = std::max<int64_t>(1, (entries + each - 1) / each);
  p.bytes = p.blocks == 1 ? 0 : static_cast<size_t>(p.blocks + 1) * (num + 1) * 4;
  return p;
}

int launch_expert_sort(const ExpertSortArgs& a) {
  const ExpertSortPlan p = expert_sort_plan(a.entries, a.num);
  if (a.idx == 0) {
    if (p.chunks == 1) return kern::expert_sort_launch<int32_t, 1>(a, p);
    return p.chunks == 4 ? kern::expert_sort_launch<int32_t, 4>(a, p) : kern::expert_sort_launch<int32_t, 16>(a, p);
  }
  if (p.chunks == 1) return kern::expert_sort_launch<int64_t, 1>(a, p);
  return p.chunks == 4 ? kern::expert_sort_launch<int64_t, 4>(a, p) : kern::expert_sort_launch<int64_t, 16>(a, p);
}

#define SEGPOLY_EXPERT_ROWS(name)                                     \
  int launch_expert_##name(const ExpertRowsArgs& a) {                 \
    if (a.dtype == kChBF16) return kern::name##_launch<kern::bf16>(a); \
    if (a.dtype == kChF16) return kern::name##_launch<kern::f16>(a);   \
    return kern::name##_launch<float>(a);                             \
  }
SEGPOLY_EXPERT_ROWS(dispatch)
SEGPOLY_EXPERT_ROWS(combine)
SEGPOLY_EXPERT_ROWS(combine_bwd)
#undef SEGPOLY_EXPERT_ROWS

}  // namespace segpoly
