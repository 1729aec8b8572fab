// Embedding lookup with scaling, and the gradient of its table:
//   out[i]     = scale * table[tokens[i]]          (zero row for a token out of range)
//   d_table[r] = scale * sum over i with tokens[i] == r of g[i]
// The lookup is a copy and bound by memory: 16-byte accesses, kRowsInFlight
// independent rows per lane.
// The gradient is summed in a fixed order without atomics, so it is the same
// every time; sums are float32 and rounded once.  A table of a few rows is
// summed in LDS, every lane group into a copy of its own, over as many
// segments of positions as fill the chip, whose sums a second kernel adds.
// For other tables a stable radix sort orders (token, position), each table
// row is one range of the sorted list, and whole chunks of kEmbChunk
// positions of one row are summed first, so that a frequent token's range
// is shared out.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../channel_ops.hpp"
#include "../launch.hpp"
#include "channel_types.hpp"

namespace segpoly {

EmbeddingPlan embedding_plan(int64_t n, int64_t rows, int64_t dim) {
  EmbeddingPlan p{};
  if (rows <= kEmbDirectRows) {
    p.segments = std::max<int64_t>(1, std::min<int64_t>((n + 63) / 64, 512));
    p.bytes = round_up(4 * p.segments * rows * dim, 256);
    return p;
  }
  p.bits = 1;
  while ((int64_t{1} << p.bits) <= rows) ++p.bits;  // keys 0 .. rows (rows: token out of range)
  p.passes = (p.bits + 9) / 10;
  p.digit_bits = (p.bits + p.passes - 1) / p.passes;
  p.blocks = n > kEmbSortAlone ? (n + kEmbSortBlock - 1) / kEmbSortBlock : 1;
  p.chunks = n / kEmbChunk;
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  for (int i = 0; i < 2; ++i) p.key[i] = take(4 * n), p.pos[i] = take(4 * n);
  p.hist = take((size_t{4} << p.digit_bits) * p.blocks);
  p.rowptr = take(4 * (rows + 1));
  p.partial = take(4 * p.chunks * round_up(dim, 8));
  p.bytes = at;
  return p;
}

namespace kern {

constexpr int kRowsInFlight = 4;

// L lanes (a power of two) walk one row in 16-byte chunks; each lane keeps
// kRowsInFlight rows in flight.
template <typename T, typename Index>
__global__ void __launch_bounds__(256)
embedding_fwd_kernel(const T* __restrict__ table, const Index* __restrict__ tokens, int64_t rows, int64_t dim,
                     int64_t n, float scale, T* __restrict__ out, int64_t out_stride, int lanes) {
  constexpr int V = Chunk<T>::kN;
  const int groups = 256 / lanes;
  const int lane = threadIdx.x % lanes;
  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / lanes) * kRowsInFlight;
  int64_t tok[kRowsInFlight];
#pragma unroll
  for (int u = 0; u < kRowsInFlight; ++u) {
    tok[u] = i0 + u < n ? static_cast<int64_t>(tokens[i0 + u]) : -1;
    if (tok[u] >= rows) tok[u] = -1;
  }
  for (int c = lane * V; c < dim; c += lanes * V) {
    u32x4 raw[kRowsInFlight];
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u) {
      raw[u] = u32x4{0, 0, 0, 0};
      if (tok[u] >= 0) raw[u] = load_raw(table + tok[u] * dim, c, static_cast<int>(dim));
    }
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u) {
      if (i0 + u >= n) break;
      float v[V];
      unpack_chunk<T>(raw[u], c, static_cast<int>(dim), v);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] *= scale;
      store_chunk(out + (i0 + u) * out_stride, c, static_cast<int>(dim), v);
    }
  }
}

// ------------------------------------------------------------ tables of a few rows

// Workgroup (s, t) sums segment s of the positions over the columns of tile t.
// A lane owns one 16-byte chunk of columns of its group's copy of the table,
// acc[group][row][tile columns]: no two lanes share an address.
template <typename T, typename Index>
__global__ void __launch_bounds__(1024 / Chunk<T>::kN)
embedding_direct_kernel(const T* __restrict__ g, int64_t g_stride, const Index* __restrict__ tokens, int64_t n,
                        int rows, int dim, int lanes, float* __restrict__ partial) {
  constexpr int V = Chunk<T>::kN, kThreads = 1024 / V, kAhead = 4;
  using F4 = float __attribute__((ext_vector_type(4)));
  extern __shared__ __attribute__((aligned(16))) float acc[];
  const int groups = kThreads / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  const int tile = lanes * V, c = static_cast<int>(blockIdx.y) * tile + lane * V;
  float* mine = acc + group * rows * tile + lane * V;
  for (int r = 0; r < rows; ++r)
#pragma unroll
    for (int t = 0; t < V; t += 4) *reinterpret_cast<F4*>(mine + r * tile + t) = F4{0.f, 0.f, 0.f, 0.f};
  const int64_t end = n * (blockIdx.x + 1) / gridDim.x;
  for (int64_t i = n * blockIdx.x / gridDim.x + group; i < end; i += groups * kAhead) {
    int tok[kAhead];
    u32x4 raw[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t q = i + u * groups;
      const int64_t t = q < end ? static_cast<int64_t>(tokens[q]) : -1;
      tok[u] = t >= 0 && t < rows ? static_cast<int>(t) : -1;
      raw[u] = load_raw(g + (q < end ? q : i) * g_stride, c, dim);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (tok[u] < 0) continue;
      float v[V];
      unpack_chunk<T>(raw[u], c, dim, v);
      float* at = mine + tok[u] * tile;
#pragma unroll
      for (int t = 0; t < V; t += 4) {
        F4 s = *reinterpret_cast<F4*>(at + t);
        s += F4{v[t], v[t + 1], v[t + 2], v[t + 3]};
        *reinterpret_cast<F4*>(at + t) = s;
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * tile; i += kThreads) {
    const int col = static_cast<int>(blockIdx.y) * tile + i % tile;
    if (col >= dim) continue;
    float s = 0.f;
    for (int q = 0; q < groups; ++q) s += acc[q * rows * tile + i];
    partial[(static_cast<int64_t>(blockIdx.x) * rows + i / tile) * dim + col] = s;
  }
}

// sums of the segments: 32 values by 32 interleaved sets of segments per
// workgroup, the sets added in order
template <typename T>
__global__ void __launch_bounds__(1024)
embedding_direct_fold_kernel(const float* __restrict__ partial, int64_t segments, int64_t values, float scale,
                             T* __restrict__ out) {
  __shared__ float lds[32 * 33];
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x % 32;
  const int set = threadIdx.x / 32;
  float s = 0.f;
  if (c < values) {
#pragma unroll 8
    for (int64_t p = set; p < segments; p += 32) s += partial[p * values + c];
  }
  lds[set * 33 + threadIdx.x % 32] = s;
  __syncthreads();
  if (threadIdx.x < 32 && c < values) {
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 32; ++q) t += lds[q * 33 + threadIdx.x];
    out[c] = static_cast<T>(t * scale);
  }
}

// ------------------------------------------------------------ sorting

template <typename Index>
__device__ __forceinline__ uint32_t token_key(Index t, int64_t rows) {
  const int64_t v = static_cast<int64_t>(t);
  return static_cast<uint32_t>(v >= 0 && v < rows ? v : rows);
}

// digit counts of each block of kEmbSortBlock positions; keys null: from the tokens
template <typename Index>
__global__ void __launch_bounds__(1024)
embedding_hist_kernel(const Index* __restrict__ tokens, const uint32_t* __restrict__ keys, int64_t rows, int64_t n,
                      int shift, int bits, uint32_t* __restrict__ hist) {
  __shared__ uint32_t count[1024];
  const int D = 1 << bits;
  for (int d = threadIdx.x; d < D; d += 1024) count[d] = 0;
  __syncthreads();
  const int64_t b0 = static_cast<int64_t>(blockIdx.x) * kEmbSortBlock;
#pragma unroll
  for (int s = 0; s < kEmbSortBlock / 1024; ++s) {
    const int64_t i = b0 + s * 1024 + threadIdx.x;
    if (i < n) {
      const uint32_t k = keys ? keys[i] : token_key(tokens[i], rows);
      atomicAdd(&count[(k >> shift) & (D - 1)], 1u);
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += 1024) hist[static_cast<int64_t>(blockIdx.x) * D + d] = count[d];
}

// exclusive sum over the 1024 threads of a workgroup
__device__ __forceinline__ uint32_t scan1024(uint32_t v, uint32_t* wave_sum) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const uint32_t t = __shfl_up(s, o);
    if (lane >= o) s += t;
  }
  if (lane == 63) wave_sum[wave] = s;
  __syncthreads();
  uint32_t before = 0;
  for (int w = 0; w < wave; ++w) before += wave_sum[w];
  __syncthreads();
  return before + s - v;
}

// One stable pass over a block of positions: wave w owns consecutive ones in
// steps of 64 (as many as share the list evenly); the lanes of a step with an equal digit are
// found by one ballot per digit bit, so a position's rank is its wave's
// running count of the digit plus the equal lanes below it.  With `Single`
// the whole list is one block and every pass runs here, through LDS.
template <typename Index, bool Single, int kSteps>
__global__ void __launch_bounds__(1024)
embedding_sort_kernel(const Index* __restrict__ tokens, const uint32_t* __restrict__ keys_in,
                      const uint32_t* __restrict__ pos_in, int64_t rows, int64_t n, int pass, int passes, int bits,
                      const uint32_t* __restrict__ hist, int64_t blocks, uint32_t* __restrict__ keys_out,
                      uint32_t* __restrict__ pos_out) {
  __shared__ uint16_t count[16 * 1024];
  __shared__ uint32_t base[1024];
  __shared__ uint32_t wave_sum[16];
  __shared__ uint32_t lkey[Single ? kSteps * 1024 : 1];
  __shared__ uint16_t lpos[Single ? kSteps * 1024 : 1];
  const int D = 1 << bits;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t b0 = static_cast<int64_t>(blockIdx.x) * kEmbSortBlock;
  const int steps = Single ? static_cast<int>((n + 1023) / 1024) : kSteps;
  const int p0 = wave * steps * 64 + lane;  // position within the block at step 0
  uint32_t key[kSteps], pos[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int64_t i = b0 + p0 + s * 64;
    key[s] = 0, pos[s] = 0;
    if (s < steps && i < n) {
      key[s] = keys_in ? keys_in[i] : token_key(tokens[i], rows);
      pos[s] = pos_in ? pos_in[i] : static_cast<uint32_t>(i);
    }
  }
  volatile uint16_t* mine = count + wave * D;
  for (int p = Single ? 0 : pass; p < (Single ? passes : pass + 1); ++p) {
    const int shift = p * bits;
    for (int d = threadIdx.x; d < 16 * D; d += 1024) count[d] = 0;
    __syncthreads();
    uint32_t rank[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (s >= steps) break;
      const bool on = b0 + p0 + s * 64 < n;
      const uint32_t d = (key[s] >> shift) & (D - 1);
      uint64_t peers = __ballot(on);
      for (int b = 0; b < bits; ++b) {
        const bool bit = (d >> b) & 1;
        const uint64_t with = __ballot(bit);
        peers &= bit ? with : ~with;
      }
      const uint32_t below = __popcll(peers & ((uint64_t{1} << lane) - 1));
      rank[s] = 0;
      if (on) {
        const uint32_t seen = mine[d];
        rank[s] = seen + below;
        if (below == 0) mine[d] = static_cast<uint16_t>(seen + __popcll(peers));
      }
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    // per digit: exclusive sums over the waves, then over the digits
    uint32_t total = 0, prior = 0;
    const int d0 = threadIdx.x;
    if (d0 < D) {
      for (int w = 0; w < 16; ++w) {
        const uint32_t c = count[w * D + d0];
        count[w * D + d0] = static_cast<uint16_t>(total);
        total += c;
      }
      if (!Single) {
        total = 0;
#pragma unroll 8
        for (int64_t b = 0; b < blocks; ++b) {
          const uint32_t c = hist[b * D + d0];
          total += c;
          if (b < static_cast<int64_t>(blockIdx.x)) prior += c;
        }
      }
    }
    const uint32_t before = scan1024(total, wave_sum);
    if (d0 < D) base[d0] = before + prior;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (s < steps && b0 + p0 + s * 64 < n) {
        const uint32_t d = (key[s] >> shift) & (D - 1);
        const uint32_t to = base[d] + count[wave * D + d] + rank[s];
        if constexpr (Single) {
          lkey[to] = key[s];
          lpos[to] = static_cast<uint16_t>(pos[s]);
        } else {
          keys_out[to] = key[s];
          pos_out[to] = pos[s];
        }
      }
    }
    if constexpr (Single) {
      __syncthreads();
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if (s < steps && p0 + s * 64 < n) {
          key[s] = lkey[p0 + s * 64];
          pos[s] = lpos[p0 + s * 64];
        }
      }
      __syncthreads();
    }
  }
  if constexpr (Single) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (s < steps && p0 + s * 64 < n) {
        keys_out[p0 + s * 64] = key[s];
        pos_out[p0 + s * 64] = pos[s];
      }
    }
  }
}

// ------------------------------------------------------------ sums

// The first `range_blocks` workgroups find rowptr[r] = first sorted position
// with key >= r (r = 0 .. rows); the others sum one chunk of kEmbChunk
// positions each into partial, where the chunk holds one row only.
template <typename T>
__global__ void __launch_bounds__(256)
embedding_chunk_kernel(const T* __restrict__ g, int64_t g_stride, const uint32_t* __restrict__ keys,
                       const uint32_t* __restrict__ pos, int64_t rows, int64_t dim, int64_t n, int64_t range_blocks,
                       int lanes, uint32_t* __restrict__ rowptr, float* __restrict__ partial, int64_t pstride) {
  constexpr int V = Chunk<T>::kN;
  __shared__ float acc_lds[256 * V];
  if (blockIdx.x < range_blocks) {
    // every stride-th key in LDS narrows the search, the last steps are in memory
    constexpr int kSamples = 1024;
    static_assert(sizeof(acc_lds) >= kSamples * 4, "samples fit");
    uint32_t* sample = reinterpret_cast<uint32_t*>(acc_lds);
    int64_t stride = 16;
    while (n > stride * kSamples) stride *= 2;
    const int samples = static_cast<int>((n + stride - 1) / stride);
    for (int i = threadIdx.x; i < samples; i += 256) sample[i] = keys[i * stride];
    __syncthreads();
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (r > rows) return;
    const uint32_t key = static_cast<uint32_t>(r);
    int slo = 0, shi = samples;  // samples below slo are < key, from shi on are >= key
    while (slo < shi) {
      const int mid = (slo + shi) / 2;
      if (sample[mid] < key)
        slo = mid + 1;
      else
        shi = mid;
    }
    int64_t lo = slo ? (slo - 1) * stride + 1 : 0, hi = slo * stride < n ? slo * stride : n;
    while (lo < hi) {
      const int64_t mid = (lo + hi) / 2;
      if (keys[mid] < key)
        lo = mid + 1;
      else
        hi = mid;
    }
    rowptr[r] = static_cast<uint32_t>(lo);
    return;
  }
  const int64_t chunk = blockIdx.x - range_blocks;
  const uint32_t k0 = keys[chunk * kEmbChunk];
  if (k0 != keys[chunk * kEmbChunk + kEmbChunk - 1] || k0 >= rows) return;
  const int groups = 256 / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  for (int c0 = 0; c0 < dim; c0 += lanes * V) {
    const int c = c0 + lane * V;
    float acc[V] = {};
    if (c < dim) {
#pragma unroll 4
      for (int j = group; j < kEmbChunk; j += groups) {
        float v[V];
        load_chunk(g + static_cast<int64_t>(pos[chunk * kEmbChunk + j]) * g_stride, c, static_cast<int>(dim), v);
#pragma unroll
        for (int t = 0; t < V; ++t) acc[t] += v[t];
      }
    }
#pragma unroll
    for (int t = 0; t < V; ++t) acc_lds[t * 256 + threadIdx.x] = acc[t];
    __syncthreads();
    if (group == 0 && c < dim) {
      for (int q = 1; q < groups; ++q)
#pragma unroll
        for (int t = 0; t < V; ++t) acc[t] += acc_lds[t * 256 + q * lanes + lane];
#pragma unroll
      for (int t = 0; t < V; ++t) partial[chunk * pstride + c + t] = acc[t];
    }
    __syncthreads();
  }
}

// One table row per workgroup (Whole) or per group of `lanes` lanes (at most
// a wave): the positions before the row's first whole chunk, the chunks' sums,
// the positions after the last, zero where the range is empty.  A lane holds
// kCols chunks of columns, so a row of positions gives that many loads at
// once; the positions themselves are read by the lanes side by side.
template <typename T, bool Whole>
__global__ void __launch_bounds__(256)
embedding_rows_kernel(const T* __restrict__ g, int64_t g_stride, const uint32_t* __restrict__ pos,
                      const uint32_t* __restrict__ rowptr, const float* __restrict__ partial, int64_t pstride,
                      int64_t rows, int dim, float scale, int lanes, T* __restrict__ out) {
  constexpr int V = Chunk<T>::kN, kCols = Whole ? 1 : 2;
  __shared__ float acc_lds[Whole ? 256 * V : 1];
  const int groups = 256 / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  const int64_t r = Whole ? static_cast<int64_t>(blockIdx.x) : static_cast<int64_t>(blockIdx.x) * groups + group;
  if (!Whole && r >= rows) return;
  const int64_t s = rowptr[r], e = rowptr[r + 1];
  int64_t c_lo = (s + kEmbChunk - 1) / kEmbChunk, c_hi = e / kEmbChunk;
  const int head = static_cast<int>(c_lo < c_hi ? c_lo * kEmbChunk - s : e - s);  // loose positions from s
  const int64_t nchunk = c_lo < c_hi ? c_hi - c_lo : 0;
  const int64_t tail0 = c_lo < c_hi ? c_hi * kEmbChunk : e;                       // loose positions from tail0 to e
  const int loose = head + static_cast<int>(e - tail0);                           // fewer than 2 kEmbChunk
  const int first = Whole ? group : 0, step = Whole ? groups : 1;
  const int wide = lanes < 64 ? lanes : 64;  // each wave of a group reads the positions for itself
  for (int c0 = 0; c0 < dim; c0 += lanes * V * kCols) {
    float acc[kCols][V] = {};
    for (int i0 = 0; i0 < loose; i0 += wide) {
      const int have = loose - i0 < wide ? loose - i0 : wide, i = i0 + lane % wide;
      const int at = i < loose ? static_cast<int>(pos[i < head ? s + i : tail0 + (i - head)]) : 0;
#pragma unroll 4
      for (int j = first; j < have; j += step) {
        const T* row = g + static_cast<int64_t>(__shfl(at, j, wide)) * g_stride;
#pragma unroll
        for (int u = 0; u < kCols; ++u) {
          float v[V];
          load_chunk(row, c0 + (lane + u * lanes) * V, dim, v);
#pragma unroll
          for (int t = 0; t < V; ++t) acc[u][t] += v[t];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kCols; ++u) {
      const int c = c0 + (lane + u * lanes) * V;
      if (c >= dim) continue;
#pragma unroll 8
      for (int64_t i = first; i < nchunk; i += step) {
        const float* p = partial + (c_lo + i) * pstride + c;
#pragma unroll
        for (int t = 0; t < V; ++t) acc[u][t] += p[t];
      }
    }
    if constexpr (Whole) {
#pragma unroll
      for (int t = 0; t < V; ++t) acc_lds[t * 256 + threadIdx.x] = acc[0][t];
      __syncthreads();
      if (group == 0)
        for (int q = 1; q < groups; ++q)
#pragma unroll
          for (int t = 0; t < V; ++t) acc[0][t] += acc_lds[t * 256 + q * lanes + lane];
      __syncthreads();
      if (group != 0) continue;
    }
#pragma unroll
    for (int u = 0; u < kCols; ++u) {
#pragma unroll
      for (int t = 0; t < V; ++t) acc[u][t] *= scale;
      store_chunk(out + r * dim, c0 + (lane + u * lanes) * V, dim, acc[u]);
    }
  }
}

// lanes that walk one row: a power of two, at most `most`
template <typename T>
int row_lanes(int64_t dim, int most = 256) {
  const int64_t chunks = (dim + Chunk<T>::kN - 1) / Chunk<T>::kN;
  int lanes = 8;
  while (lanes < most && lanes < chunks) lanes *= 2;
  return lanes;
}

template <typename T, typename Index>
int embedding_fwd_launch(const EmbeddingArgs& a) {
  const int lanes = row_lanes<T>(a.dim);
  const int64_t per = 256 / lanes * kRowsInFlight;
  hipLaunchKernelGGL((embedding_fwd_kernel<T, Index>), dim3(static_cast<unsigned>((a.n + per - 1) / per)), dim3(256),
                     0, static_cast<hipStream_t>(a.stream), static_cast<const T*>(a.table),
                     static_cast<const Index*>(a.tokens), a.rows, a.dim, a.n, a.scale, static_cast<T*>(a.out),
                     a.out_stride, lanes);
  return static_cast<int>(hipGetLastError());
}

template <typename T, typename Index>
int embedding_bwd_launch(const EmbeddingArgs& a) {
  const hipStream_t st = static_cast<hipStream_t>(a.stream);
  const EmbeddingPlan p = embedding_plan(a.n, a.rows, a.dim);
  char* ws = static_cast<char*>(a.workspace);
  if (p.segments) {
    constexpr int V = Chunk<T>::kN, kThreads = 1024 / V;
    const int lanes = row_lanes<T>(a.dim, kThreads);
    const unsigned tiles = static_cast<unsigned>((a.dim + lanes * V - 1) / (lanes * V));
    float* sums = static_cast<float*>(a.workspace);
    hipLaunchKernelGGL((embedding_direct_kernel<T, Index>), dim3(static_cast<unsigned>(p.segments), tiles),
                       dim3(kThreads), static_cast<size_t>(a.rows) * 1024 * 4, st, static_cast<const T*>(a.grad),
                       a.grad_stride, static_cast<const Index*>(a.tokens), a.n, static_cast<int>(a.rows),
                       static_cast<int>(a.dim), lanes, sums);
    int rc = static_cast<int>(hipGetLastError());
    if (rc) return rc;
    const int64_t values = a.rows * a.dim;
    hipLaunchKernelGGL((embedding_direct_fold_kernel<T>), dim3(static_cast<unsigned>((values + 31) / 32)), dim3(1024), 0,
                       st, sums, p.segments, values, a.scale, static_cast<T*>(a.out));
    return static_cast<int>(hipGetLastError());
  }
  uint32_t* key[2] = {reinterpret_cast<uint32_t*>(ws + p.key[0]), reinterpret_cast<uint32_t*>(ws + p.key[1])};
  uint32_t* pos[2] = {reinterpret_cast<uint32_t*>(ws + p.pos[0]), reinterpret_cast<uint32_t*>(ws + p.pos[1])};
  uint32_t* hist = reinterpret_cast<uint32_t*>(ws + p.hist);
  uint32_t* rowptr = reinterpret_cast<uint32_t*>(ws + p.rowptr);
  float* partial = reinterpret_cast<float*>(ws + p.partial);
  const Index* tokens = static_cast<const Index*>(a.tokens);
  int last = 0;
  if (p.blocks == 1) {
    hipLaunchKernelGGL((embedding_sort_kernel<Index, true, kEmbSortAlone / 1024>), dim3(1), dim3(1024), 0, st, tokens, nullptr, nullptr, a.rows, a.n, 0, p.passes,
                       p.digit_bits, nullptr, int64_t{1}, key[0], pos[0]);
  } else {
    for (int q = 0; q < p.passes; ++q) {
      const uint32_t* kin = q ? key[last] : nullptr;
      const uint32_t* pin = q ? pos[last] : nullptr;
      const int to = q ? 1 - last : 0;
      hipLaunchKernelGGL((embedding_hist_kernel<Index>), dim3(static_cast<unsigned>(p.blocks)), dim3(1024), 0, st,
                         tokens, kin, a.rows, a.n, q * p.digit_bits, p.digit_bits, hist);
      hipLaunchKernelGGL((embedding_sort_kernel<Index, false, kEmbSortBlock / 1024>), dim3(static_cast<unsigned>(p.blocks)), dim3(1024), 0,
                         st, tokens, kin, pin, a.rows, a.n, q, p.passes, p.digit_bits, hist, p.blocks, key[to],
                         pos[to]);
      last = to;
    }
  }
  const int lanes = row_lanes<T>(a.dim);
  const int64_t range_blocks = (a.rows + 1 + 255) / 256;
  hipLaunchKernelGGL((embedding_chunk_kernel<T>), dim3(static_cast<unsigned>(range_blocks + p.chunks)), dim3(256), 0,
                     st, static_cast<const T*>(a.grad), a.grad_stride, key[last], pos[last], a.rows, a.dim, a.n,
                     range_blocks, lanes, rowptr, partial, round_up(a.dim, 8));
  // few rows: each is long, so a workgroup shares one; many: a group of at most a wave each
  const int dim = static_cast<int>(a.dim);
  if (a.rows < 2048) {
    hipLaunchKernelGGL((embedding_rows_kernel<T, true>), dim3(static_cast<unsigned>(a.rows)), dim3(256), 0, st,
                       static_cast<const T*>(a.grad), a.grad_stride, pos[last], rowptr, partial,
                       round_up(a.dim, 8), a.rows, dim, a.scale, lanes, static_cast<T*>(a.out));
  } else {
    const int narrow = row_lanes<T>(a.dim, 64), each = 256 / narrow;
    hipLaunchKernelGGL((embedding_rows_kernel<T, false>), dim3(static_cast<unsigned>((a.rows + each - 1) / each)),
                       dim3(256), 0, st, static_cast<const T*>(a.grad), a.grad_stride, pos[last], rowptr, partial,
                       round_up(a.dim, 8), a.rows, dim, a.scale, narrow, static_cast<T*>(a.out));
  }
  return static_cast<int>(hipGetLastError());
}

template <typename T>
int embedding_dispatch(const EmbeddingArgs& a, bool backward) {
  if (a.idx == kI32)
    return backward ? embedding_bwd_launch<T, int32_t>(a) : embedding_fwd_launch<T, int32_t>(a);
  return backward ? embedding_bwd_launch<T, int64_t>(a) : embedding_fwd_launch<T, int64_t>(a);
}

int embedding_any(const EmbeddingArgs& a, bool backward) {
  if (a.dtype == kChBF16) return embedding_dispatch<bf16>(a, backward);
  if (a.dtype == kChF16) return embedding_dispatch<f16>(a, backward);
  return embedding_dispatch<float>(a, backward);
}

}  // namespace kern

int launch_embedding_fwd(const EmbeddingArgs& a) { return kern::embedding_any(a, false); }
int launch_embedding_bwd(const EmbeddingArgs& a) { return kern::embedding_any(a, true); }

}  // namespace segpoly
