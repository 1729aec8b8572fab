// Embedding lookup with scaling, and the gradient of its table:
//   out[i]     = scale * table[tokens[i]]          (zero row for a token out of range)
//   d_table[r] = scale * sum over i with tokens[i] == r of g[i]
// The lookup is a copy and bound by memory: 16-byte accesses, kRowsInFlight
// independent rows per lane.
// The gradient is summed in a fixed order without atomics, so it is the same
// every time; sums are float32 and rounded once.  A table of a few rows is
// summed in LDS, every lane group into a copy of its own, over as many
// segments of positions as fill the chip, whose sums a second kernel adds.
// For other tables a stable sort orders (token, position), each table row is
// one range of the sorted list, and whole chunks of kEmbChunk positions of one
// row are summed first, so that a frequent token's range is shared out.  The
// sort is one launch where every workgroup can read all tokens and keep those
// of its rows in LDS, a radix sort above.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../channel_ops.hpp"
#include "../launch.hpp"
#include "channel_types.hpp"
#include "column_sums.hpp"

namespace segpoly {

EmbeddingPlan embedding_plan(int64_t n, int64_t rows, int64_t dim) {
  EmbeddingPlan p{};
  if (rows <= kEmbDirectRows) {
    // 512 workgroups over the segments and the tiles of 1024 columns
    p.segments = std::max<int64_t>(1, std::min<int64_t>((n + 15) / 16, 512 / std::max<int64_t>(1, (dim + 1023) / 1024)));
    p.bytes = round_up(4 * p.segments * rows * dim, 256);
    return p;
  }
  const bool order = n <= kEmbOrderTokens && rows <= kEmbOrderRows;
  p.groups = order ? kEmbGroups : 1;
  p.per_group = (rows + p.groups - 1) / p.groups;
  p.keys = p.per_group * p.groups;
  p.bits = 1;
  while ((int64_t{1} << p.bits) <= rows) ++p.bits;  // keys 0 .. rows (rows: token out of range)
  p.passes = order ? 0 : (p.bits + 9) / 10;
  p.digit_bits = order ? 0 : (p.bits + p.passes - 1) / p.passes;
  p.blocks = (n + kEmbSortBlock - 1) / kEmbSortBlock;
  p.chunks = n / kEmbChunk;
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  for (int i = 0; i < (order ? 1 : 2); ++i) p.key[i] = take(4 * n), p.pos[i] = take(4 * n);
  p.hist = take((size_t{4} << p.digit_bits) * (p.blocks + 1));
  p.rowptr = take(4 * (p.keys + 1));
  p.partial = take(4 * p.chunks * round_up(dim, 8));
  p.bytes = at;
  return p;
}

namespace kern {

constexpr int kRowsInFlight = 4;
// Workgroups of a launch at most, which has fewer than 2^32 threads: longer lists
// and larger tables take several.
constexpr int64_t kMostBlocks = int64_t{1} << 22;

// `lanes` lanes (a power of two) walk one row in 16-byte chunks; each lane keeps
// kRowsInFlight rows in flight.  32768 rows of 2048 bf16 on one MI355X: 42 us,
// 134 MB written.
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
// acc[group][row][tile columns]: no two lanes share an address.  50000 positions
// into 10 rows of 128 f32 on one MI355X: 11 us and 3 us for the segments' sums (a
// group's twelve rows in three rounds of loads, one after another);
// sorted as a large table 27 us.
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
  const int tile_bits = __builtin_ctz(tile);  // a power of two, as the lanes are
#pragma unroll 4
  for (int i = threadIdx.x; i < rows << tile_bits; i += kThreads) {
    const int r = i >> tile_bits, col = static_cast<int>(blockIdx.y) * tile + (i & (tile - 1));
    float s = 0.f;
    for (int q = 0; q < groups; ++q) s += acc[((q * rows) << tile_bits) + i];
    if (col < dim) partial[(static_cast<int64_t>(blockIdx.x) * rows + r) * dim + col] = s;
  }
}

// sums of the segments
template <typename T>
__global__ void __launch_bounds__(1024)
embedding_direct_fold_kernel(const float* __restrict__ partial, int64_t segments, int64_t values, float scale,
                             T* __restrict__ out) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x % 32;
  const float t = column_sum(partial, segments, values, values, c);
  if (threadIdx.x < 32 && c < values) out[c] = static_cast<T>(t * scale);
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

// Counts of the workgroups before each, and of all, for 64 digits a workgroup: the
// counts of kEmbScanBlocks workgroups and more, which the sorting workgroups would
// otherwise each add up alone, in time that grows with their square.
__global__ void __launch_bounds__(1024)
embedding_scan_kernel(uint32_t* __restrict__ hist, int64_t blocks, int D) {
  __shared__ uint32_t sum[16][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int d = blockIdx.x * 64 + lane;
  const bool on = d < D;
  const int64_t b0 = blocks * wave / 16, b1 = blocks * (wave + 1) / 16;
  uint32_t own = 0;
  if (on) {
#pragma unroll 8
    for (int64_t b = b0; b < b1; ++b) own += hist[b * D + d];
  }
  sum[wave][lane] = own;
  __syncthreads();
  uint32_t before = 0;
  for (int w = 0; w < wave; ++w) before += sum[w][lane];
  if (!on) return;
#pragma unroll 8
  for (int64_t b = b0; b < b1; ++b) {
    const uint32_t c = hist[b * D + d];
    hist[b * D + d] = before;
    before += c;
  }
  if (wave == 15) hist[blocks * D + d] = before;
}

// lanes of the wave that are on and have the same key of `bits` bits, by one ballot per bit
__device__ __forceinline__ uint64_t equal_lanes(bool on, uint32_t key, int bits) {
  uint64_t peers = __ballot(on);
  for (int b = 0; b < bits; ++b) {
    const bool bit = (key >> b) & 1;
    const uint64_t with = __ballot(bit);
    peers &= bit ? with : ~with;
  }
  return peers;
}
__device__ __forceinline__ uint32_t lanes_below(uint64_t mask) {
  return __popcll(mask & ((uint64_t{1} << (threadIdx.x % 64)) - 1));
}

// One stable pass over a block of positions: wave w owns 256 consecutive
// ones in four steps of 64; a position's rank is its wave's running count of
// the digit plus the equal lanes below it.
template <typename Index>
__global__ void __launch_bounds__(1024)
embedding_sort_kernel(const Index* __restrict__ tokens, const uint32_t* __restrict__ keys_in,
                      const uint32_t* __restrict__ pos_in, int64_t rows, int64_t n, int shift, int bits,
                      const uint32_t* __restrict__ hist, int64_t blocks, uint32_t* __restrict__ keys_out,
                      uint32_t* __restrict__ pos_out) {
  constexpr int kSteps = kEmbSortBlock / 1024;
  __shared__ uint16_t count[16 * 1024];
  __shared__ uint32_t base[1024];
  __shared__ uint32_t wave_sum[16];
  const int D = 1 << bits;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kEmbSortBlock + wave * 256 + lane;
  uint32_t key[kSteps], pos[kSteps], rank[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int64_t i = i0 + s * 64;
    key[s] = 0, pos[s] = 0;
    if (i < n) {
      key[s] = keys_in ? keys_in[i] : token_key(tokens[i], rows);
      pos[s] = pos_in ? pos_in[i] : static_cast<uint32_t>(i);
    }
  }
  for (int d = threadIdx.x; d < 16 * D; d += 1024) count[d] = 0;
  __syncthreads();
  volatile uint16_t* mine = count + wave * D;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const bool on = i0 + s * 64 < n;
    const uint32_t d = (key[s] >> shift) & (D - 1);
    const uint64_t peers = equal_lanes(on, d, bits);
    const uint32_t below = lanes_below(peers);
    rank[s] = 0;
    if (on) {
      const uint32_t seen = mine[d];
      rank[s] = seen + below;
      if (below == 0) mine[d] = static_cast<uint16_t>(seen + __popcll(peers));
    }
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  // per digit: exclusive sums over the waves, then over the digits and the workgroups before
  uint32_t total = 0, prior = 0;
  const int d0 = threadIdx.x;
  if (d0 < D) {
    for (int w = 0; w < 16; ++w) {
      const uint32_t c = count[w * D + d0];
      count[w * D + d0] = static_cast<uint16_t>(total);
      total += c;
    }
    total = 0;
    if (blocks >= kEmbScanBlocks) {  // added up by embedding_scan_kernel
      prior = hist[static_cast<int64_t>(blockIdx.x) * D + d0];
      total = hist[blocks * D + d0];
    } else {
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
    if (i0 + s * 64 < n) {
      const uint32_t d = (key[s] >> shift) & (D - 1);
      const uint32_t to = base[d] + count[wave * D + d] + rank[s];
      keys_out[to] = key[s];
      pos_out[to] = pos[s];
    }
  }
}

// The whole order in one launch.  Workgroup w reads all tokens, wave by wave
// consecutive ones, keeps those of the rows r = w modulo kEmbGroups in LDS in
// order, counts those of the groups before w, which is where its ranges
// start, and sorts what it kept by r / kEmbGroups as above.  Every workgroup
// reads the same tokens, at most 256 KB, from its L2.  16384 tokens into 32768
// rows on one MI355X: 16 us; as two radix passes of two launches each 29 us.
template <typename Index>
__global__ void __launch_bounds__(1024)
embedding_order_kernel(const Index* __restrict__ tokens, int64_t rows, int n, int per_group, int bits,
                       uint32_t* __restrict__ keys_out, uint32_t* __restrict__ pos_out,
                       uint32_t* __restrict__ rowptr) {
  constexpr int kSteps = kEmbOrderTokens / 1024, kKeys = kEmbOrderRows / kEmbGroups;
  __shared__ uint16_t list_key[kEmbOrderTokens];
  __shared__ uint16_t list_pos[kEmbOrderTokens];
  __shared__ uint16_t count[16 * kKeys];
  __shared__ uint32_t wave_sum[16], wave_kept[16], wave_before[16];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const uint32_t group = blockIdx.x;
  const int steps = (n + 1023) / 1024, i0 = wave * steps * 64 + lane;
  uint32_t key[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int i = i0 + s * 64;
    key[s] = s < steps && i < n ? token_key(tokens[i], rows) : static_cast<uint32_t>(rows);
  }
  uint32_t kept = 0, before = 0;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if (s >= steps) break;
    const bool valid = key[s] < static_cast<uint32_t>(rows);
    const uint32_t of = key[s] % kEmbGroups;
    kept += __popcll(__ballot(valid && of == group));
    before += __popcll(__ballot(valid && of < group));
  }
  if (lane == 0) wave_kept[wave] = kept, wave_before[wave] = before;
  for (int d = threadIdx.x; d < 16 * per_group; d += 1024) count[d] = 0;
  __syncthreads();
  uint32_t at = 0, length = 0, first = 0;  // this wave's place in the list, the list's length, the group's first range
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    if (w < wave) at += wave_kept[w];
    length += wave_kept[w];
    first += wave_before[w];
  }
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if (s >= steps) break;
    const bool mine = key[s] < static_cast<uint32_t>(rows) && key[s] % kEmbGroups == group;
    const uint64_t all = __ballot(mine);
    if (mine) {
      const uint32_t to = at + lanes_below(all);
      list_key[to] = static_cast<uint16_t>(key[s] / kEmbGroups);
      list_pos[to] = static_cast<uint16_t>(i0 + s * 64);
    }
    at += __popcll(all);
  }
  __syncthreads();
  // counts of each wave's share of the list, then its first place of each key
  const int share = (length + 1023) / 1024 * 64;
  volatile uint16_t* my = count + wave * per_group;
  for (int s = 0; s < share; s += 64) {
    const uint32_t i = wave * share + s + lane;
    const bool on = i < length;
    const uint32_t k = on ? list_key[i] : 0;
    const uint64_t peers = equal_lanes(on, k, bits);
    if (on && lanes_below(peers) == 0) my[k] = static_cast<uint16_t>(my[k] + __popcll(peers));
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  uint32_t total = 0;
  const int k0 = threadIdx.x;
  if (k0 < per_group)
    for (int w = 0; w < 16; ++w) total += count[w * per_group + k0];
  const uint32_t start = scan1024(total, wave_sum);
  if (k0 < per_group) {
    rowptr[group * per_group + k0] = first + start;
    uint32_t place = start;
    for (int w = 0; w < 16; ++w) {
      const uint32_t c = count[w * per_group + k0];
      count[w * per_group + k0] = static_cast<uint16_t>(place);
      place += c;
    }
  }
  __syncthreads();
  for (int s = 0; s < share; s += 64) {
    const uint32_t i = wave * share + s + lane;
    const bool on = i < length;
    const uint32_t k = on ? list_key[i] : 0;
    const uint64_t peers = equal_lanes(on, k, bits);
    const uint32_t below = lanes_below(peers);
    if (on) {
      const uint32_t seen = my[k], to = first + seen + below;
      keys_out[to] = group * per_group + k;
      pos_out[to] = list_pos[i];
      if (below == 0) my[k] = static_cast<uint16_t>(seen + __popcll(peers));
    }
    __builtin_amdgcn_wave_barrier();
  }
  if (group == kEmbGroups - 1) {
    const uint32_t end = first + length;
    if (threadIdx.x == 0) rowptr[kEmbGroups * per_group] = end;
    for (uint32_t i = end + threadIdx.x; i < static_cast<uint32_t>(n); i += 1024)
      keys_out[i] = kEmbGroups * static_cast<uint32_t>(per_group);  // tokens out of range
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
                       int64_t chunks, int lanes, uint32_t* __restrict__ rowptr, float* __restrict__ partial, int64_t pstride) {
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
  const int groups = 256 / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  for (int64_t chunk = blockIdx.x - range_blocks; chunk < chunks; chunk += gridDim.x - range_blocks) {
    const uint32_t k0 = keys[chunk * kEmbChunk];
    if (k0 != keys[chunk * kEmbChunk + kEmbChunk - 1] || k0 >= rows) continue;
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
}

// Adds to acc the items first, first + step, ... of a range [s, e) of the sorted
// list, for the columns c0 + (lane + u lanes) V: the positions before the first
// whole chunk and after the last, then the chunks' sums.
template <typename T, int kCols>
__device__ __forceinline__ void sum_range(const T* __restrict__ g, int64_t g_stride, const uint32_t* __restrict__ pos,
                                          const float* __restrict__ partial, int64_t pstride, int64_t s, int64_t e,
                                          int dim, int c0, int lane, int lanes, int first, int step,
                                          float (&acc)[kCols][Chunk<T>::kN]) {
  constexpr int V = Chunk<T>::kN;
  const int64_t c_lo = (s + kEmbChunk - 1) / kEmbChunk, c_hi = e / kEmbChunk;
  const bool whole = c_lo < c_hi;
  const int head = static_cast<int>(whole ? c_lo * kEmbChunk - s : e - s);
  const int64_t tail = whole ? c_hi * kEmbChunk : e;
  const int loose = head + static_cast<int>(e - tail);  // fewer than 2 kEmbChunk
#pragma unroll 4
  for (int i = first; i < loose; i += step) {
    const T* row = g + static_cast<int64_t>(pos[i < head ? s + i : tail + (i - head)]) * g_stride;
#pragma unroll
    for (int u = 0; u < kCols; ++u) {
      float v[V];
      load_chunk(row, c0 + (lane + u * lanes) * V, dim, v);
#pragma unroll
      for (int t = 0; t < V; ++t) acc[u][t] += v[t];
    }
  }
  if (!whole) return;
#pragma unroll 4
  for (int64_t i = c_lo + first; i < c_hi; i += step) {
#pragma unroll
    for (int u = 0; u < kCols; ++u) {
      const int c = c0 + (lane + u * lanes) * V;
      if (c >= dim) continue;
      const float* p = partial + i * pstride + c;
#pragma unroll
      for (int t = 0; t < V; ++t) acc[u][t] += p[t];
    }
  }
}

// A workgroup takes 16 table rows, or one for each of its groups of `lanes`
// lanes (at most a wave), every gridDim.x-th: frequent tokens are often
// neighbours.  It writes zeros for its empty ranges, all threads together: most
// rows of a large table have no token, and the dependent loads of the others'
// sums take longer than all the zeros.  Then a group of lanes sums a short range
// alone; a range of more than kAlone items is shared out over all groups, whose
// sums are added in order: the few frequent tokens would otherwise be the
// kernel's last groups.  (kAlone 8, 16, 32: 100000 tokens spread evenly over 16000
// rows of 64 bf16 87, 47, 45 us, a text's 65, 59, 59; 16384 of a text over 50000
// 28, 28, 31.)  Few: one row per workgroup.  32768 x 1024 bf16, 16384 tokens: 20 us,
// 3.9 TB/s (one row per 64 lanes, empty or not: 41 us).
template <typename T, bool Few>
__global__ void __launch_bounds__(256)
embedding_rows_kernel(const T* __restrict__ g, int64_t g_stride, const uint32_t* __restrict__ pos,
                      const uint32_t* __restrict__ rowptr, const float* __restrict__ partial, int64_t pstride,
                      int64_t first_row, int64_t rows, int groups_of_rows, int64_t per_group, int dim, float scale,
                      int lanes, T* __restrict__ out) {
  constexpr int V = Chunk<T>::kN, kCols = 2, kAlone = Few ? -1 : 16;
  __shared__ float acc_lds[256 * V * kCols];
  __shared__ uint32_t range[2][32];
  __shared__ int long_rows[32], long_count;
  const int groups = 256 / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  const int here = Few ? 1 : groups > 16 ? groups : 16;  // rows of this workgroup
  auto row_of = [=](int q) { return first_row + blockIdx.x + static_cast<int64_t>(q) * gridDim.x; };
  auto items = [](int64_t s, int64_t e) {  // loads of a lane that sums the range alone
    const int64_t c_lo = (s + kEmbChunk - 1) / kEmbChunk, c_hi = e / kEmbChunk;
    return c_lo < c_hi ? e - s - (c_hi - c_lo) * (kEmbChunk - 1) : e - s;
  };
  if (threadIdx.x == 0) long_count = 0;
  __syncthreads();
  if (threadIdx.x < here) {
    const int64_t r = row_of(threadIdx.x);
    const int64_t at = r < rows ? r % groups_of_rows * per_group + r / groups_of_rows : 0;
    const uint32_t s = r < rows ? rowptr[at] : 0, e = r < rows ? rowptr[at + 1] : 0;
    range[0][threadIdx.x] = s;
    range[1][threadIdx.x] = e;
    // the order of the list does not matter: its rows are independent
    if (r < rows && items(s, e) > kAlone) long_rows[atomicAdd(&long_count, 1)] = threadIdx.x;
  }
  __syncthreads();
  auto put = [&](int64_t r, int c0, float(&acc)[kCols][V]) {
#pragma unroll
    for (int u = 0; u < kCols; ++u) {
#pragma unroll
      for (int t = 0; t < V; ++t) acc[u][t] *= scale;
      store_chunk(out + r * dim, c0 + (lane + u * lanes) * V, dim, acc[u]);
    }
  };
  if constexpr (!Few) {
    const int chunks = (dim + V - 1) / V;
    for (int i = threadIdx.x; i < here * chunks; i += 256) {
      const int q = i / chunks;
      constexpr float zero[V] = {};
      if (row_of(q) < rows && range[0][q] == range[1][q])
        store_chunk(out + row_of(q) * dim, i % chunks * V, dim, zero);
    }
    for (int q = group; q < here; q += groups) {
      const int64_t s = range[0][q], e = range[1][q];
      if (s == e || items(s, e) > kAlone) continue;
      for (int c0 = 0; c0 < dim; c0 += lanes * V * kCols) {
        float acc[kCols][V] = {};
        sum_range<T, kCols>(g, g_stride, pos, partial, pstride, s, e, dim, c0, lane, lanes, 0, 1, acc);
        put(row_of(q), c0, acc);
      }
    }
  }
  for (int k = 0; k < long_count; ++k) {
    const int q = long_rows[k];
    const int64_t s = range[0][q], e = range[1][q];
    for (int c0 = 0; c0 < dim; c0 += lanes * V * kCols) {
      float acc[kCols][V] = {};
      sum_range<T, kCols>(g, g_stride, pos, partial, pstride, s, e, dim, c0, lane, lanes, group, groups, acc);
#pragma unroll
      for (int u = 0; u < kCols; ++u)
#pragma unroll
        for (int t = 0; t < V; ++t) acc_lds[(u * V + t) * 256 + threadIdx.x] = acc[u][t];
      __syncthreads();
      if (group == 0) {
        for (int o = 1; o < groups; ++o)
#pragma unroll
          for (int u = 0; u < kCols; ++u)
#pragma unroll
            for (int t = 0; t < V; ++t) acc[u][t] += acc_lds[(u * V + t) * 256 + o * lanes + lane];
        put(row_of(q), c0, acc);
      }
      __syncthreads();
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
  for (int64_t first = 0, slice = kMostBlocks * per; first < a.n; first += slice) {
    const int64_t n = std::min(a.n - first, slice);
    hipLaunchKernelGGL((embedding_fwd_kernel<T, Index>), dim3(static_cast<unsigned>((n + per - 1) / per)), dim3(256), 0,
                       static_cast<hipStream_t>(a.stream), static_cast<const T*>(a.table),
                       static_cast<const Index*>(a.tokens) + first, a.rows, a.dim, n, a.scale,
                       static_cast<T*>(a.out) + first * a.out_stride, a.out_stride, lanes);
    if (const int rc = static_cast<int>(hipGetLastError())) return rc;
  }
  return 0;
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
  if (p.groups > 1) {
    int bits = 0;
    while ((1 << bits) < p.per_group) ++bits;
    hipLaunchKernelGGL((embedding_order_kernel<Index>), dim3(kEmbGroups), dim3(1024), 0, st, tokens, a.rows,
                       static_cast<int>(a.n), static_cast<int>(p.per_group), bits, key[0], pos[0], rowptr);
    if (const int rc = static_cast<int>(hipGetLastError())) return rc;
  } else {
    for (int q = 0; q < p.passes && p.blocks; ++q) {
      const uint32_t* kin = q ? key[last] : nullptr;
      const uint32_t* pin = q ? pos[last] : nullptr;
      const int to = q ? 1 - last : 0;
      hipLaunchKernelGGL((embedding_hist_kernel<Index>), dim3(static_cast<unsigned>(p.blocks)), dim3(1024), 0, st,
                         tokens, kin, a.rows, a.n, q * p.digit_bits, p.digit_bits, hist);
      if (const int rc = static_cast<int>(hipGetLastError())) return rc;
      if (p.blocks >= kEmbScanBlocks) {
        hipLaunchKernelGGL(embedding_scan_kernel, dim3(((1u << p.digit_bits) + 63) / 64), dim3(1024), 0, st, hist,
                           p.blocks, 1 << p.digit_bits);
        if (const int rc = static_cast<int>(hipGetLastError())) return rc;
      }
      hipLaunchKernelGGL((embedding_sort_kernel<Index>), dim3(static_cast<unsigned>(p.blocks)), dim3(1024), 0, st,
                         tokens, kin, pin, a.rows, a.n, q * p.digit_bits, p.digit_bits, hist, p.blocks, key[to],
                         pos[to]);
      if (const int rc = static_cast<int>(hipGetLastError())) return rc;
      last = to;
    }
  }
  const int lanes = row_lanes<T>(a.dim);
  const int64_t range_blocks = p.groups > 1 ? 0 : (a.rows + 1 + 255) / 256;
  const int64_t chunk_blocks = range_blocks + std::min(p.chunks, kMostBlocks);
  if (chunk_blocks > 0) {
    hipLaunchKernelGGL((embedding_chunk_kernel<T>), dim3(static_cast<unsigned>(chunk_blocks)), dim3(256), 0, st,
                       static_cast<const T*>(a.grad), a.grad_stride, key[last], pos[last], p.keys, a.dim, a.n,
                       range_blocks, p.chunks, lanes, rowptr, partial, round_up(a.dim, 8));
    if (const int rc = static_cast<int>(hipGetLastError())) return rc;
  }
  const int narrow = row_lanes<T>(a.dim, 64), each = std::max(256 / narrow, 16);
  // One row a workgroup where rows are too few for the chip in sixteens, or have many
  // tokens each.  One MI355X, us with one row and with sixteen:
  //   tokens, even       16384                       100000
  //   rows            1000        4000    16000      2000        4000       16000
  //   64 bf16         25, 132     36, 33  88, 20     52, 172     61, 159    114, 87
  //   1024 bf16       31, 84      34, 42  61, 34     72, 136     76, 121    104, 94
  //   128 f32         20, 47      23, 25  42, 22     48, 85      51, 82      70, 67
  const bool few = a.rows < 2048 || a.n >= 16 * a.rows;
  auto* sum = few ? embedding_rows_kernel<T, true> : embedding_rows_kernel<T, false>;
  // as many rows a launch as its workgroups may be
  for (int64_t first = 0, slice = kMostBlocks * each; first < a.rows; first += slice) {
    const int64_t end = std::min(a.rows, first + slice), here = end - first;
    hipLaunchKernelGGL(sum, dim3(static_cast<unsigned>(few ? here : (here + each - 1) / each)), dim3(256), 0, st,
                       static_cast<const T*>(a.grad), a.grad_stride, pos[last], rowptr, partial, round_up(a.dim, 8), first,
                       end, p.groups, p.per_group, static_cast<int>(a.dim), a.scale, narrow, static_cast<T*>(a.out));
    if (const int rc = static_cast<int>(hipGetLastError())) return rc;
  }
  return 0;
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
