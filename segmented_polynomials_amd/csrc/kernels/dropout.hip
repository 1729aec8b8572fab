// Dropout with a counter-based generator:
//   out = residual + keep x / (1 - p),
//   keep[row, col] = word col % 4 of philox(counter (col / 4, row, offset), key seed) >= p 2^32
// with Philox 4x32-10 of Salmon et al., "Parallel random numbers: as easy as 1,
// 2, 3" (2011): ten rounds of two 32 x 32 -> 64-bit products.  The mask of an
// element depends on the seed, the offset and its place alone, so the gradient
// makes it again and nothing is stored.  A thread's 16-byte chunk begins at a
// multiple of four columns: each generator call serves four neighbours.
// Bound by memory: x and the residual are read once, the output is written
// once; the twenty products of a call cost less than their elements' transfers.
// One MI355X: 16384 x 2048 bf16 with a residual 42 us, 4.8 TB/s; 20000 x 128 float32
// 7 us, a launch of one round.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../channel_ops.hpp"
#include "channel_types.hpp"

namespace segpoly {
namespace kern {

struct Words {
  uint32_t w[4];
};

__device__ __forceinline__ Words philox(uint32_t c0, uint32_t c1, uint64_t c23, uint64_t key) {
  uint32_t c2 = static_cast<uint32_t>(c23), c3 = static_cast<uint32_t>(c23 >> 32);
  uint32_t k0 = static_cast<uint32_t>(key), k1 = static_cast<uint32_t>(key >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = uint64_t{0xD2511F53} * c0, b = uint64_t{0xCD9E8D57} * c2;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(b);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9;
    k1 += 0xBB67AE85;
  }
  return Words{{c0, c1, c2, c3}};
}

constexpr int kDropChunks = 4;  // of a thread, in flight together

// A workgroup takes 256 * kDropChunks chunks one after another of the rows'.
template <typename T, bool Residual, bool Rows>
__global__ void __launch_bounds__(256)
dropout_kernel(DropoutArgs a, uint32_t row_chunks, int64_t blocks) {
  constexpr int V = Chunk<T>::kN, U = kDropChunks;
  const int dim = static_cast<int>(a.dim);
  const uint64_t key = a.seed + (a.state ? static_cast<uint64_t>(a.state[0]) : 0);
  const uint64_t offset = a.offset + (a.state ? static_cast<uint64_t>(a.state[1]) : 0);
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t first = b * (256 * U), row0 = first / row_chunks;
    const uint32_t chunk0 = static_cast<uint32_t>(first % row_chunks) + threadIdx.x;
    int64_t row[U];
    int col[U];
    bool any[U];
    u32x4 x[U], res[U];
    Words words[U][Rows ? 1 : V / 4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t at = chunk0 + u * 256, r = at / row_chunks;
      row[u] = row0 + r;
      col[u] = row[u] < a.n ? static_cast<int>(at - r * row_chunks) * V : dim;  // nothing past the last row
      any[u] = !a.drop_all;
      if constexpr (Rows) {
        words[u][0] = philox(0, static_cast<uint32_t>(row[u]), offset, key);
        any[u] = any[u] && words[u][0].w[0] >= a.below;
      }
      const int64_t at_row = row[u] < a.n ? row[u] : 0;
      x[u] = load_raw(static_cast<const T*>(a.x) + at_row * a.x_stride, any[u] ? col[u] : dim, dim);
      if constexpr (Residual)
        res[u] = load_raw(static_cast<const T*>(a.residual) + at_row * a.residual_stride, col[u], dim);
    }
    if constexpr (!Rows) {
      if (a.below != 0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int q = 0; q < V / 4; ++q)
            words[u][q] = philox(static_cast<uint32_t>(col[u] / 4 + q), static_cast<uint32_t>(row[u]), offset, key);
      } else {  // all are kept
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int q = 0; q < V / 4; ++q) words[u][q] = Words{{0, 0, 0, 0}};
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[V], s[V];
      unpack_chunk<T>(x[u], col[u], dim, v);
      if constexpr (Residual) unpack_chunk<T>(res[u], col[u], dim, s);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // chosen, not multiplied: what is dropped counts for nothing, NaN included
        bool keep = any[u];
        if constexpr (!Rows) keep = keep && words[u][i / 4].w[i % 4] >= a.below;
        v[i] = keep ? v[i] * a.scale : 0.f;
        if constexpr (Residual) v[i] += s[i];
      }
      const int64_t at_row = row[u] < a.n ? row[u] : 0;
      store_chunk(static_cast<T*>(a.out) + at_row * a.out_stride, col[u], dim, v);
    }
  }
}

template <typename T>
int dropout_launch(const DropoutArgs& a) {
  const int64_t row_chunks = (a.dim + Chunk<T>::kN - 1) / Chunk<T>::kN;
  const int64_t blocks = (a.n * row_chunks + 256 * kDropChunks - 1) / (256 * kDropChunks);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(blocks, 1 << 22)));
  const hipStream_t st = static_cast<hipStream_t>(a.stream);
  auto* kernel = a.residual ? (a.rows ? dropout_kernel<T, true, true> : dropout_kernel<T, true, false>)
                            : (a.rows ? dropout_kernel<T, false, true> : dropout_kernel<T, false, false>);
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, a, static_cast<uint32_t>(row_chunks), blocks);
  return static_cast<int>(hipGetLastError());
}

}  // namespace kern

int launch_dropout(const DropoutArgs& a) {
  if (a.dtype == kChBF16) return kern::dropout_launch<kern::bf16>(a);
  if (a.dtype == kChF16) return kern::dropout_launch<kern::f16>(a);
  return kern::dropout_launch<float>(a);
}

}  // namespace segpoly
