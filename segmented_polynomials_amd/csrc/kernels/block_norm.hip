// The join of two residual blocks in one pass over the rows:
//   y = x + res_scale * gate(f) * (norm(f) * w_post)
//   h = norm(y) * w_pre
// norm(v) = (v - m) / sqrt(mean((v - m)^2) + eps), m = mean(v) (layer) or 0
// (rms); gate absent, one value per row, or one per element, taken as given
// or through a sigmoid.  The backward starts from the stored y:
//   dy  = gy + N(y, gh * w_pre),   N(v, q) = (q - n mean(q n) [- mean(q)]) / s
//         with n = norm(v), s = sqrt(mean((v - m)^2) + eps), the bracket for layer
//   df  = N(f, dy * res_scale * gate * w_post), the parameters' gradients the
//   column sums over the rows.
// Both directions are bound by memory: a row is held in registers from its
// one read to its one write, so every tensor crosses HBM once; statistics are
// float32 and the variance is taken about the mean (two passes over
// registers).  G lanes hold one row, kE = 8 elements per lane while the row
// fits in a workgroup; up to 64 lanes the reductions need no barrier, so
// narrow rows share a wave.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../channel_ops.hpp"
#include "../launch.hpp"
#include "channel_types.hpp"

namespace segpoly {

int64_t block_norm_parts(int64_t n, int64_t dim) {
  // one row group of G lanes holds 8 elements per lane; workgroups of 256
  // lanes or one row, about 1024 lanes resident per compute unit
  int64_t lanes = 16;
  while (lanes < 1024 && lanes * 8 < dim) lanes *= 2;
  const int64_t per = lanes < 256 ? 256 / lanes : 1;
  const int64_t threads = lanes < 256 ? 256 : lanes;
  const int64_t groups = (n + per - 1) / per;
  return std::max<int64_t>(1, std::min<int64_t>(groups, 256 * (1024 / threads)));
}

namespace kern {

enum { kGateNone = 0, kGateRow = 1, kGateElement = 2 };

// Sums of K values over the G lanes of a row; every lane gets them.
template <int G, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* lds) {
#pragma unroll
  for (int o = (G < 64 ? G : 64) / 2; o > 0; o /= 2)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], o);
  if constexpr (G > 64) {
    constexpr int W = G / 64;
    const int wave = threadIdx.x / 64 % W, base = threadIdx.x / G * W * K;
    __syncthreads();  // the previous sums have been read
    if (threadIdx.x % 64 == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) lds[base + wave * K + k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += lds[base + w * K + k];
      v[k] = s;
    }
  }
}

// Lane l of a row holds the chunks c = l, l + G, ...: R chunks of V elements.
template <typename T, int G, int E>
struct RowMap {
  static constexpr int V = Chunk<T>::kN;
  static constexpr int R = E / V;
  __device__ __forceinline__ static int col(int r) { return ((threadIdx.x % G) + r * G) * V; }
  __device__ __forceinline__ static void load(const T* row, int dim, float (&v)[E]) {
#pragma unroll
    for (int r = 0; r < R; ++r) load_chunk(row + col(r), dim - col(r), v + r * V);
  }
  __device__ __forceinline__ static void store(T* row, int dim, const float (&v)[E]) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (col(r) < dim) store_chunk(row + col(r), dim - col(r), v + r * V);
  }
  __device__ __forceinline__ static void params(const float* p, int dim, float fill, float (&v)[E]) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = col(r) + j;
        v[r * V + j] = c < dim ? (p ? p[c] : fill) : 0.f;
      }
  }
  __device__ __forceinline__ static bool on(int i, int dim) { return col(i / V) + i % V < dim; }
};

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + __expf(-v)); }

template <typename T, int G, int E>
__global__ void __launch_bounds__(G < 256 ? 256 : G)
block_norm_fwd_kernel(BlockNormArgs a) {
  using Map = RowMap<T, G, E>;
  constexpr int kPer = G < 256 ? 256 / G : 1;
  __shared__ float lds[64];
  const int dim = static_cast<int>(a.dim);
  const float inv = 1.f / dim;
  const bool layer = a.kind != 0;
  // parameters stay in registers over the rows
  float wpost[E], rs[E], wpre[E];
  Map::params(a.w_post, dim, 1.f, wpost);
  Map::params(a.res_scale, dim, 1.f, rs);
  Map::params(a.w_pre, dim, 0.f, wpre);
#pragma unroll
  for (int i = 0; i < E; ++i) wpost[i] *= rs[i];
  const int64_t steps = (a.n + kPer - 1) / kPer;
  for (int64_t it = blockIdx.x; it < steps; it += gridDim.x) {
    const int64_t row = it * kPer + threadIdx.x / G;
    const bool live = row < a.n;  // kPer > 1 implies G <= 128: whole groups are idle together
    const int d = live ? dim : 0;
    float f[E], x[E], gate[E], grow = 1.f;
    Map::load(static_cast<const T*>(a.f) + (live ? row * a.f_stride : 0), d, f);
    Map::load(static_cast<const T*>(a.x) + (live ? row * a.x_stride : 0), d, x);
    if (a.gate_mode == kGateElement) Map::load(static_cast<const T*>(a.gate) + (live ? row * a.gate_stride : 0), d, gate);
    if (a.gate_mode == kGateRow && live) {
      grow = static_cast<float>(static_cast<const T*>(a.gate)[row * a.gate_stride]);
      if (a.gate_act) grow = sigmoid(grow);
    }
    float mean = 0.f;
    if (layer) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < E; ++i) s[0] += f[i];
      row_sum<G, 1>(s, lds);
      mean = s[0] * inv;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) {
      f[i] = Map::on(i, d) ? f[i] - mean : 0.f;
      q[0] += f[i] * f[i];
    }
    row_sum<G, 1>(q, lds);
    const float rf = rsqrtf(q[0] * inv + a.eps) * grow;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      float b = f[i] * rf * wpost[i];
      if (a.gate_mode == kGateElement) b *= a.gate_act ? sigmoid(gate[i]) : gate[i];
      x[i] += b;
    }
    T* y = static_cast<T*>(a.y) + (live ? row * a.dim : 0);
    Map::store(y, d, x);
    if (a.h) {
      mean = 0.f;
      if (layer) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) s[0] += Map::on(i, d) ? x[i] : 0.f;
        row_sum<G, 1>(s, lds);
        mean = s[0] * inv;
      }
      q[0] = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        x[i] = Map::on(i, d) ? x[i] - mean : 0.f;
        q[0] += x[i] * x[i];
      }
      row_sum<G, 1>(q, lds);
      const float ry = rsqrtf(q[0] * inv + a.eps);
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] *= ry * wpre[i];
      Map::store(static_cast<T*>(a.h) + (live ? row * a.dim : 0), d, x);
    }
  }
}

// Workgroup b takes the row groups b, b + gridDim.x, ...; its column sums go
// to partial row b of the workspace, [parts][3][dim] float32, and
// block_norm_fold_kernel adds the partial rows in order.
template <typename T, int G, int E>
__global__ void __launch_bounds__(G < 256 ? 256 : G)
block_norm_bwd_kernel(BlockNormArgs a) {
  using Map = RowMap<T, G, E>;
  constexpr int kPer = G < 256 ? 256 / G : 1;
  constexpr int kThreads = G < 256 ? 256 : G;
  __shared__ float lds[96];
  __shared__ float fold[kPer > 1 ? kThreads * E : 1];
  const int dim = static_cast<int>(a.dim);
  const float inv = 1.f / dim;
  const bool layer = a.kind != 0, next = a.w_pre != nullptr;
  float spost[E] = {}, sscale[E] = {}, spre[E] = {};
  const int64_t steps = (a.n + kPer - 1) / kPer;
  for (int64_t it = blockIdx.x; it < steps; it += gridDim.x) {
    const int64_t row = it * kPer + threadIdx.x / G;
    const bool live = row < a.n;
    const int d = live ? dim : 0;
    float f[E], dy[E], gate[E], grow = 1.f, act_row = 1.f;
    Map::load(static_cast<const T*>(a.f) + (live ? row * a.f_stride : 0), d, f);
    Map::load(static_cast<const T*>(a.gy) + (live ? row * a.gy_stride : 0), d, dy);
    if (a.gate_mode == kGateElement) Map::load(static_cast<const T*>(a.gate) + (live ? row * a.gate_stride : 0), d, gate);
    if (a.gate_mode == kGateRow && live) {
      grow = static_cast<float>(static_cast<const T*>(a.gate)[row * a.gate_stride]);
      if (a.gate_act) {
        grow = sigmoid(grow);
        act_row = grow * (1.f - grow);
      }
    }
    float s1[3] = {0.f, 0.f, 0.f};  // sums of f, y, q = gh * w_pre
    float s2[3] = {0.f, 0.f, 0.f};  // of (f - m)^2, (y - m)^2, q (y - m)
    if (next) {
      float y[E], q[E], gh[E], wpre[E];
      Map::load(static_cast<const T*>(a.x) + (live ? row * a.x_stride : 0), d, y);
      Map::load(static_cast<const T*>(a.gh) + (live ? row * a.gh_stride : 0), d, gh);
      Map::params(a.w_pre, dim, 0.f, wpre);
#pragma unroll
      for (int i = 0; i < E; ++i) q[i] = gh[i] * wpre[i];
      if (layer) {
#pragma unroll
        for (int i = 0; i < E; ++i) s1[0] += f[i], s1[1] += y[i], s1[2] += q[i];
        row_sum<G, 3>(s1, lds);
      }
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const bool on = Map::on(i, d);
        f[i] = on ? f[i] - s1[0] * inv : 0.f;
        y[i] = on ? y[i] - s1[1] * inv : 0.f;
        s2[0] += f[i] * f[i];
        s2[1] += y[i] * y[i];
        s2[2] += q[i] * y[i];
      }
      row_sum<G, 3>(s2, lds);
      const float ry = rsqrtf(s2[1] * inv + a.eps);
      const float k = s2[2] * inv * ry * ry, mq = s1[2] * inv;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        dy[i] += (q[i] - y[i] * k - mq) * ry;
        spre[i] += gh[i] * (y[i] * ry);
      }
    } else {
      if (layer) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) s[0] += f[i];
        row_sum<G, 1>(s, lds);
        s1[0] = s[0];
      }
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < E; ++i) {
        f[i] = Map::on(i, d) ? f[i] - s1[0] * inv : 0.f;
        s[0] += f[i] * f[i];
      }
      row_sum<G, 1>(s, lds);
      s2[0] = s[0];
    }
    Map::store(static_cast<T*>(a.gx) + (live ? row * a.dim : 0), d, dy);
    const float rf = rsqrtf(s2[0] * inv + a.eps);
    float wpost[E], rs[E];
    Map::params(a.w_post, dim, 1.f, wpost);
    Map::params(a.res_scale, dim, 1.f, rs);
    float s3[3] = {0.f, 0.f, 0.f};  // sums of p = dy rs gate w_post, p f, dy rs v
    float dg[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const bool on = Map::on(i, d);
      const float nf = f[i] * rf, v = nf * wpost[i];
      float g = grow, dact = 1.f;
      if (a.gate_mode == kGateElement) {
        g = gate[i];
        if (a.gate_act) {
          g = sigmoid(g);
          dact = g * (1.f - g);
        }
      }
      const float e = on ? dy[i] : 0.f;
      sscale[i] += e * g * v;
      const float er = e * rs[i];
      dg[i] = er * v * dact;
      s3[2] += dg[i];
      spost[i] += er * g * nf;
      dy[i] = er * g * wpost[i];
      s3[0] += dy[i];
      s3[1] += dy[i] * f[i];
    }
    if (a.gate_mode == kGateElement) Map::store(static_cast<T*>(a.ggate) + (live ? row * a.dim : 0), d, dg);
    row_sum<G, 3>(s3, lds);
    if (a.gate_mode == kGateRow && live && threadIdx.x % G == 0)
      static_cast<T*>(a.ggate)[row] = static_cast<T>(s3[2] * act_row);
    const float k = s3[1] * inv * rf * rf, mp = layer ? s3[0] * inv : 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) dy[i] = (dy[i] - f[i] * k - mp) * rf;
    Map::store(static_cast<T*>(a.gf) + (live ? row * a.dim : 0), d, dy);
  }
  float* part = static_cast<float*>(a.workspace) + static_cast<int64_t>(blockIdx.x) * 3 * dim;
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    float(&v)[E] = s == 0 ? spost : s == 1 ? sscale : spre;
    if constexpr (kPer > 1) {  // the row groups of the workgroup, in order
      __syncthreads();
#pragma unroll
      for (int i = 0; i < E; ++i) fold[i * kThreads + threadIdx.x] = v[i];
      __syncthreads();
      if (threadIdx.x < G)
        for (int q = 1; q < kPer; ++q)
#pragma unroll
          for (int i = 0; i < E; ++i) v[i] += fold[i * kThreads + q * G + threadIdx.x];
    }
    if (threadIdx.x < G) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = Map::col(i / Map::V) + i % Map::V;
        if (c < dim) part[s * dim + c] = v[i];
      }
    }
  }
}

// column sums of the partial rows: 16 columns by 64 interleaved row sets per
// workgroup, the sets added in order
__global__ void __launch_bounds__(1024)
block_norm_fold_kernel(const float* __restrict__ partial, int64_t parts, int64_t dim, float* __restrict__ gpost,
                       float* __restrict__ gscale, float* __restrict__ gpre) {
  __shared__ float lds[64 * 17];
  float* out = blockIdx.y == 0 ? gpost : blockIdx.y == 1 ? gscale : gpre;
  if (!out) return;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 16 + threadIdx.x % 16;
  const int set = threadIdx.x / 16;
  float s = 0.f;
  if (c < dim) {
#pragma unroll 4
    for (int64_t p = set; p < parts; p += 64) s += partial[(p * 3 + blockIdx.y) * dim + c];
  }
  lds[set * 17 + threadIdx.x % 16] = s;
  __syncthreads();
  if (threadIdx.x < 16 && c < dim) {
    float t = 0.f;
    for (int q = 0; q < 64; ++q) t += lds[q * 17 + threadIdx.x];
    out[c] = t;
  }
}

template <typename T, int G, int E>
int block_norm_launch(const BlockNormArgs& a, bool backward) {
  constexpr int kThreads = G < 256 ? 256 : G;
  constexpr int kPer = kThreads / G;
  const hipStream_t st = static_cast<hipStream_t>(a.stream);
  if (!backward) {
    const int64_t steps = (a.n + kPer - 1) / kPer;
    const int64_t grid = std::min<int64_t>(steps, 256 * (2048 / kThreads));
    hipLaunchKernelGGL((block_norm_fwd_kernel<T, G, E>), dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, st, a);
    return static_cast<int>(hipGetLastError());
  }
  hipLaunchKernelGGL((block_norm_bwd_kernel<T, G, E>), dim3(static_cast<unsigned>(a.parts)), dim3(kThreads), 0, st, a);
  hipLaunchKernelGGL(block_norm_fold_kernel, dim3(static_cast<unsigned>((a.dim + 15) / 16), 3), dim3(1024), 0, st,
                     static_cast<const float*>(a.workspace), a.parts, a.dim, a.gpost, a.gscale, a.gpre);
  return static_cast<int>(hipGetLastError());
}

template <typename T>
int block_norm_rows(const BlockNormArgs& a, bool backward) {
  if (a.dim <= 128) return block_norm_launch<T, 16, 8>(a, backward);
  if (a.dim <= 256) return block_norm_launch<T, 32, 8>(a, backward);
  if (a.dim <= 512) return block_norm_launch<T, 64, 8>(a, backward);
  if (a.dim <= 1024) return block_norm_launch<T, 128, 8>(a, backward);
  if (a.dim <= 2048) return block_norm_launch<T, 256, 8>(a, backward);
  if (a.dim <= 4096) return block_norm_launch<T, 512, 8>(a, backward);
  if (a.dim <= 8192) return block_norm_launch<T, 1024, 8>(a, backward);
  return block_norm_launch<T, 1024, 16>(a, backward);
}

int block_norm_any(const BlockNormArgs& a, bool backward) {
  if (a.dtype == kChBF16) return block_norm_rows<bf16>(a, backward);
  if (a.dtype == kChF16) return block_norm_rows<f16>(a, backward);
  return block_norm_rows<float>(a, backward);
}

}  // namespace kern

int launch_block_norm_fwd(const BlockNormArgs& a) { return kern::block_norm_any(a, false); }
int launch_block_norm_bwd(const BlockNormArgs& a) { return kern::block_norm_any(a, true); }

}  // namespace segpoly
