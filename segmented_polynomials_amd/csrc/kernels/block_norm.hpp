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
// registers).  G lanes hold one row, E = 8 elements per lane while the row
// fits in a workgroup; up to 64 lanes the reductions need no barrier, so
// narrow rows share a wave.  One MI355X, bf16 with a gate per element: forward of
// 16384 x 2048 65 us, 5.2 TB/s; backward of 8192 x 4096 111 us, 4.8 TB/s (a copy of
// 1 GiB: 5.1).  Before the next row was loaded ahead and the parameters came by
// 16-byte loads, 98 and 373 us.  Above 4096 columns the backward has no registers
// for the next row: 4096 x 8192 115 us, 4.7 TB/s; above 8192 not for its own
// sixteen elements a lane: 2048 x 16384 436 us, 1.2 TB/s (forward 64 us).  Backward of
// 20000 x 128 float32: 17 us for 12 at the copy's rate, workgroups of two steps each,
// whose first loads and last sums nothing covers.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../channel_ops.hpp"
#include "../launch.hpp"
#include "channel_types.hpp"

namespace segpoly {

// Workgroups of a loop over `steps`: at most `most`, each with the same
// number of steps but the last.
int64_t block_norm_even_grid(int64_t steps, int64_t most);

namespace kern {

int block_norm_fold(const BlockNormArgs& a);

enum { kGateNone = 0, kGateRow = 1, kGateElement = 2 };

// Sums of K values over the G lanes of a row; every lane gets them.  `lds`
// holds two halves used in turn: a half is written again only after the
// barrier of the sum between, when all have read it.
template <int G, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* lds, int& half) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lane_sum<(G < 64 ? G : 64)>(v[k]);
  if constexpr (G > 64) {
    constexpr int W = G / 64;
    float* at = lds + half * 64 + threadIdx.x / G * W * K;
    half ^= 1;
    if (threadIdx.x % 64 == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) at[k * W + threadIdx.x / 64 % W] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lane_sum<W>(at[k * W + threadIdx.x % W]);
  }
}

// Lane l of a row holds the chunks c = l, l + G, ...: R chunks of V elements.
template <typename T, int G, int E>
struct RowMap {
  static constexpr int V = Chunk<T>::kN;
  static constexpr int R = E / V;
  u32x4 raw[R];
  __device__ __forceinline__ static int col(int r) { return (static_cast<int>(threadIdx.x % G) + r * G) * V; }
  __device__ __forceinline__ void load(const T* row, int dim) {
#pragma unroll
    for (int r = 0; r < R; ++r) raw[r] = load_raw(row, col(r), dim);
  }
  __device__ __forceinline__ void values(int dim, float (&v)[E]) const {
#pragma unroll
    for (int r = 0; r < R; ++r) unpack_chunk<T>(raw[r], col(r), dim, v + r * V);
  }
  __device__ __forceinline__ static void store(T* row, int dim, const float (&v)[E]) {
#pragma unroll
    for (int r = 0; r < R; ++r) store_chunk(row, col(r), dim, v + r * V);
  }
  // float32 parameters of the lane's columns, all ones without them
  __device__ __forceinline__ static void params(const float* p, int dim, float (&v)[E]) {
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      if (p)
        load_chunk(p, col(i / V) + i % V, dim, v + i);
      else
        v[i] = v[i + 1] = v[i + 2] = v[i + 3] = 1.f;
    }
  }
  // v - mean within the row, zero past its end
  __device__ __forceinline__ static void centre(float (&v)[E], float mean, int dim) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = col(i / V) < dim - i % V ? v[i] - mean : 0.f;
  }
};

// Elem: a gate per element.  The next row's chunks are loaded before the
// present row is worked on, so the loads of one row cover the reductions of
// another.
template <typename T, int G, int E, bool Elem, bool Layer>
__global__ void __launch_bounds__(G < 256 ? 256 : G)
block_norm_fwd_kernel(BlockNormArgs a) {
  using Map = RowMap<T, G, E>;
  constexpr int kPer = G < 256 ? 256 / G : 1;
  __shared__ float lds[128];
  int half = 0;
  const int dim = static_cast<int>(a.dim);
  const float inv = 1.f / dim;
  const int64_t steps = (a.n + kPer - 1) / kPer;
  Map rf, rx, rg;
  T row_gate = T(1.f);
  auto fetch = [&](int64_t it) {
    const int64_t row = it * kPer + threadIdx.x / G;
    const int d = row < a.n ? dim : 0;
    const int64_t at = row < a.n ? row : 0;
    rf.load(static_cast<const T*>(a.f) + at * a.f_stride, d);
    rx.load(static_cast<const T*>(a.x) + at * a.x_stride, d);
    if constexpr (Elem)
      rg.load(static_cast<const T*>(a.gate) + at * a.gate_stride, d);
    else if (a.gate_mode == kGateRow)
      row_gate = static_cast<const T*>(a.gate)[at * a.gate_stride];
  };
  int64_t it = blockIdx.x;
  fetch(it);  // the grid has at most `steps` workgroups
  float wpost[E], wpre[E];
  {
    float rs[E];
    Map::params(a.w_post, dim, wpost);
    Map::params(a.res_scale, dim, rs);
    Map::params(a.w_pre, dim, wpre);
#pragma unroll
    for (int i = 0; i < E; ++i) wpost[i] *= rs[i];
  }
  for (; it < steps; it += gridDim.x) {
    const int64_t row = it * kPer + threadIdx.x / G;
    const int d = row < a.n ? dim : 0;  // whole groups are idle together
    float f[E], x[E], gate[E], grow = static_cast<float>(row_gate);
    rf.values(d, f);
    rx.values(d, x);
    if constexpr (Elem) rg.values(d, gate);
    if (it + gridDim.x < steps) fetch(it + gridDim.x);
    if (a.gate_act) {
      if constexpr (Elem) {
#pragma unroll
        for (int i = 0; i < E; ++i) gate[i] = sigmoid(gate[i]);
      } else {
        grow = a.gate_mode == kGateRow ? sigmoid(grow) : 1.f;
      }
    }
    if constexpr (Layer) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < E; ++i) s[0] += f[i];
      row_sum<G, 1>(s, lds, half);
      Map::centre(f, s[0] * inv, d);
    }
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) q[0] += f[i] * f[i];
    row_sum<G, 1>(q, lds, half);
    const float rstd = rsqrtf(q[0] * inv + a.eps) * grow;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float b = f[i] * rstd * wpost[i];
      if constexpr (Elem)
        x[i] += b * gate[i];
      else
        x[i] += b;
    }
    const int64_t at = d ? row * a.dim : 0;
    Map::store(static_cast<T*>(a.y) + at, d, x);
    if (a.h) {
      if constexpr (Layer) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) s[0] += x[i];
        row_sum<G, 1>(s, lds, half);
        Map::centre(x, s[0] * inv, d);
      }
      q[0] = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) q[0] += x[i] * x[i];
      row_sum<G, 1>(q, lds, half);
      const float ry = rsqrtf(q[0] * inv + a.eps);
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] *= ry * wpre[i];
      Map::store(static_cast<T*>(a.h) + at, d, x);
    }
  }
}

// Workgroup b takes the row groups b, b + gridDim.x, ....  Two column sums
// serve the three parameters, S = sum of dy gate norm(f) and the sum of
// gh norm(y): grad w_post = res_scale S and grad res_scale = w_post S.  They go
// to partial row b of the workspace, [parts][2][dim] float32, and
// block_norm_fold_kernel adds the partial rows in order.
template <typename T, int G, int E, bool Elem, bool Layer>
__global__ void __launch_bounds__(G < 256 ? 256 : G, G < 512 ? 3 : 4)
block_norm_bwd_kernel(BlockNormArgs a) {
  using Map = RowMap<T, G, E>;
  constexpr int kPer = G < 256 ? 256 / G : 1;
  constexpr int kThreads = G < 256 ? 256 : G;
  __shared__ float lds[128];
  __shared__ float fold[kPer > 1 ? kThreads * E : 1];
  constexpr bool kAhead = G < 1024;  // a workgroup of 16 waves has no registers left for the next row
  int half = 0;
  const int dim = static_cast<int>(a.dim);
  const float inv = 1.f / dim;
  const bool next = a.w_pre != nullptr;  // else y and gh stay zero, and so does what comes of them
  const int64_t steps = (a.n + kPer - 1) / kPer;
  Map rf, rgy, rg, ry{}, rgh{};
  T row_gate = T(1.f);
  auto fetch = [&](int64_t it) {
    const int64_t row = it * kPer + threadIdx.x / G;
    const int d = row < a.n ? dim : 0;
    const int64_t at = row < a.n ? row : 0;
    rf.load(static_cast<const T*>(a.f) + at * a.f_stride, d);
    rgy.load(static_cast<const T*>(a.gy) + at * a.gy_stride, d);
    if (next) {
      ry.load(static_cast<const T*>(a.x) + at * a.x_stride, d);
      rgh.load(static_cast<const T*>(a.gh) + at * a.gh_stride, d);
    }
    if constexpr (Elem)
      rg.load(static_cast<const T*>(a.gate) + at * a.gate_stride, d);
    else if (a.gate_mode == kGateRow)
      row_gate = static_cast<const T*>(a.gate)[at * a.gate_stride];
  };
  int64_t it = blockIdx.x;
  if (kAhead && it < steps) fetch(it);  // no rows: the sums are zero
  float spost[E] = {}, spre[E] = {};
  // c = res_scale w_post and w_pre wait in LDS, four columns an access: the
  // registers they would take all the time hold the next row
  using F4 = float __attribute__((ext_vector_type(4)));
  __shared__ F4 param[2][E / 4][G];
  if (threadIdx.x < G) {
    float p[E], rs[E];
    Map::params(a.w_post, dim, p);
    Map::params(a.res_scale, dim, rs);
#pragma unroll
    for (int i = 0; i < E; ++i) param[0][i / 4][threadIdx.x][i % 4] = p[i] * rs[i];
    Map::params(a.w_pre, dim, p);
#pragma unroll
    for (int i = 0; i < E; ++i) param[1][i / 4][threadIdx.x][i % 4] = p[i];
  }
  __syncthreads();
  auto param_at = [&](int which, float(&v)[E]) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const F4 q = param[which][i][threadIdx.x % G];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i * 4 + j] = q[j];
    }
  };
  for (; it < steps; it += gridDim.x) {
    const int64_t row = it * kPer + threadIdx.x / G;
    const int d = row < a.n ? dim : 0;
    const int64_t at = d ? row * a.dim : 0;
    if constexpr (!kAhead) fetch(it);
    float f[E], dy[E], y[E], gh[E], gate[E], grow = static_cast<float>(row_gate), act_row = 1.f;
    rf.values(d, f);
    rgy.values(d, dy);
    ry.values(d, y);
    rgh.values(d, gh);
    if constexpr (Elem) rg.values(d, gate);
    if (kAhead && it + gridDim.x < steps) fetch(it + gridDim.x);
    if (!Elem && a.gate_mode == kGateRow && a.gate_act) {
      grow = sigmoid(grow);
      act_row = grow * (1.f - grow);
    }
    float q[E];
    param_at(1, q);
#pragma unroll
    for (int i = 0; i < E; ++i) q[i] *= gh[i];
    float s2[3] = {0.f, 0.f, 0.f};  // sums of (f - m)^2, (y - m)^2, q (y - m), with q = gh w_pre
    float mq = 0.f;
    if constexpr (Layer) {
      float s1[3] = {0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < E; ++i) s1[0] += f[i], s1[1] += y[i], s1[2] += q[i];
      row_sum<G, 3>(s1, lds, half);
      Map::centre(f, s1[0] * inv, d);
      Map::centre(y, s1[1] * inv, d);
      mq = s1[2] * inv;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      s2[0] += f[i] * f[i];
      s2[1] += y[i] * y[i];
      s2[2] += q[i] * y[i];
    }
    row_sum<G, 3>(s2, lds, half);
    {
      // zero without a row or a second norm: with eps = 0 the root of their zeros is
      // infinite, and its product with them NaN in the column sums of all rows
      const float ryv = next && d ? rsqrtf(s2[1] * inv + a.eps) : 0.f;
      const float k = s2[2] * inv * ryv * ryv;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        dy[i] += (q[i] - y[i] * k - mq) * ryv;
        spre[i] += gh[i] * (y[i] * ryv);
      }
    }
    Map::store(static_cast<T*>(a.gx) + at, d, dy);
    if constexpr (Layer) Map::centre(dy, 0.f, d);  // the means reached past the row's end
    const float rstd = d ? rsqrtf(s2[0] * inv + a.eps) : 0.f;
    float c[E];
    param_at(0, c);
    float s3[3] = {0.f, 0.f, 0.f};  // sums of p = dy c gate, p f, dy c norm(f)
    if constexpr (Elem) {
      float dg[E];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        float g = gate[i], dact = 1.f;
        if (a.gate_act) {
          g = sigmoid(g);
          dact = g * (1.f - g);
        }
        const float nf = f[i] * rstd, e = dy[i] * c[i];
        spost[i] += dy[i] * g * nf;
        dg[i] = e * nf * dact;
        dy[i] = e * g;
        s3[0] += dy[i];
        s3[1] += dy[i] * f[i];
      }
      Map::store(static_cast<T*>(a.ggate) + at, d, dg);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float nf = f[i] * rstd, e = dy[i] * c[i];
        spost[i] += dy[i] * grow * nf;
        s3[2] += e * nf;
        dy[i] = e * grow;
        s3[0] += dy[i];
        s3[1] += dy[i] * f[i];
      }
    }
    row_sum<G, 3>(s3, lds, half);
    if (!Elem && a.gate_mode == kGateRow && d && threadIdx.x % G == 0)
      static_cast<T*>(a.ggate)[row] = static_cast<T>(s3[2] * act_row);
    const float k = s3[1] * inv * rstd * rstd, mp = Layer ? s3[0] * inv : 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) dy[i] = (dy[i] - f[i] * k - mp) * rstd;
    Map::store(static_cast<T*>(a.gf) + at, d, dy);
  }
  float* part = static_cast<float*>(a.workspace) + static_cast<int64_t>(blockIdx.x) * 2 * dim;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float(&v)[E] = s == 0 ? spost : spre;
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
    if (threadIdx.x < G)
#pragma unroll
      for (int i = 0; i < E; i += 4) store_chunk(part + s * dim, Map::col(i / Map::V) + i % Map::V, dim, v + i);
  }
}

template <typename T, int G, int E, bool Elem, bool Layer>
int block_norm_launch(const BlockNormArgs& a, bool backward) {
  constexpr int kThreads = G < 256 ? 256 : G;
  constexpr int kPer = kThreads / G;
  const hipStream_t st = static_cast<hipStream_t>(a.stream);
  if (!backward) {
    const int64_t grid = block_norm_even_grid((a.n + kPer - 1) / kPer, 256 * (2048 / kThreads));
    hipLaunchKernelGGL((block_norm_fwd_kernel<T, G, E, Elem, Layer>), dim3(static_cast<unsigned>(grid)),
                       dim3(kThreads), 0, st, a);
    return static_cast<int>(hipGetLastError());
  }
  hipLaunchKernelGGL((block_norm_bwd_kernel<T, G, E, Elem, Layer>), dim3(static_cast<unsigned>(a.parts)),
                     dim3(kThreads), 0, st, a);
  const int rc = static_cast<int>(hipGetLastError());
  return rc ? rc : block_norm_fold(a);
}

template <typename T, int G, int E>
int block_norm_launch(const BlockNormArgs& a, bool backward) {
  if (a.gate_mode == kGateElement)
    return a.kind ? block_norm_launch<T, G, E, true, true>(a, backward)
                  : block_norm_launch<T, G, E, true, false>(a, backward);
  return a.kind ? block_norm_launch<T, G, E, false, true>(a, backward)
                : block_norm_launch<T, G, E, false, false>(a, backward);
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

}  // namespace kern
}  // namespace segpoly
