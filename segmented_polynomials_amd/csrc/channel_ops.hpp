// Arguments of the invariant-channel kernels (embedding, block norm, gated
// feed-forward): host and device.
#pragma once
#include <cstddef>
#include <cstdint>

namespace segpoly {

// dtype codes of the C ABI that the invariant-channel operators take
enum : int { kChF32 = 0, kChBF16 = 2, kChF16 = 3 };

inline int64_t channel_dtype_bytes(int dtype) { return dtype == kChF32 ? 4 : 2; }
inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

struct EmbeddingArgs {
  const void* table;   // forward
  const void* grad;    // backward: [n, dim], row stride grad_stride
  const void* tokens;
  void* out;           // forward: [n, dim], row stride out_stride; backward: [rows, dim]
  int64_t rows, dim, n, out_stride, grad_stride;
  float scale;
  int dtype, idx;
  void* workspace;     // backward
  void* stream;
};

// Sorted positions per uniform chunk of the embedding gradient.
constexpr int kEmbChunk = 16;
// Tokens one workgroup ranks in a sorting pass.
constexpr int kEmbSortBlock = 4096;
// Counts of this many sorting workgroups and more are added up by a kernel of their
// own.  64 columns bf16 of 200000 rows, one MI355X, by each workgroup and by the kernel:
// 300000 tokens (74 workgroups) 90 and 91 us, 524288 (128) 111 and 105, 2^24 6227 and 2971.
constexpr int64_t kEmbScanBlocks = 128;
// Lists up to this many tokens into up to this many rows are ordered in one
// launch: kEmbGroups workgroups, group w those of the rows r = w modulo kEmbGroups.
constexpr int kEmbGroups = 256;
constexpr int64_t kEmbOrderTokens = 32768;
constexpr int64_t kEmbOrderRows = 512 * kEmbGroups;
// Tables of at most this many rows are summed in LDS, without a sort: as many as
// have 1024 columns in 64 KB.  16 rows, one MI355X, us in LDS and sorted: 16384 tokens
// of 64 bf16 11 and 24, of 1024 bf16 45 and 42 (a text's 67); 100000 14 and 39, 120
// and 118 (283).
constexpr int kEmbDirectRows = 16;

// Device workspace of the embedding gradient, as byte offsets.
struct EmbeddingPlan {
  int64_t segments;  // of positions, of a table summed in LDS; else 0
  // Row r has range (r % groups) * per_group + r / groups of the sorted list.
  int groups;              // kEmbGroups for a list ordered in one launch, else 1
  int64_t per_group, keys;  // keys: ranges, and the key of a token out of range
  int bits, passes, digit_bits;
  int64_t blocks, chunks;
  size_t key[2], pos[2], hist, rowptr, partial, bytes;
};
EmbeddingPlan embedding_plan(int64_t n, int64_t rows, int64_t dim);

int launch_embedding_fwd(const EmbeddingArgs& a);
int launch_embedding_bwd(const EmbeddingArgs& a);

struct BlockNormArgs {
  const void *x, *f, *gate;
  const float *w_post, *res_scale, *w_pre;
  const void *gy, *gh;
  void *y, *h;                  // forward outputs
  void *gx, *gf, *ggate;        // backward outputs
  float *gpost, *gscale, *gpre;
  int64_t n, dim;
  int64_t x_stride, f_stride, gate_stride, gy_stride, gh_stride;  // of inputs; outputs are contiguous
  float eps;
  int dtype, kind, gate_mode, gate_act;
  void* workspace;              // backward
  int64_t parts;
  void* stream;
};
// widest row one workgroup holds in registers
constexpr int64_t kBlockNormMaxDim = 16384;
// workgroups of the backward's row loop = partial rows of its column sums
int64_t block_norm_parts(int64_t n, int64_t dim);
int launch_block_norm_fwd(const BlockNormArgs& a);
int launch_block_norm_bwd(const BlockNormArgs& a);

enum : int { kActSilu = 0, kActGelu = 1, kActRelu = 2, kActSigmoid = 3 };

struct GatedFfnArgs {
  const void *x, *w_gate, *w_up, *w_down;  // [n, d_in], [hidden, d_in] twice, [d_out, hidden]
  const void* gout;                        // backward: [n, d_out]
  void* out;                               // forward: [n, d_out]
  void *gx, *gw_gate, *gw_up, *gw_down;    // backward, contiguous
  int64_t n, d_in, hidden, d_out;
  int64_t x_stride, gout_stride, out_stride;
  int dtype, act;
  void* workspace;
  void* stream;
};
// workspace bytes for any strides and alignments of these sizes; none for no rows
size_t gated_ffn_workspace_bytes(int dtype, int64_t n, int64_t d_in, int64_t hidden, int64_t d_out, bool backward);
int launch_gated_ffn_fwd(const GatedFfnArgs& a);
int launch_gated_ffn_bwd(const GatedFfnArgs& a);

}  // namespace segpoly
