// C ABI of the invariant-channel operators: embedding lookup, block norm,
// gated feed-forward, each with its backward.  Host code.
#include <hip/hip_runtime_api.h>

#include <string>

#include "capi_channel.hpp"
#include "channel_ops.hpp"
#include "segpoly.h"

using namespace segpoly;

namespace {

int check_embedding(int dtype, int idx_dtype, int64_t rows, int64_t dim, int64_t n) {
  int rc = check_dtype(dtype);
  if (rc) return rc;
  if (idx_dtype != SEGPOLY_I32 && idx_dtype != SEGPOLY_I64) return fail(SEGPOLY_E_INVALID, "bad index dtype");
  if (rows < 0 || dim < 0 || n < 0) return fail(SEGPOLY_E_INVALID, "negative size");
  if (rows >= kMaxGridX - 1 || n >= kMaxGridX || dim > kMaxWidth)
    return fail(SEGPOLY_E_UNSUPPORTED, "too many rows or tokens, or rows too wide");
  return SEGPOLY_OK;
}

int check_norm(int dtype, int kind, int gate_mode, int gate_act, double eps, int64_t n, int64_t dim) {
  int rc = check_dtype(dtype);
  if (rc) return rc;
  if (kind != SEGPOLY_NORM_RMS && kind != SEGPOLY_NORM_LAYER) return fail(SEGPOLY_E_INVALID, "bad norm kind");
  if (gate_mode < SEGPOLY_GATE_NONE || gate_mode > SEGPOLY_GATE_ELEMENT) return fail(SEGPOLY_E_INVALID, "bad gate mode");
  if (gate_act != SEGPOLY_GATE_ACT_NONE && gate_act != SEGPOLY_GATE_ACT_SIGMOID)
    return fail(SEGPOLY_E_INVALID, "bad gate activation");
  if (!(eps >= 0)) return fail(SEGPOLY_E_INVALID, "eps must not be negative");
  if (n < 0 || dim < 0) return fail(SEGPOLY_E_INVALID, "negative size");
  if (dim > kBlockNormMaxDim) return fail(SEGPOLY_E_UNSUPPORTED, "rows wider than 16384");
  if (n >= kMaxGridX) return fail(SEGPOLY_E_UNSUPPORTED, "too many rows");
  return SEGPOLY_OK;
}

int check_ffn(int dtype, int act, int64_t n, int64_t d_in, int64_t hidden, int64_t d_out) {
  int rc = check_dtype(dtype);
  if (rc) return rc;
  if (act < SEGPOLY_ACT_SILU || act > SEGPOLY_ACT_SIGMOID) return fail(SEGPOLY_E_INVALID, "bad activation");
  if (n < 0) return fail(SEGPOLY_E_INVALID, "negative size");
  if (d_in < 1 || hidden < 1 || d_out < 1) return fail(SEGPOLY_E_INVALID, "widths must be positive");
  if (d_in > kMaxWidth || hidden > kMaxWidth || d_out > kMaxWidth || n >= kMaxGridX)
    return fail(SEGPOLY_E_UNSUPPORTED, "widths above 2^21 or too many rows");
  return SEGPOLY_OK;
}

}  // namespace

extern "C" {

int embedding_fwd(int dtype, const void* table, int64_t rows, int64_t dim, const void* tokens, int idx_dtype,
                  int64_t n, double scale, void* out, int64_t out_stride, void* stream) {
  int rc = check_embedding(dtype, idx_dtype, rows, dim, n);
  if (rc) return rc;
  if (out_stride < dim) return fail(SEGPOLY_E_INVALID, "out_stride below dim");
  if (n == 0 || dim == 0) return ok();
  if ((rows && !table) || !tokens || !out) return fail(SEGPOLY_E_INVALID, "null buffer");
  if ((rc = check_aligned(channel_dtype_bytes(dtype), {table, out}))) return rc;
  if ((rc = check_aligned(index_bytes(idx_dtype), {tokens}))) return rc;
  EmbeddingArgs a{};
  a.table = table, a.tokens = tokens, a.out = out, a.rows = rows, a.dim = dim, a.n = n, a.out_stride = out_stride;
  a.scale = static_cast<float>(scale), a.dtype = dtype, a.idx = idx_dtype, a.stream = stream;
  return launched(launch_embedding_fwd(a), "embedding");
}

int embedding_bwd_workspace(int64_t n, int64_t rows, int64_t dim, size_t* bytes) {
  if (!bytes) return fail(SEGPOLY_E_INVALID, "null bytes");
  int rc = check_embedding(SEGPOLY_F32, SEGPOLY_I32, rows, dim, n);
  if (rc) return rc;
  *bytes = rows == 0 || dim == 0 ? 0 : embedding_plan(n, rows, dim).bytes;
  return ok();
}

int embedding_bwd(int dtype, const void* grad_out, int64_t grad_stride, const void* tokens, int idx_dtype, int64_t n,
                  int64_t rows, int64_t dim, double scale, void* grad_table, void* workspace, size_t workspace_bytes,
                  void* stream) {
  int rc = check_embedding(dtype, idx_dtype, rows, dim, n);
  if (rc) return rc;
  if (grad_stride < 0) return fail(SEGPOLY_E_INVALID, "negative stride");
  if (rows == 0 || dim == 0) return ok();
  if (!grad_table || (n && (!grad_out || !tokens))) return fail(SEGPOLY_E_INVALID, "null buffer");
  if ((rc = check_aligned(channel_dtype_bytes(dtype), {grad_table, grad_out}))) return rc;
  if ((rc = check_aligned(index_bytes(idx_dtype), {tokens}))) return rc;
  rc = check_workspace(workspace, workspace_bytes, embedding_plan(n, rows, dim).bytes);
  if (rc) return rc;
  EmbeddingArgs a{};
  a.grad = grad_out, a.tokens = tokens, a.out = grad_table, a.rows = rows, a.dim = dim, a.n = n;
  a.grad_stride = grad_stride, a.scale = static_cast<float>(scale), a.dtype = dtype, a.idx = idx_dtype;
  a.workspace = workspace, a.stream = stream;
  return launched(launch_embedding_bwd(a), "embedding gradient");
}

int block_norm_fwd(int dtype, int kind, int gate_mode, int gate_act, const void* x, int64_t x_stride, const void* f,
                   int64_t f_stride, const void* gate, int64_t gate_stride, const void* w_post, const void* res_scale,
                   const void* w_pre, double eps, int64_t n, int64_t dim, void* y, void* h, void* stream) {
  int rc = check_norm(dtype, kind, gate_mode, gate_act, eps, n, dim);
  if (rc) return rc;
  if (x_stride < 0 || f_stride < 0 || gate_stride < 0) return fail(SEGPOLY_E_INVALID, "negative stride");
  if (n == 0 || dim == 0) return ok();
  if (!x || !f || !w_post || !y || (gate_mode != SEGPOLY_GATE_NONE && !gate))
    return fail(SEGPOLY_E_INVALID, "null buffer");
  if ((w_pre != nullptr) != (h != nullptr)) return fail(SEGPOLY_E_INVALID, "w_pre and h come together");
  if ((rc = check_aligned(channel_dtype_bytes(dtype), {x, f, gate, y, h}))) return rc;
  if ((rc = check_aligned(4, {w_post, res_scale, w_pre}))) return rc;
  BlockNormArgs a{};
  a.x = x, a.f = f, a.gate = gate, a.w_post = static_cast<const float*>(w_post);
  a.res_scale = static_cast<const float*>(res_scale), a.w_pre = static_cast<const float*>(w_pre), a.y = y, a.h = h;
  a.n = n, a.dim = dim, a.x_stride = x_stride, a.f_stride = f_stride, a.gate_stride = gate_stride;
  a.eps = static_cast<float>(eps), a.dtype = dtype, a.kind = kind, a.gate_mode = gate_mode, a.gate_act = gate_act;
  a.stream = stream;
  return launched(launch_block_norm_fwd(a), "block norm");
}

int block_norm_bwd_workspace(int64_t n, int64_t dim, size_t* bytes) {
  if (!bytes) return fail(SEGPOLY_E_INVALID, "null bytes");
  int rc = check_norm(SEGPOLY_F32, SEGPOLY_NORM_RMS, SEGPOLY_GATE_NONE, SEGPOLY_GATE_ACT_NONE, 0, n, dim);
  if (rc) return rc;
  *bytes = dim == 0 ? 0 : static_cast<size_t>(block_norm_parts(n, dim)) * 2 * dim * 4;
  return ok();
}

int block_norm_bwd(int dtype, int kind, int gate_mode, int gate_act, const void* y, int64_t y_stride, const void* grad_y,
                   int64_t grad_y_stride, const void* grad_h, int64_t grad_h_stride, const void* f, int64_t f_stride,
                   const void* gate, int64_t gate_stride, const void* w_post, const void* res_scale, const void* w_pre,
                   double eps, int64_t n, int64_t dim, void* grad_x, void* grad_f, void* grad_gate, void* grad_w_post,
                   void* grad_res_scale, void* grad_w_pre, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_norm(dtype, kind, gate_mode, gate_act, eps, n, dim);
  if (rc) return rc;
  if (y_stride < 0 || grad_y_stride < 0 || grad_h_stride < 0 || f_stride < 0 || gate_stride < 0)
    return fail(SEGPOLY_E_INVALID, "negative stride");
  if (dim == 0) return ok();
  if (!w_post || !grad_w_post || (res_scale && !grad_res_scale) || (w_pre && !grad_w_pre))
    return fail(SEGPOLY_E_INVALID, "null parameter or parameter gradient");
  if (n && (!grad_y || !f || !grad_x || !grad_f || (gate_mode != SEGPOLY_GATE_NONE && (!gate || !grad_gate)) ||
            (w_pre && (!y || !grad_h))))
    return fail(SEGPOLY_E_INVALID, "null buffer");
  if ((rc = check_aligned(channel_dtype_bytes(dtype), {y, grad_y, grad_h, f, gate, grad_x, grad_f, grad_gate}))) return rc;
  if ((rc = check_aligned(4, {w_post, res_scale, w_pre, grad_w_post, grad_res_scale, grad_w_pre}))) return rc;
  const int64_t parts = block_norm_parts(n, dim);
  rc = check_workspace(workspace, workspace_bytes, static_cast<size_t>(parts) * 2 * dim * 4);
  if (rc) return rc;
  BlockNormArgs a{};
  a.x = y, a.gy = grad_y, a.gh = grad_h, a.f = f, a.gate = gate, a.w_post = static_cast<const float*>(w_post);
  a.res_scale = static_cast<const float*>(res_scale), a.w_pre = static_cast<const float*>(w_pre);
  a.gx = grad_x, a.gf = grad_f, a.ggate = grad_gate, a.gpost = static_cast<float*>(grad_w_post);
  a.gscale = res_scale ? static_cast<float*>(grad_res_scale) : nullptr;
  a.gpre = w_pre ? static_cast<float*>(grad_w_pre) : nullptr;
  a.n = n, a.dim = dim, a.x_stride = y_stride, a.gy_stride = grad_y_stride, a.gh_stride = grad_h_stride;
  a.f_stride = f_stride, a.gate_stride = gate_stride, a.eps = static_cast<float>(eps), a.dtype = dtype, a.kind = kind;
  a.gate_mode = gate_mode, a.gate_act = gate_act, a.workspace = workspace, a.parts = parts, a.stream = stream;
  return launched(launch_block_norm_bwd(a), "block norm gradient");
}

int gated_ffn_workspace(int dtype, int64_t n, int64_t d_in, int64_t hidden, int64_t d_out, int backward,
                        size_t* bytes) {
  if (!bytes) return fail(SEGPOLY_E_INVALID, "null bytes");
  int rc = check_ffn(dtype, SEGPOLY_ACT_SILU, n, d_in, hidden, d_out);
  if (rc) return rc;
  *bytes = gated_ffn_workspace_bytes(dtype, n, d_in, hidden, d_out, backward != 0);
  return ok();
}

int gated_ffn_fwd(int dtype, int act, const void* x, int64_t x_stride, const void* w_gate, const void* w_up,
                  const void* w_down, int64_t n, int64_t d_in, int64_t hidden, int64_t d_out, void* out,
                  int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_ffn(dtype, act, n, d_in, hidden, d_out);
  if (rc) return rc;
  x_stride = row_stride(n, x_stride, d_in);
  if (x_stride < 0 || x_stride > kMaxWidth || out_stride < d_out) return fail(SEGPOLY_E_INVALID, "bad row stride");
  if (n == 0) return ok();
  if (!x || !w_gate || !w_up || !w_down || !out) return fail(SEGPOLY_E_INVALID, "null buffer");
  if ((rc = check_aligned(channel_dtype_bytes(dtype), {x, w_gate, w_up, w_down, out}))) return rc;
  rc = check_workspace(workspace, workspace_bytes,
                       gated_ffn_workspace_bytes(dtype, n, d_in, hidden, d_out, false));
  if (rc) return rc;
  GatedFfnArgs a{};
  a.x = x, a.w_gate = w_gate, a.w_up = w_up, a.w_down = w_down, a.out = out, a.n = n, a.d_in = d_in;
  a.hidden = hidden, a.d_out = d_out, a.x_stride = x_stride, a.out_stride = out_stride, a.dtype = dtype, a.act = act;
  a.workspace = workspace, a.stream = stream;
  return launched(launch_gated_ffn_fwd(a), "gated feed-forward");
}

int gated_ffn_bwd(int dtype, int act, const void* x, int64_t x_stride, const void* w_gate, const void* w_up,
                  const void* w_down, const void* grad_out, int64_t grad_out_stride, int64_t n, int64_t d_in,
                  int64_t hidden, int64_t d_out, void* grad_x, void* grad_w_gate, void* grad_w_up, void* grad_w_down,
                  void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_ffn(dtype, act, n, d_in, hidden, d_out);
  if (rc) return rc;
  x_stride = row_stride(n, x_stride, d_in);
  grad_out_stride = row_stride(n, grad_out_stride, d_out);
  if (x_stride < 0 || x_stride > kMaxWidth || grad_out_stride < 0 || grad_out_stride > kMaxWidth)
    return fail(SEGPOLY_E_INVALID, "bad row stride");
  if (n && (!x || !w_gate || !w_up || !w_down || !grad_out)) return fail(SEGPOLY_E_INVALID, "null buffer");
  const int weights = (grad_w_gate != nullptr) + (grad_w_up != nullptr) + (grad_w_down != nullptr);
  if (weights != 0 && weights != 3) return fail(SEGPOLY_E_INVALID, "the three weight gradients come together");
  if (!weights && !grad_x) return fail(SEGPOLY_E_INVALID, "no gradient requested");
  if ((rc = check_aligned(channel_dtype_bytes(dtype), {x, w_gate, w_up, w_down, grad_out, grad_x, grad_w_gate, grad_w_up,
                                                       grad_w_down})))
    return rc;
  rc = check_workspace(workspace, workspace_bytes, gated_ffn_workspace_bytes(dtype, n, d_in, hidden, d_out, true));
  if (rc) return rc;
  GatedFfnArgs a{};
  a.x = x, a.w_gate = w_gate, a.w_up = w_up, a.w_down = w_down, a.gout = grad_out, a.gx = grad_x;
  a.gw_gate = grad_w_gate, a.gw_up = grad_w_up, a.gw_down = grad_w_down, a.n = n, a.d_in = d_in, a.hidden = hidden;
  a.d_out = d_out, a.x_stride = x_stride, a.gout_stride = grad_out_stride, a.dtype = dtype, a.act = act;
  a.workspace = workspace, a.stream = stream;
  return launched(launch_gated_ffn_bwd(a), "gated feed-forward gradient");
}

}  // extern "C"
