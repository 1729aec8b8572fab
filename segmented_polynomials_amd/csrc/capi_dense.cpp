// C ABI of the dense layer.  Host code.
#include <hip/hip_runtime_api.h>

#include <algorithm>

#include "capi_channel.hpp"
#include "channel_ops.hpp"
#include "segpoly.h"

using namespace segpoly;

namespace {

int check_dense(int dtype, int act, int64_t n, int64_t d_in, int64_t d_out) {
  int rc = check_dtype(dtype);
  if (rc) return rc;
  if (act < SEGPOLY_ACT_SILU || act > SEGPOLY_ACT_NONE) return fail(SEGPOLY_E_INVALID, "bad activation");
  if (n < 0) return fail(SEGPOLY_E_INVALID, "negative size");
  if (d_in < 1 || d_out < 1) return fail(SEGPOLY_E_INVALID, "widths must be positive");
  if (d_in > kMaxWidth || d_out > kMaxWidth || n >= kMaxGridX)
    return fail(SEGPOLY_E_UNSUPPORTED, "widths above 2^21 or too many rows");
  // a launch has fewer than 2^32 threads: 2^24 workgroups of 256, of tiles of 64 x 64
  const auto tiles = [](int64_t v) { return (v + 63) / 64; };
  const int64_t wide = tiles(std::max(d_in, d_out));
  if (tiles(n) * wide >= int64_t{1} << 24 || tiles(d_in) * tiles(d_out) >= int64_t{1} << 24)
    return fail(SEGPOLY_E_UNSUPPORTED, "more than 2^24 tiles of 64 x 64");
  return SEGPOLY_OK;
}

}  // namespace

extern "C" {

int dense_workspace(int dtype, int act, int64_t n, int64_t d_in, int64_t d_out, int backward, size_t* bytes) {
  if (!bytes) return fail(SEGPOLY_E_INVALID, "null bytes");
  int rc = check_dense(dtype, act, n, d_in, d_out);
  if (rc) return rc;
  *bytes = dense_workspace_bytes(dtype, act, n, d_in, d_out, backward != 0);
  return ok();
}

int dense_fwd(int dtype, int act, const void* x, int64_t x_stride, const void* w, const void* bias, const void* residual,
              int64_t residual_stride, int64_t n, int64_t d_in, int64_t d_out, void* out, int64_t out_stride,
              void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_dense(dtype, act, n, d_in, d_out);
  if (rc) return rc;
  x_stride = row_stride(n, x_stride, d_in);
  if (x_stride < 0 || x_stride > kMaxWidth || residual_stride < 0 || out_stride < d_out)
    return fail(SEGPOLY_E_INVALID, "bad row stride");
  if (n == 0) return ok();
  if (!x || !w || !out) return fail(SEGPOLY_E_INVALID, "null buffer");
  if ((rc = check_aligned(channel_dtype_bytes(dtype), {x, w, bias, residual, out}))) return rc;
  rc = check_workspace(workspace, workspace_bytes, dense_workspace_bytes(dtype, act, n, d_in, d_out, false));
  if (rc) return rc;
  DenseArgs a{};
  a.x = x, a.w = w, a.bias = bias, a.residual = residual, a.out = out, a.n = n, a.d_in = d_in, a.d_out = d_out;
  a.x_stride = x_stride, a.residual_stride = residual_stride, a.out_stride = out_stride, a.dtype = dtype, a.act = act;
  a.workspace = workspace, a.stream = stream;
  return launched(launch_dense_fwd(a), "dense layer");
}

int dense_bwd(int dtype, int act, const void* x, int64_t x_stride, const void* w, const void* bias, const void* grad_out,
              int64_t grad_out_stride, int64_t n, int64_t d_in, int64_t d_out, void* grad_x, void* grad_w,
              void* grad_bias, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_dense(dtype, act, n, d_in, d_out);
  if (rc) return rc;
  x_stride = row_stride(n, x_stride, d_in);
  grad_out_stride = row_stride(n, grad_out_stride, d_out);
  if (x_stride < 0 || x_stride > kMaxWidth || grad_out_stride < 0 || grad_out_stride > kMaxWidth)
    return fail(SEGPOLY_E_INVALID, "bad row stride");
  if (n && (!x || !w || !grad_out)) return fail(SEGPOLY_E_INVALID, "null buffer");
  if (!grad_x && !grad_w && !grad_bias) return fail(SEGPOLY_E_INVALID, "no gradient requested");
  if ((rc = check_aligned(channel_dtype_bytes(dtype), {x, w, bias, grad_out, grad_x, grad_w, grad_bias}))) return rc;
  rc = check_workspace(workspace, workspace_bytes, dense_workspace_bytes(dtype, act, n, d_in, d_out, true));
  if (rc) return rc;
  DenseArgs a{};
  a.x = x, a.w = w, a.bias = bias, a.gout = grad_out, a.gx = grad_x, a.gw = grad_w, a.gbias = grad_bias, a.n = n;
  a.d_in = d_in, a.d_out = d_out, a.x_stride = x_stride, a.gout_stride = grad_out_stride, a.dtype = dtype, a.act = act;
  a.workspace = workspace, a.stream = stream;
  return launched(launch_dense_bwd(a), "dense layer gradient");
}

}  // extern "C"
