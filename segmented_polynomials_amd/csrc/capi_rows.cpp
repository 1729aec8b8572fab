// C ABI of dropout and of the routing of rows to experts.  Host code.
#include <hip/hip_runtime_api.h>

#include <cmath>

#include "capi_channel.hpp"
#include "channel_ops.hpp"
#include "segpoly.h"

using namespace segpoly;

namespace {

int check_sort(int64_t entries, int64_t num) {
  if (entries < 0 || num < 1) return fail(SEGPOLY_E_INVALID, "negative number of entries, or no expert");
  if (entries >= kMaxGridX) return fail(SEGPOLY_E_UNSUPPORTED, "too many entries");
  if (num > kMaxExperts) return fail(SEGPOLY_E_UNSUPPORTED, "more than 2048 experts");
  return SEGPOLY_OK;
}

int check_rows(int dtype, int64_t n, int64_t k, int64_t num, int64_t dim) {
  int rc = check_dtype(dtype);
  if (rc) return rc;
  if (n < 0 || dim < 0 || k < 1) return fail(SEGPOLY_E_INVALID, "negative size, or no choice a row");
  if (n >= kMaxGridX || k >= kMaxGridX || dim > kMaxWidth)
    return fail(SEGPOLY_E_UNSUPPORTED, "too many rows or choices, or rows too wide");
  return check_sort(n * k, num);
}

int dropout(int dtype, int mode, const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, double p,
            uint64_t seed, uint64_t offset, const void* state, int64_t n, int64_t dim, void* out, int64_t out_stride,
            void* stream) {
  int rc = check_dtype(dtype);
  if (rc) return rc;
  if (mode != SEGPOLY_DROPOUT_ELEMENT && mode != SEGPOLY_DROPOUT_ROW) return fail(SEGPOLY_E_INVALID, "bad dropout mode");
  if (!(p >= 0 && p <= 1)) return fail(SEGPOLY_E_INVALID, "p must be between 0 and 1");
  if (n < 0 || dim < 0) return fail(SEGPOLY_E_INVALID, "negative size");
  if (n >= kMaxGridX || dim > kMaxWidth) return fail(SEGPOLY_E_UNSUPPORTED, "too many rows, or rows too wide");
  if (x_stride < 0 || residual_stride < 0) return fail(SEGPOLY_E_INVALID, "negative stride");
  if (out_stride < dim) return fail(SEGPOLY_E_INVALID, "out_stride below dim");
  if (n == 0 || dim == 0) return ok();
  if (!x || !out) return fail(SEGPOLY_E_INVALID, "null buffer");
  if ((rc = check_aligned(channel_dtype_bytes(dtype), {x, residual, out}))) return rc;
  if ((rc = check_aligned(8, {state}))) return rc;
  DropoutArgs a{};
  a.x = x, a.residual = residual, a.out = out, a.n = n, a.dim = dim, a.x_stride = x_stride;
  a.residual_stride = residual_stride, a.out_stride = out_stride, a.seed = seed, a.offset = offset;
  a.state = static_cast<const int64_t*>(state);
  const double words = std::nearbyint(p * 4294967296.0);
  a.drop_all = words >= 4294967296.0;
  a.below = a.drop_all ? 0xffffffffu : static_cast<uint32_t>(words);
  a.scale = p < 1 ? static_cast<float>(1 / (1 - p)) : 0.f;
  a.dtype = dtype, a.rows = mode == SEGPOLY_DROPOUT_ROW, a.stream = stream;
  return launched(launch_dropout(a), "dropout");
}

}  // namespace

extern "C" {

int dropout_fwd(int dtype, int mode, const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                double p, uint64_t seed, uint64_t offset, const void* state, int64_t n, int64_t dim, void* out,
                int64_t out_stride, void* stream) {
  return dropout(dtype, mode, x, x_stride, residual, residual_stride, p, seed, offset, state, n, dim, out, out_stride,
                 stream);
}

int dropout_bwd(int dtype, int mode, const void* grad_out, int64_t grad_out_stride, double p, uint64_t seed,
                uint64_t offset, const void* state, int64_t n, int64_t dim, void* grad_x, int64_t grad_x_stride,
                void* stream) {
  return dropout(dtype, mode, grad_out, grad_out_stride, nullptr, 0, p, seed, offset, state, n, dim, grad_x,
                 grad_x_stride, stream);
}

int expert_sort_workspace(int64_t entries, int64_t num_experts, size_t* bytes) {
  if (!bytes) return fail(SEGPOLY_E_INVALID, "null bytes");
  int rc = check_sort(entries, num_experts);
  if (rc) return rc;
  *bytes = expert_sort_plan(entries, num_experts).bytes;
  return ok();
}

int expert_sort(const void* experts, int idx_dtype, int64_t entries, int64_t num_experts, void* order, void* place,
                void* offsets, void* ids, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_sort(entries, num_experts);
  if (rc) return rc;
  if (idx_dtype != SEGPOLY_I32 && idx_dtype != SEGPOLY_I64) return fail(SEGPOLY_E_INVALID, "bad index dtype");
  if (!offsets || (entries && (!experts || !order || !place || !ids))) return fail(SEGPOLY_E_INVALID, "null buffer");
  if ((rc = check_aligned(index_bytes(idx_dtype), {experts}))) return rc;
  if ((rc = check_aligned(4, {order, place, offsets, ids}))) return rc;
  rc = check_workspace(workspace, workspace_bytes, expert_sort_plan(entries, num_experts).bytes);
  if (rc) return rc;
  ExpertSortArgs a{};
  a.experts = experts, a.entries = entries, a.num = static_cast<int>(num_experts), a.idx = idx_dtype;
  a.order = static_cast<int*>(order), a.place = static_cast<int*>(place), a.offsets = static_cast<int*>(offsets);
  a.ids = static_cast<int*>(ids), a.counts = static_cast<int*>(workspace), a.stream = stream;
  return launched(launch_expert_sort(a), "expert sort");
}

int expert_dispatch_fwd(int dtype, const void* x, int64_t x_stride, const void* place, const void* offsets,
                        int64_t num_experts, int64_t n, int64_t k, int64_t dim, void* xs, void* stream) {
  int rc = check_rows(dtype, n, k, num_experts, dim);
  if (rc) return rc;
  if (x_stride < 0) return fail(SEGPOLY_E_INVALID, "negative stride");
  if (n == 0 || dim == 0) return ok();
  if (!x || !place || !offsets || !xs) return fail(SEGPOLY_E_INVALID, "null buffer");
  if ((rc = check_aligned(channel_dtype_bytes(dtype), {x, xs}))) return rc;
  if ((rc = check_aligned(4, {place, offsets}))) return rc;
  ExpertRowsArgs a{};
  a.x = x, a.x_stride = x_stride, a.place = static_cast<const int*>(place);
  a.total = static_cast<const int*>(offsets) + num_experts, a.out = xs, a.n = n, a.k = k, a.dim = dim;
  a.dtype = dtype, a.stream = stream;
  return launched(launch_expert_dispatch(a), "expert dispatch");
}

int expert_dispatch_bwd(int dtype, const void* grad_xs, int64_t grad_xs_stride, const void* place, const void* offsets,
                        int64_t num_experts, int64_t n, int64_t k, int64_t dim, void* grad_x, int64_t grad_x_stride,
                        void* stream) {
  int rc = check_rows(dtype, n, k, num_experts, dim);
  if (rc) return rc;
  if (grad_xs_stride < 0) return fail(SEGPOLY_E_INVALID, "negative stride");
  if (grad_x_stride < dim) return fail(SEGPOLY_E_INVALID, "grad_x_stride below dim");
  if (n == 0 || dim == 0) return ok();
  if (!grad_xs || !place || !offsets || !grad_x) return fail(SEGPOLY_E_INVALID, "null buffer");
  if ((rc = check_aligned(channel_dtype_bytes(dtype), {grad_xs, grad_x}))) return rc;
  if ((rc = check_aligned(4, {place, offsets}))) return rc;
  ExpertRowsArgs a{};
  a.ys = grad_xs, a.ys_stride = grad_xs_stride, a.place = static_cast<const int*>(place);
  a.total = static_cast<const int*>(offsets) + num_experts, a.out = grad_x, a.out_stride = grad_x_stride;
  a.n = n, a.k = k, a.dim = dim, a.dtype = dtype, a.stream = stream;
  return launched(launch_expert_combine(a), "expert dispatch gradient");
}

int expert_combine_fwd(int dtype, const void* ys, int64_t ys_stride, const void* place, const void* offsets,
                       int64_t num_experts, const void* weights, const void* residual, int64_t residual_stride, int64_t n,
                       int64_t k, int64_t dim, void* out, int64_t out_stride, void* stream) {
  int rc = check_rows(dtype, n, k, num_experts, dim);
  if (rc) return rc;
  if (ys_stride < 0 || residual_stride < 0) return fail(SEGPOLY_E_INVALID, "negative stride");
  if (out_stride < dim) return fail(SEGPOLY_E_INVALID, "out_stride below dim");
  if (n == 0 || dim == 0) return ok();
  if (!ys || !place || !offsets || !weights || !out) return fail(SEGPOLY_E_INVALID, "null buffer");
  if ((rc = check_aligned(channel_dtype_bytes(dtype), {ys, residual, out}))) return rc;
  if ((rc = check_aligned(4, {place, offsets, weights}))) return rc;
  ExpertRowsArgs a{};
  a.ys = ys, a.ys_stride = ys_stride, a.place = static_cast<const int*>(place);
  a.total = static_cast<const int*>(offsets) + num_experts, a.weights = static_cast<const float*>(weights);
  a.residual = residual, a.residual_stride = residual_stride, a.out = out, a.out_stride = out_stride;
  a.n = n, a.k = k, a.dim = dim, a.dtype = dtype, a.stream = stream;
  return launched(launch_expert_combine(a), "expert combine");
}

int expert_combine_bwd(int dtype, const void* grad_out, int64_t grad_out_stride, const void* ys, int64_t ys_stride,
                       const void* place, const void* offsets, int64_t num_experts, const void* weights, int64_t n,
                       int64_t k, int64_t dim, void* grad_ys, void* grad_weights, void* stream) {
  int rc = check_rows(dtype, n, k, num_experts, dim);
  if (rc) return rc;
  if (grad_out_stride < 0 || ys_stride < 0) return fail(SEGPOLY_E_INVALID, "negative stride");
  if (n == 0) return ok();
  if (!place || !offsets || !weights || !grad_weights || (dim && (!grad_out || !ys || !grad_ys)))
    return fail(SEGPOLY_E_INVALID, "null buffer");
  if ((rc = check_aligned(channel_dtype_bytes(dtype), {grad_out, ys, grad_ys}))) return rc;
  if ((rc = check_aligned(4, {place, offsets, weights, grad_weights}))) return rc;
  ExpertRowsArgs a{};
  a.x = grad_out, a.x_stride = grad_out_stride, a.ys = ys, a.ys_stride = ys_stride;
  a.place = static_cast<const int*>(place), a.total = static_cast<const int*>(offsets) + num_experts;
  a.weights = static_cast<const float*>(weights), a.out = grad_ys, a.grad_weights = static_cast<float*>(grad_weights);
  a.n = n, a.k = k, a.dim = dim, a.dtype = dtype, a.stream = stream;
  return launched(launch_expert_combine_bwd(a), "expert combine gradient");
}

}  // extern "C"
