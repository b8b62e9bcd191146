// C ABI of the operators beside the selection: argument validation (pure host code, before
// any HIP call), launch cuts and dispatch.
#include <cmath>
#include <cstdlib>

#include "ds_rows.h"

namespace {

int elem_bytes(int dtype) { return dtype == DS_BF16 ? 2 : 4; }
bool known(int dtype) { return dtype == DS_BF16 || dtype == DS_FP32; }
bool misaligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Rows of n elements, `stride` apart: sizes in range and the byte offsets in 63 bits.
bool rows_ok(int64_t rows, int64_t n, int64_t stride) {
  return rows >= 0 && n >= 1 && n <= INT32_MAX && stride >= n && (rows == 0 || stride <= INT64_MAX / 4 / rows);
}

// Whether any of `rows` runs of a_len bytes, a_step apart from a on, shares a byte with any of those of b
// (steps are not below lengths). Rows that lie among one another, as columns of one matrix do, need not.
bool share_bytes(const void* a, int64_t a_step, int64_t a_len, const void* b, int64_t b_step, int64_t b_len,
                 int64_t rows) {
  // the distance of the first runs; runs i of a and j of b meet when d + j b_step - i a_step lies in (-b_len, a_len)
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  if (d >= (rows - 1) * a_step + a_len || -d >= (rows - 1) * b_step + b_len) return false;
  if (rows == 1) return true;
  if (a_step == b_step) {  // only the two differences j - i that bring d within one step of 0 can meet
    int64_t t = -d / a_step;
    if (-d % a_step < 0) --t;
    return (std::llabs(t) < rows && d + t * a_step > -b_len) || (std::llabs(t + 1) < rows && d + (t + 1) * a_step < a_len);
  }
  for (int64_t i = 0, j = 0; i < rows && j < rows;) {
    const int64_t at = d + j * b_step - i * a_step;
    if (at >= a_len) ++i;
    else if (at <= -b_len) ++j;
    else return true;
  }
  return false;
}

int check_route(int64_t rows, int64_t experts, int64_t row_stride, int k, int dtype, const ds_route_config* cfg,
                ds_route_config* out) {
  if (!known(dtype)) return DS_ERR_INVALID_ARG;
  if (!rows_ok(rows, experts, row_stride)) return DS_ERR_INVALID_ARG;
  if (k < 1 || k > experts) return DS_ERR_INVALID_ARG;
  if (experts > DS_MAX_EXPERTS || k > DS_MAX_ROUTE_K) return DS_ERR_UNSUPPORTED;
  ds_route_config c = cfg ? *cfg : ds_route_config{DS_SCORE_SOFTMAX, 1, 1, 1, 0, 1.0f};
  if (c.score != DS_SCORE_SOFTMAX && c.score != DS_SCORE_SIGMOID) return DS_ERR_INVALID_ARG;
  if (c.groups == 0) c.groups = 1;
  if (c.topk_groups == 0) c.topk_groups = c.groups;
  if (c.group_top == 0) c.group_top = 1;
  if (c.groups < 1 || c.topk_groups < 1 || c.topk_groups > c.groups || experts % c.groups != 0)
    return DS_ERR_INVALID_ARG;
  const int64_t size = experts / c.groups;
  if (c.group_top < 1 || c.group_top > 2 || c.group_top > size || size * c.topk_groups < k) return DS_ERR_INVALID_ARG;
  if (c.groups > DS_MAX_ROUTE_GROUPS) return DS_ERR_UNSUPPORTED;
  if (!std::isfinite(c.scale)) return DS_ERR_INVALID_ARG;
  *out = c;
  return DS_OK;
}

int status(hipError_t e) { return e == hipSuccess ? DS_OK : DS_ERR_LAUNCH; }

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return DS_OK;
  if (!ws || have < need) return DS_ERR_WORKSPACE;
  return misaligned(ws, 8) ? DS_ERR_ALIGNMENT : DS_OK;
}

size_t softmax_bytes(int64_t rows, const ds::RowCut& c) { return static_cast<size_t>(rows) * c.slices * sizeof(float2); }

}  // namespace

extern "C" {

int ds_route(const void* x, int64_t rows, int64_t experts, int64_t row_stride, int k, int dtype, const float* bias,
             const ds_route_config* cfg, float* out_weights, int32_t* out_idx, int32_t* counts, void* stream) {
  ds_route_config c;
  const int st = check_route(rows, experts, row_stride, k, dtype, cfg, &c);
  if (st != DS_OK || rows == 0) return st;
  if (!x || (!out_weights && !out_idx) || (counts && !out_idx)) return DS_ERR_INVALID_ARG;
  if (misaligned(x, elem_bytes(dtype)) || misaligned(bias, 4) || misaligned(out_weights, 4) || misaligned(out_idx, 4) ||
      misaligned(counts, 4))
    return DS_ERR_ALIGNMENT;
  (void)hipGetLastError();
  ds::RouteParams p{};
  p.x = x;
  p.rows = rows;
  p.row_stride = row_stride;
  p.experts = static_cast<int32_t>(experts);
  p.k = k;
  p.bias = bias;
  p.groups = c.groups;
  p.group_size = static_cast<int32_t>(experts / c.groups);
  p.topk_groups = c.topk_groups;
  p.group_top = c.group_top;
  p.renorm = c.renormalize != 0;
  p.scale = c.scale;
  p.out_weights = out_weights;
  p.out_idx = out_idx;
  p.counts = counts;
  return status(ds::launch_route(dtype, c.score, p, static_cast<hipStream_t>(stream)));
}

int ds_route_grad(const void* x, int64_t rows, int64_t experts, int64_t row_stride, int k, int dtype,
                  const ds_route_config* cfg, const int32_t* idx, const float* grad_weights, void* grad_x,
                  int64_t grad_stride, void* stream) {
  ds_route_config c;
  const int st = check_route(rows, experts, row_stride, k, dtype, cfg, &c);
  if (st != DS_OK) return st;
  if (!rows_ok(rows, experts, grad_stride)) return DS_ERR_INVALID_ARG;
  if (rows == 0) return DS_OK;
  if (!x || !idx || !grad_weights || !grad_x) return DS_ERR_INVALID_ARG;
  const int eb = elem_bytes(dtype);
  if (misaligned(x, eb) || misaligned(idx, 4) || misaligned(grad_weights, 4) || misaligned(grad_x, eb))
    return DS_ERR_ALIGNMENT;
  // over x itself: the wave that writes a row has read it before
  const bool over = x == grad_x && (row_stride == grad_stride || rows == 1);
  if (!over && share_bytes(x, row_stride * eb, experts * eb, grad_x, grad_stride * eb, experts * eb, rows))
    return DS_ERR_INVALID_ARG;
  (void)hipGetLastError();
  ds::RouteGradParams p{};
  p.x = x;
  p.rows = rows;
  p.row_stride = row_stride;
  p.experts = static_cast<int32_t>(experts);
  p.k = k;
  p.renorm = c.renormalize != 0;
  p.scale = c.scale;
  p.idx = idx;
  p.grad = grad_weights;
  p.out = grad_x;
  p.out_stride = grad_stride;
  return status(ds::launch_route_grad(dtype, c.score, p, static_cast<hipStream_t>(stream)));
}

int ds_softmax_workspace_size(int64_t rows, int64_t n, int dtype, size_t* bytes) {
  if (!bytes || !known(dtype) || !rows_ok(rows, n, n)) return DS_ERR_INVALID_ARG;
  *bytes = softmax_bytes(rows, ds::cut_softmax(rows, n, dtype));
  return DS_OK;
}

int ds_softmax(const void* x, int64_t rows, int64_t n, int64_t row_stride, int dtype, const float* temperature,
               void* out, int64_t out_stride, int out_dtype, void* workspace, size_t ws_bytes, void* stream) {
  if (!known(dtype) || !known(out_dtype)) return DS_ERR_INVALID_ARG;
  if (!rows_ok(rows, n, row_stride) || !rows_ok(rows, n, out_stride)) return DS_ERR_INVALID_ARG;
  if (rows == 0) return DS_OK;
  if (!x || !out) return DS_ERR_INVALID_ARG;
  const int xb = elem_bytes(dtype), ob = elem_bytes(out_dtype);
  if (misaligned(x, xb) || misaligned(out, ob) || misaligned(temperature, 4)) return DS_ERR_ALIGNMENT;
  if (share_bytes(x, row_stride * xb, n * xb, out, out_stride * ob, n * ob, rows)) return DS_ERR_INVALID_ARG;
  const ds::RowCut c = ds::cut_softmax(rows, n, dtype);
  const int st = check_workspace(workspace, ws_bytes, softmax_bytes(rows, c));
  if (st != DS_OK) return st;
  (void)hipGetLastError();
  ds::SoftmaxParams p{};
  p.x = x;
  p.rows = rows;
  p.n = n;
  p.row_stride = row_stride;
  p.temperature = temperature;
  p.out = out;
  p.out_stride = out_stride;
  p.slice = c.slice;
  p.slices = c.slices;
  p.part = static_cast<float2*>(workspace);
  return status(ds::launch_softmax(dtype, out_dtype, p, static_cast<hipStream_t>(stream)));
}

int ds_topk_softmax(const void* vals, const int32_t* idx, int64_t rows, int k, int dtype, const int32_t* ks,
                    const float* temperature, const float* top_p, int64_t n, void* out, int64_t out_stride,
                    int out_dtype, float* out_list, void* stream) {
  if (!known(dtype) || !known(out_dtype)) return DS_ERR_INVALID_ARG;
  if (!rows_ok(rows, n, out ? out_stride : n) || k < 1 || k > n) return DS_ERR_INVALID_ARG;
  if (k > DS_MAX_K) return DS_ERR_UNSUPPORTED;
  if (rows == 0) return DS_OK;
  if (!vals || !idx || (!out && !out_list)) return DS_ERR_INVALID_ARG;
  if (misaligned(vals, elem_bytes(dtype)) || misaligned(idx, 4) || misaligned(out, elem_bytes(out_dtype)) ||
      misaligned(ks, 4) || misaligned(temperature, 4) || misaligned(top_p, 4) || misaligned(out_list, 4))
    return DS_ERR_ALIGNMENT;
  const ds::RowCut c = out ? ds::cut_list_softmax(rows, n) : ds::RowCut{n, 1};
  (void)hipGetLastError();
  ds::ListSoftmaxParams p{};
  p.vals = vals;
  p.idx = idx;
  p.rows = rows;
  p.k = k;
  p.ks = ks;
  p.temperature = temperature;
  p.top_p = top_p;
  p.n = n;
  p.out = out;
  p.out_stride = out_stride;
  p.out_list = out_list;
  p.slice = c.slice;
  p.slices = c.slices;
  return status(ds::launch_list_softmax(dtype, out_dtype, p, static_cast<hipStream_t>(stream)));
}

int ds_verify_workspace_size(int64_t batch, int64_t n, int dtype, size_t* bytes) {
  if (!bytes || !known(dtype) || !rows_ok(batch, n, n)) return DS_ERR_INVALID_ARG;
  *bytes = ds::cut_verify(batch, n, dtype).bytes;
  return DS_OK;
}

int ds_verify(const void* target, int64_t target_stride, const void* draft, int64_t draft_stride,
              const int32_t* draft_tokens, const int32_t* draft_lens, const float* accept_u, const float* sample_u,
              int64_t batch, int drafts, int64_t n, int dtype, int32_t* out_tokens, int32_t* out_accepted,
              void* workspace, size_t ws_bytes, void* stream) {
  if (!known(dtype)) return DS_ERR_INVALID_ARG;
  if (drafts < 0 || batch < 0 || batch > INT32_MAX) return DS_ERR_INVALID_ARG;
  if (drafts > DS_MAX_DRAFTS) return DS_ERR_UNSUPPORTED;
  if (!rows_ok(batch * (drafts + 1), n, target_stride)) return DS_ERR_INVALID_ARG;
  if (draft && drafts > 0 && !rows_ok(batch * drafts, n, draft_stride)) return DS_ERR_INVALID_ARG;
  if (batch == 0) return DS_OK;
  if (!target || !sample_u || !out_tokens || !out_accepted) return DS_ERR_INVALID_ARG;
  if (drafts > 0 && (!draft_tokens || !accept_u)) return DS_ERR_INVALID_ARG;
  const int eb = elem_bytes(dtype);
  if (misaligned(target, eb) || misaligned(draft, eb) || misaligned(draft_tokens, 4) || misaligned(draft_lens, 4) ||
      misaligned(accept_u, 4) || misaligned(sample_u, 4) || misaligned(out_tokens, 4) || misaligned(out_accepted, 4))
    return DS_ERR_ALIGNMENT;
  const ds::VerifyCut c = ds::cut_verify(batch, n, dtype);
  const int st = check_workspace(workspace, ws_bytes, c.bytes);
  if (st != DS_OK) return st;
  (void)hipGetLastError();
  ds::VerifyParams p{};
  p.target = target;
  p.target_stride = target_stride;
  p.draft = drafts > 0 ? draft : nullptr;
  p.draft_stride = draft_stride;
  p.tokens = draft_tokens;
  p.lens = draft_lens;
  p.accept_u = accept_u;
  p.sample_u = sample_u;
  p.batch = batch;
  p.drafts = drafts;
  p.n = n;
  p.out_tokens = out_tokens;
  p.out_accepted = out_accepted;
  p.slice = c.slice;
  p.slices = c.slices;
  p.part = static_cast<double*>(workspace);
  return status(ds::launch_verify(dtype, p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
