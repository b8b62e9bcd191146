// C ABI of the operators behind a router: argument validation (pure host code, before any HIP
// call), launch cuts and dispatch.
#include <initializer_list>

#include "ds_expert.h"

namespace {

int elem_bytes(int dtype) { return dtype == DS_BF16 ? 2 : 4; }
bool known(int dtype) { return dtype == DS_BF16 || dtype == DS_FP32; }
bool known8(int dtype) { return dtype == DS_E4M3 || dtype == DS_E5M2; }
bool misaligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }
int status(hipError_t e) { return e == hipSuccess ? DS_OK : DS_ERR_LAUNCH; }

// Rows of n elements, `stride` apart: sizes in range and the byte offsets in 63 bits.
bool rows_ok(int64_t rows, int64_t n, int64_t stride) {
  return rows >= 0 && rows <= INT32_MAX && n >= 1 && n <= INT32_MAX && stride >= n &&
         (rows == 0 || stride <= INT64_MAX / 8 / rows);
}

// The bytes from a tensor's first element to its last.
struct Range {
  uintptr_t lo, hi;
};
Range range(const void* p, int64_t rows, int64_t step_bytes, int64_t row_bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return !p || rows <= 0 || row_bytes <= 0 ? Range{0, 0} : Range{lo, lo + (rows - 1) * step_bytes + row_bytes};
}
Range range(const void* p, int64_t bytes) { return range(p, 1, 0, bytes); }

// Whether an output's range meets an input's or another output's.
bool meet(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }
bool clash(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range* o = outs.begin(); o != outs.end(); ++o) {
    for (const Range& i : ins)
      if (meet(*o, i)) return true;
    for (const Range* q = outs.begin(); q != o; ++q)
      if (meet(*o, *q)) return true;
  }
  return false;
}

int check_plan_sizes(int64_t rows, int k, int experts, int align) {
  if (rows < 0 || k < 1 || experts < 1 || align < 1) return DS_ERR_INVALID_ARG;
  if (k > DS_MAX_ROUTE_K || experts > DS_MAX_EXPERTS || align > DS_MAX_EXPERT_ALIGN) return DS_ERR_UNSUPPORTED;
  return rows > INT32_MAX / k ? DS_ERR_INVALID_ARG : DS_OK;
}

int64_t capacity_of(int64_t rows, int k, int experts, int align) {
  const int64_t slots = rows * k, ends = slots < experts ? slots : experts;
  return (slots + ends * (align - 1)) / align * align;
}

int check_plan(const ds_expert_plan* p) {
  if (!p) return DS_ERR_INVALID_ARG;
  const int st = check_plan_sizes(p->rows, p->k, p->experts, p->align);
  if (st != DS_OK) return st;
  if (p->capacity < capacity_of(p->rows, p->k, p->experts, p->align) || p->capacity > INT32_MAX)
    return DS_ERR_INVALID_ARG;
  if (!p->offsets || (p->rows > 0 && !p->place) || (p->capacity > 0 && !p->order)) return DS_ERR_INVALID_ARG;
  return misaligned(p->place, 4) || misaligned(p->order, 4) || misaligned(p->offsets, 4) ? DS_ERR_ALIGNMENT : DS_OK;
}

Range place_range(const ds_expert_plan& p) { return range(p.place, p.rows * p.k * 4); }
Range order_range(const ds_expert_plan& p) { return range(p.order, p.capacity * 4); }
Range offsets_range(const ds_expert_plan& p) { return range(p.offsets, (p.experts + 1) * 4); }

ds::Plan plan_of(const ds_expert_plan& p) {
  return {p.place, p.order, p.offsets, p.rows, p.capacity, p.k, p.experts, p.align};
}

size_t sort_bytes(const ds::SortCut& c, int experts) {
  return c.chunks > 1 ? static_cast<size_t>(c.chunks) * ds::counts_wide(experts) * sizeof(int32_t) : 0;
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
int64_t blocks_of(int64_t v) { return (v + DS_BLOCK - 1) / DS_BLOCK; }

}  // namespace

extern "C" {

int ds_expert_capacity(int64_t rows, int k, int experts, int align, int64_t* capacity) {
  if (!capacity) return DS_ERR_INVALID_ARG;
  const int st = check_plan_sizes(rows, k, experts, align);
  if (st != DS_OK) return st;
  const int64_t c = capacity_of(rows, k, experts, align);
  if (c > INT32_MAX) return DS_ERR_INVALID_ARG;
  *capacity = c;
  return DS_OK;
}

int ds_expert_sort_workspace_size(int64_t rows, int k, int experts, size_t* bytes) {
  if (!bytes) return DS_ERR_INVALID_ARG;
  const int st = check_plan_sizes(rows, k, experts, 1);
  if (st != DS_OK) return st;
  *bytes = sort_bytes(ds::cut_sort(rows * k), experts);
  return DS_OK;
}

int ds_expert_sort(const int32_t* idx, const ds_expert_plan* plan, void* workspace, size_t ws_bytes, void* stream) {
  int st = check_plan(plan);
  if (st != DS_OK) return st;
  if (plan->rows > 0 && !idx) return DS_ERR_INVALID_ARG;
  if (misaligned(idx, 4)) return DS_ERR_ALIGNMENT;
  const int64_t slots = plan->rows * plan->k;
  const ds::SortCut c = ds::cut_sort(slots);
  const size_t need = sort_bytes(c, plan->experts);
  if (need > 0) {
    if (!workspace || ws_bytes < need) return DS_ERR_WORKSPACE;
    if (misaligned(workspace, 16)) return DS_ERR_ALIGNMENT;
  }
  if (clash({place_range(*plan), order_range(*plan), offsets_range(*plan), range(need ? workspace : nullptr, need)},
            {range(idx, slots * 4)}))
    return DS_ERR_INVALID_ARG;
  (void)hipGetLastError();
  ds::SortParams p{};
  p.idx = idx;
  p.slots = slots;
  p.experts = plan->experts;
  p.align = plan->align;
  p.place = plan->place;
  p.order = plan->order;
  p.offsets = plan->offsets;
  p.capacity = plan->capacity;
  p.chunk = c.chunk;
  p.chunks = c.chunks;
  p.counts = static_cast<int32_t*>(workspace);
  return status(ds::launch_sort(p, static_cast<hipStream_t>(stream)));
}

int ds_expert_gather(const void* x, int64_t n, int64_t row_stride, int dtype, const ds_expert_plan* plan, void* out,
                     int64_t out_stride, void* stream) {
  if (!known(dtype)) return DS_ERR_INVALID_ARG;
  const int st = check_plan(plan);
  if (st != DS_OK) return st;
  if (!rows_ok(plan->rows, n, row_stride) || !rows_ok(plan->capacity, n, out_stride)) return DS_ERR_INVALID_ARG;
  if (plan->capacity == 0) return DS_OK;
  if ((plan->rows > 0 && !x) || !out) return DS_ERR_INVALID_ARG;
  const int eb = elem_bytes(dtype);
  if (misaligned(x, eb) || misaligned(out, eb)) return DS_ERR_ALIGNMENT;
  if (clash({range(out, plan->capacity, out_stride * eb, n * eb)},
            {range(x, plan->rows, row_stride * eb, n * eb), place_range(*plan), order_range(*plan), offsets_range(*plan)}))
    return DS_ERR_INVALID_ARG;
  (void)hipGetLastError();
  ds::MoveParams p{};
  p.plan = plan_of(*plan);
  p.x = x;
  p.x_stride = row_stride;
  p.n = n;
  p.out = out;
  p.out_stride = out_stride;
  return status(ds::launch_gather(dtype, p, static_cast<hipStream_t>(stream)));
}

int ds_expert_combine(const void* y, int64_t n, int64_t y_stride, int dtype, const ds_expert_plan* plan,
                      const float* weights, void* out, int64_t out_stride, void* stream) {
  if (!known(dtype)) return DS_ERR_INVALID_ARG;
  const int st = check_plan(plan);
  if (st != DS_OK) return st;
  if (!rows_ok(plan->capacity, n, y_stride) || !rows_ok(plan->rows, n, out_stride)) return DS_ERR_INVALID_ARG;
  if (plan->rows == 0) return DS_OK;
  if (!y || !out) return DS_ERR_INVALID_ARG;
  const int eb = elem_bytes(dtype);
  if (misaligned(y, eb) || misaligned(out, eb) || misaligned(weights, 4)) return DS_ERR_ALIGNMENT;
  if (clash({range(out, plan->rows, out_stride * eb, n * eb)},
            {range(y, plan->capacity, y_stride * eb, n * eb), range(weights, plan->rows * plan->k * 4),
             place_range(*plan), order_range(*plan), offsets_range(*plan)}))
    return DS_ERR_INVALID_ARG;
  (void)hipGetLastError();
  ds::MoveParams p{};
  p.plan = plan_of(*plan);
  p.x = y;
  p.x_stride = y_stride;
  p.n = n;
  p.weights = weights;
  p.out = out;
  p.out_stride = out_stride;
  return status(ds::launch_combine(dtype, p, static_cast<hipStream_t>(stream)));
}

int ds_expert_combine_grad(const void* g, int64_t g_stride, const void* y, int64_t y_stride, int64_t n, int dtype,
                           const ds_expert_plan* plan, const float* weights, void* grad_y, int64_t grad_stride,
                           float* grad_weights, void* stream) {
  if (!known(dtype)) return DS_ERR_INVALID_ARG;
  const int st = check_plan(plan);
  if (st != DS_OK) return st;
  if (!rows_ok(plan->rows, n, g_stride)) return DS_ERR_INVALID_ARG;
  if (grad_weights && !rows_ok(plan->capacity, n, y_stride)) return DS_ERR_INVALID_ARG;
  if (grad_y && !rows_ok(plan->capacity, n, grad_stride)) return DS_ERR_INVALID_ARG;
  if (plan->capacity == 0) return DS_OK;
  if (!grad_y && !grad_weights) return DS_ERR_INVALID_ARG;
  if (plan->rows > 0 && (!g || (grad_weights && !y))) return DS_ERR_INVALID_ARG;
  const int eb = elem_bytes(dtype);
  if (misaligned(g, eb) || misaligned(grad_y, eb) || misaligned(weights, 4) || misaligned(grad_weights, 4))
    return DS_ERR_ALIGNMENT;
  if (grad_weights && misaligned(y, eb)) return DS_ERR_ALIGNMENT;
  const int64_t slots4 = plan->rows * plan->k * 4;
  // over y itself: the lane that writes an element has read it before
  const bool over = grad_weights && y == grad_y && y_stride == grad_stride;
  if (clash({range(grad_y, plan->capacity, grad_stride * eb, n * eb), range(grad_weights, slots4)},
            {range(g, plan->rows, g_stride * eb, n * eb),
             grad_weights && !over ? range(y, plan->capacity, y_stride * eb, n * eb) : Range{0, 0},
             range(weights, slots4), place_range(*plan), order_range(*plan), offsets_range(*plan)}))
    return DS_ERR_INVALID_ARG;
  (void)hipGetLastError();
  ds::MoveParams p{};
  p.plan = plan_of(*plan);
  p.x = grad_weights ? y : nullptr;
  p.x_stride = y_stride;
  p.g = g;
  p.g_stride = g_stride;
  p.n = n;
  p.weights = weights;
  p.out = grad_y;
  p.out_stride = grad_stride;
  p.out_weights = grad_weights;
  return status(ds::launch_combine_grad(dtype, p, static_cast<hipStream_t>(stream)));
}

int ds_block_quantize(const void* x, int64_t rows, int64_t n, int64_t row_stride, int dtype, int layout,
                      const ds_expert_plan* plan, void* q, int64_t q_stride, int q_dtype, float* scales, void* stream) {
  if (!known(dtype) || !known8(q_dtype)) return DS_ERR_INVALID_ARG;
  if (layout != DS_BLOCK_ROW && layout != DS_BLOCK_COLUMN && layout != DS_BLOCK_TILE) return DS_ERR_INVALID_ARG;
  if (!rows_ok(rows, n, row_stride)) return DS_ERR_INVALID_ARG;
  int64_t positions = rows;
  if (plan) {
    const int st = check_plan(plan);
    if (st != DS_OK) return st;
    if (layout == DS_BLOCK_TILE || plan->rows != rows || (layout == DS_BLOCK_COLUMN && plan->align % DS_BLOCK != 0))
      return DS_ERR_INVALID_ARG;
    positions = plan->capacity;
  }
  const bool column = layout == DS_BLOCK_COLUMN;
  const int64_t q_rows = column ? n : positions, q_cols = up(column ? positions : n, 16);
  if (q_cols > INT32_MAX || q_stride < q_cols || (q_rows > 0 && q_stride > INT64_MAX / 8 / q_rows))
    return DS_ERR_INVALID_ARG;
  if (positions == 0) return DS_OK;
  if ((rows > 0 && !x) || !q || !scales) return DS_ERR_INVALID_ARG;
  const int eb = elem_bytes(dtype);
  if (misaligned(x, eb) || misaligned(q, 16) || q_stride % 16 != 0 || misaligned(scales, 4)) return DS_ERR_ALIGNMENT;
  const int64_t n_scales = (layout == DS_BLOCK_TILE ? blocks_of(rows) : q_rows) * blocks_of(column ? positions : n);
  if (clash({range(q, q_rows, q_stride, q_cols), range(scales, n_scales * 4)},
            {range(x, rows, row_stride * eb, n * eb), plan ? place_range(*plan) : Range{0, 0},
             plan ? order_range(*plan) : Range{0, 0}, plan ? offsets_range(*plan) : Range{0, 0}}))
    return DS_ERR_INVALID_ARG;
  (void)hipGetLastError();
  ds::QuantizeParams p{};
  if (plan) p.plan = plan_of(*plan);
  p.x = x;
  p.rows = rows;
  p.n = n;
  p.row_stride = row_stride;
  p.q = static_cast<uint8_t*>(q);
  p.q_stride = q_stride;
  p.scales = scales;
  return status(ds::launch_quantize(dtype, q_dtype, layout, p, static_cast<hipStream_t>(stream)));
}

int ds_block_product(const ds_block_operand* a, const ds_block_operand* b, int64_t m, int64_t n, int64_t k, int group,
                     int groups, const int32_t* offsets, void* out, int64_t out_stride, int out_dtype, void* stream) {
  const bool exact = (out_dtype & DS_EXACT_SUMS) != 0;
  out_dtype &= ~DS_EXACT_SUMS;
  if (!a || !b || !known8(a->dtype) || !known8(b->dtype) || !known(out_dtype)) return DS_ERR_INVALID_ARG;
  if (group != DS_GROUP_NONE && group != DS_GROUP_ROWS && group != DS_GROUP_INNER) return DS_ERR_INVALID_ARG;
  if (groups < 1 || (group == DS_GROUP_NONE && (groups != 1 || offsets)) || (group != DS_GROUP_NONE && !offsets))
    return DS_ERR_INVALID_ARG;
  if (a->scale_rows != 1 || (b->scale_rows != 1 && b->scale_rows != DS_BLOCK)) return DS_ERR_INVALID_ARG;
  if (group == DS_GROUP_INNER && b->scale_rows != 1) return DS_ERR_INVALID_ARG;
  if (b->dtype != DS_E4M3 || groups > DS_MAX_EXPERTS) return DS_ERR_UNSUPPORTED;
  if (m < 0 || m > INT32_MAX || n < 1 || n > INT32_MAX || k < 0 || k > INT32_MAX) return DS_ERR_INVALID_ARG;
  const int64_t b_rows = n * (group == DS_GROUP_ROWS ? groups : 1), out_rows = m * (group == DS_GROUP_INNER ? groups : 1);
  if (a->stride < k || b->stride < k || out_stride < n || (m > 0 && a->stride > INT64_MAX / 8 / m) ||
      b->stride > INT64_MAX / 8 / b_rows || (out_rows > 0 && out_stride > INT64_MAX / 8 / out_rows))
    return DS_ERR_INVALID_ARG;
  if (m == 0) return DS_OK;
  if (!out || (k > 0 && (!a->q || !b->q || !a->scales || !b->scales))) return DS_ERR_INVALID_ARG;
  const int ob = elem_bytes(out_dtype);
  if (k % 16 != 0 || misaligned(offsets, 4) || misaligned(out, ob)) return DS_ERR_ALIGNMENT;
  if (k > 0 && (a->stride % 16 != 0 || b->stride % 16 != 0 || misaligned(a->q, 16) || misaligned(b->q, 16) ||
                misaligned(a->scales, 4) || misaligned(b->scales, 4)))
    return DS_ERR_ALIGNMENT;
  const int64_t kb = blocks_of(k);
  const int64_t b_scales = (b->scale_rows == 1 ? b_rows : blocks_of(n) * (group == DS_GROUP_ROWS ? groups : 1)) * kb;
  if (clash({range(out, out_rows, out_stride * ob, n * ob)},
            {range(a->q, m, a->stride, k), range(b->q, b_rows, b->stride, k), range(a->scales, m * kb * 4),
             range(b->scales, b_scales * 4), range(offsets, (groups + 1) * 4)}))
    return DS_ERR_INVALID_ARG;
  (void)hipGetLastError();
  ds::ProductParams p{};
  p.a = static_cast<const uint8_t*>(a->q);
  p.b = static_cast<const uint8_t*>(b->q);
  p.sa = a->scales;
  p.sb = b->scales;
  p.a_stride = a->stride;
  p.b_stride = b->stride;
  p.m = m;
  p.n = n;
  p.k = k;
  p.blocks = static_cast<int32_t>(kb);
  p.groups = groups;
  p.offsets = offsets;
  p.out = out;
  p.out_stride = out_stride;
  return status(
      ds::launch_product(a->dtype, b->scale_rows, group, out_dtype, exact, p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
