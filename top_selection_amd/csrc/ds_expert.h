#pragma once
// Interface between the C-ABI layer of the operators behind a router (ds_expert_api.cpp) and
// their kernels (ds_expert.hip, ds_blocks.hip, ds_product.hip). Not installed.
#include "ds_rows.h"

namespace ds {

// A plan as the kernels read it (see ds_expert_plan).
struct Plan {
  const int32_t* place;
  const int32_t* order;
  const int32_t* offsets;
  int64_t rows;
  int64_t capacity;
  int32_t k;
  int32_t experts;
  int32_t align;
};

// The sort: `chunks` workgroups of `chunk` slots each.
struct SortParams {
  const int32_t* idx;
  int64_t slots;
  int32_t experts;
  int32_t align;
  int32_t* place;
  int32_t* order;
  int32_t* offsets;
  int64_t capacity;
  int64_t chunk;
  int32_t chunks;
  int32_t* counts;  // [chunks][counts_wide(experts)], the workspace (NULL for one chunk)
};
struct SortCut {
  int64_t chunk;
  int32_t chunks;
};
SortCut cut_sort(int64_t slots);
// A chunk's counts, in whole vectors of four.
__host__ __device__ constexpr int32_t counts_wide(int32_t experts) { return (experts + 3) / 4 * 4; }
// n slots in whole runs of `align`. The result is a position, below 2^31; n + align - 1 may not be.
__host__ __device__ constexpr int32_t padded(int32_t n, int32_t align) {
  return static_cast<int32_t>((static_cast<uint32_t>(n) + static_cast<uint32_t>(align - 1)) / static_cast<uint32_t>(align) *
                              static_cast<uint32_t>(align));
}
static_assert(padded(0, 126) == 0 && padded(1, 126) == 126 && padded(2147483546, 126) == 2147483646, "");
hipError_t launch_sort(const SortParams& p, hipStream_t s);

// Gather, combine and its gradient: teams of lanes walk a row in vectors.
struct MoveParams {
  Plan plan;
  const void* x;       // gather: x; combine: y; gradient: y
  int64_t x_stride;
  const void* g;       // gradient: g
  int64_t g_stride;
  int64_t n;
  const float* weights;
  void* out;           // gather, combine: out; gradient: grad_y
  int64_t out_stride;
  float* out_weights;  // gradient: grad_weights
  // set by the launcher
  int64_t pad_units;   // workgroups in front that clear padding
  int64_t unit0;
};
hipError_t launch_gather(int dtype, MoveParams p, hipStream_t s);
hipError_t launch_combine(int dtype, MoveParams p, hipStream_t s);
hipError_t launch_combine_grad(int dtype, MoveParams p, hipStream_t s);

struct QuantizeParams {
  Plan plan;           // place NULL: no plan
  const void* x;
  int64_t rows;
  int64_t n;
  int64_t row_stride;
  uint8_t* q;
  int64_t q_stride;
  float* scales;
  // set by the launcher
  int64_t pad_units;
  int64_t unit0;
  int64_t col_units;  // columns: workgroups across, for each of `xcds`
  int64_t xcds;
};
hipError_t launch_quantize(int dtype, int q_dtype, int layout, QuantizeParams p, hipStream_t s);

struct ProductParams {
  const uint8_t* a;
  const uint8_t* b;
  const float* sa;
  const float* sb;
  int64_t a_stride;
  int64_t b_stride;
  int64_t m;
  int64_t n;
  int64_t k;
  int32_t blocks;      // ceil(k / 128): scales of a row
  int32_t groups;
  const int32_t* offsets;
  void* out;
  int64_t out_stride;
  // set by the launcher
  int64_t m_tiles;     // an upper bound for DS_GROUP_ROWS
  int64_t n_tiles;
  int64_t unit0;
  int64_t units;
};
hipError_t launch_product(int a_dtype, int b_scale_rows, int group, int out_dtype, bool exact, ProductParams p, hipStream_t s);

}  // namespace ds
