#pragma once
// Interface between the C-ABI layer of the row operators (ds_rows_api.cpp) and their kernels
// (ds_route.hip, ds_probs.hip, ds_verify.hip). Not installed.
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/dstopk.h"

namespace ds {

struct RouteParams {
  const void* x;
  int64_t rows;
  int64_t row_stride;  // elements
  int32_t experts;
  int32_t k;
  const float* bias;   // NULL, or [experts]
  int32_t groups;
  int32_t group_size;
  int32_t topk_groups;
  int32_t group_top;
  int32_t renorm;
  float scale;
  float* out_weights;
  int32_t* out_idx;
  int32_t* counts;
  // set by the launcher: experts of a group (all without a limit), and how lanes share them
  int32_t run;
  int32_t per_lane;
  int32_t lanes_log2;
};

struct RouteGradParams {
  const void* x;
  int64_t rows;
  int64_t row_stride;
  int32_t experts;
  int32_t k;
  int32_t renorm;
  float scale;
  const int32_t* idx;
  const float* grad;
  void* out;
  int64_t out_stride;
};

struct SoftmaxParams {
  const void* x;
  int64_t rows;
  int64_t n;
  int64_t row_stride;
  const float* temperature;
  void* out;
  int64_t out_stride;
  int64_t slice;   // elements per workgroup
  int32_t slices;  // workgroups per row
  int64_t unit0;   // (row, slice) of a launch's first workgroup, set by the launcher
  float2* part;    // [rows][slices]: (maximum, sum of exp against it)
  int32_t together;  // no slices: log2 of the workgroups per row, set by the launcher
};

struct ListSoftmaxParams {
  const void* vals;
  const int32_t* idx;
  int64_t rows;
  int32_t k;
  const int32_t* ks;
  const float* temperature;
  const float* top_p;
  int64_t n;
  void* out;
  int64_t out_stride;
  float* out_list;
  int64_t slice;
  int32_t slices;
  int64_t unit0;
};

struct VerifyParams {
  const void* target;
  int64_t target_stride;
  const void* draft;
  int64_t draft_stride;
  const int32_t* tokens;
  const int32_t* lens;
  const float* accept_u;
  const float* sample_u;
  int64_t batch;
  int32_t drafts;
  int64_t n;
  int32_t* out_tokens;
  int32_t* out_accepted;
  int64_t slice;   // units per workgroup
  int32_t slices;
  int64_t unit0;
  double* part;    // [batch][units]: the units' sums (ds_verify.hip)
  int2* verdicts;  // [batch], after them; set by the launcher
};

hipError_t launch_route(int dtype, int score, const RouteParams& p, hipStream_t s);
hipError_t launch_route_grad(int dtype, int score, const RouteGradParams& p, hipStream_t s);
hipError_t launch_softmax(int dtype, int out_dtype, const SoftmaxParams& p, hipStream_t s);
hipError_t launch_list_softmax(int dtype, int out_dtype, const ListSoftmaxParams& p, hipStream_t s);
hipError_t launch_verify(int dtype, VerifyParams p, hipStream_t s);

// The compute units that a launch is sized for (MI355X).
constexpr int64_t kCus = 256;

// The most workgroups of a launch (of at most 1024 threads: a grid holds fewer than 2^32);
// longer work is launched in turns (`unit0` on).
constexpr int64_t kMaxUnits = 1 << 21;

// How a row of n elements is cut: `slices` workgroups of `slice` elements each.
struct RowCut {
  int64_t slice;
  int32_t slices;
};
RowCut cut_softmax(int64_t rows, int64_t n, int dtype);
RowCut cut_list_softmax(int64_t rows, int64_t n);

// How sequences are cut for the verification: `slices` workgroups of `slice` units each, and
// the workspace for the units' sums (slices == 0: one workgroup per sequence and no workspace).
struct VerifyCut {
  int64_t slice;
  int32_t slices;
  size_t bytes;
};
VerifyCut cut_verify(int64_t batch, int64_t n, int dtype);

}  // namespace ds
