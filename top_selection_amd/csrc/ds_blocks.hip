// Blocks of 128 to 8-bit floats and their scales.
#include "ds_expert.h"
#include "ds_rows_device.h"

namespace ds {
namespace {

// scale = max(|block|, 2^-100) / largest; q = x / scale. The quotient is the correctly rounded one by
// Markstein's theorem: with inv the correctly rounded reciprocal and q0 = x inv, q0 + (x - q0 scale) inv in
// two fused steps is x / scale rounded once, as long as the remainder is no subnormal: blocks below 2^-60
// divide.
template <int QT>
struct Eight;
template <>
struct Eight<DS_E4M3> {
  static constexpr float kLargest = 448.0f;
  template <bool HIGH>
  static __device__ __forceinline__ int pack(float a, float b, int old) {
    return __builtin_amdgcn_cvt_pk_fp8_f32(a, b, old, HIGH);
  }
};
template <>
struct Eight<DS_E5M2> {
  static constexpr float kLargest = 57344.0f;
  template <bool HIGH>
  static __device__ __forceinline__ int pack(float a, float b, int old) {
    return __builtin_amdgcn_cvt_pk_bf8_f32(a, b, old, HIGH);
  }
};

// |v| as an integer that orders magnitudes, infinities and NaN above them.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

struct Scale {
  float scale, inv;
  bool tiny;
};
template <int QT>
__device__ __forceinline__ Scale scale_of(uint32_t most) {
  if (most >= 0x7F800000u) return {__uint_as_float(0x7FC00000u), 0.0f, false};
  const float top = fmaxf(__uint_as_float(most), 0x1p-100f);
  const float scale = top / Eight<QT>::kLargest;
  return {scale, 1.0f / scale, top < 0x1p-60f};
}

// Four elements. A block without a scale is 0 (its infinities and NaN are not converted).
template <int QT>
__device__ __forceinline__ uint32_t quantize4(float a, float b, float c, float d, const Scale& s) {
  const auto one = [&](float v) {
    if (s.tiny) return v / s.scale;
    const float q0 = v * s.inv;
    return __builtin_fmaf(__builtin_fmaf(-q0, s.scale, v), s.inv, q0);
  };
  if (s.inv == 0.0f) return 0;
  const int lo = Eight<QT>::template pack<false>(one(a), one(b), 0);
  return static_cast<uint32_t>(Eight<QT>::template pack<true>(one(c), one(d), lo));
}

// Sixteen elements of a row from column c on, 0 past n.
template <int DT>
__device__ __forceinline__ void load16(const typename Elem<DT>::T* row, int64_t c, int64_t n, float (&v)[16]) {
  constexpr int V = Elem<DT>::kPer16;
  using Vt = Vec<DT, V>;
  if (c + 16 <= n) {
#pragma unroll
    for (int i = 0; i < 16; i += V) {
      const typename Vt::type d = *reinterpret_cast<const typename Vt::unaligned*>(row + c + i);
#pragma unroll
      for (int e = 0; e < V; ++e) v[i + e] = Elem<DT>::widen(d[e]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = c + i < n ? Elem<DT>::widen(row[c + i]) : 0.0f;
  }
}

__device__ __forceinline__ uint32_t most16(const float (&v)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, magnitude(v[i]));
  return m;
}

template <int QT>
__device__ __forceinline__ uint4 quantize16(const float (&v)[16], const Scale& s) {
  return {quantize4<QT>(v[0], v[1], v[2], v[3], s), quantize4<QT>(v[4], v[5], v[6], v[7], s),
          quantize4<QT>(v[8], v[9], v[10], v[11], s), quantize4<QT>(v[12], v[13], v[14], v[15], s)};
}

__device__ __forceinline__ int64_t plan_end(const Plan& q) {
  const int64_t end = q.offsets[q.experts];
  return end < 0 ? 0 : end < q.capacity ? end : q.capacity;
}

constexpr int kPadRun = 16;

// Eight lanes take a block of a row, sixteen elements each.
template <int DT, int QT>
__global__ __launch_bounds__(256) void quantize_row_kernel(QuantizeParams p) {
  using T = typename Elem<DT>::T;
  const int64_t nb = (p.n + 127) / 128, nc = (p.n + 15) / 16 * 16;
  int64_t unit = p.unit0 + blockIdx.x;
  if (unit < p.pad_units) {
    // padding rows: zeros, of the smallest scale
    const Plan& q = p.plan;
    const int parts = (q.align - 1 + kPadRun - 1) / kPadRun, e = static_cast<int>(unit / parts);
    const int part = static_cast<int>(unit % parts);
    int64_t lo = q.offsets[e], hi = q.offsets[e + 1];
    lo = lo < 0 ? 0 : lo;
    hi = hi < q.capacity ? hi : q.capacity;
    const Scale none = scale_of<QT>(0);
    for (int i = 0; i < kPadRun; ++i) {
      const int64_t at = hi - 1 - part * kPadRun - i;
      if (at < lo || at < hi - (q.align - 1)) break;
      const int s = q.order[at];
      if (s >= 0 && s < q.rows * q.k) break;
      for (int64_t c = threadIdx.x * 16; c < nc; c += 256 * 16)
        *reinterpret_cast<uint4*>(p.q + at * p.q_stride + c) = {0, 0, 0, 0};
      for (int64_t b = threadIdx.x; b < nb; b += 256) p.scales[at * nb + b] = none.scale;
    }
    return;
  }
  unit -= p.pad_units;
  const int64_t id = unit * 32 + threadIdx.x / 8, r = id / nb, b = id - r * nb;
  if (r >= p.rows) return;  // whole teams of eight lanes
  const int64_t c = b * 128 + threadIdx.x % 8 * 16;
  float v[16];
  load16<DT>(static_cast<const T*>(p.x) + r * p.row_stride, c, p.n, v);
  const uint32_t most = row_reduce<3>(most16(v), [](uint32_t a, uint32_t q) { return max(a, q); });
  const Scale s = scale_of<QT>(most);
  const uint4 q = quantize16<QT>(v, s);
  const auto put = [&](int64_t at) {
    if (c < nc) *reinterpret_cast<uint4*>(p.q + at * p.q_stride + c) = q;
    if (threadIdx.x % 8 == 0) p.scales[at * nb + b] = s.scale;
  };
  if (!p.plan.place) {
    put(r);
    return;
  }
  for (int j = 0; j < p.plan.k; ++j) {
    const int pos = p.plan.place[r * p.plan.k + j];
    if (pos >= 0 && pos < p.plan.capacity) put(pos);
  }
}

// A workgroup takes 128 positions of 64 columns through LDS; four lanes take a column.
template <int DT, int QT>
__global__ __launch_bounds__(256) void quantize_column_kernel(QuantizeParams p) {
  using T = typename Elem<DT>::T;
  constexpr int V = Elem<DT>::kPer16, kCols = 64, kPerRow = kCols / V, kRows = 256 / kPerRow;
  using Vt = Vec<DT, V>;
  __shared__ T tile[128][kCols + 4 / sizeof(T)];
  const bool sorted = p.plan.place != nullptr;
  const int64_t P = sorted ? p.plan.capacity : p.rows, end = sorted ? plan_end(p.plan) : P;
  const int64_t col_units = (p.n + kCols - 1) / kCols, unit = p.unit0 + blockIdx.x;
  const int64_t p0 = unit / col_units * 128, c0 = unit % col_units * kCols;
  if (p0 >= end) return;
  const int tc = threadIdx.x % kPerRow * V;
  for (int i = threadIdx.x / kPerRow; i < 128; i += kRows) {
    int64_t r = -1;
    if (p0 + i < end) {
      r = p0 + i;
      if (sorted) {
        const int s = p.plan.order[p0 + i];
        r = s >= 0 && s < p.plan.rows * p.plan.k ? s / p.plan.k : -1;
      }
    }
    typename Vt::type d = {};
    if (r >= 0) {
      const T* row = static_cast<const T*>(p.x) + r * p.row_stride + c0 + tc;
      if (c0 + tc + V <= p.n) {
        d = *reinterpret_cast<const typename Vt::unaligned*>(row);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (c0 + tc + e < p.n) d[e] = row[e];
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) tile[i][tc + e] = d[e];
  }
  __syncthreads();
  const int col = threadIdx.x / 4, part = threadIdx.x % 4;
  if (c0 + col >= p.n) return;
  float v[2][16];
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i / 16][i % 16] = Elem<DT>::widen(tile[part * 32 + i][col]);
  const uint32_t most =
      row_reduce<2>(max(most16(v[0]), most16(v[1])), [](uint32_t a, uint32_t b) { return max(a, b); });
  const Scale s = scale_of<QT>(most);
  const int64_t wide = (P + 15) / 16 * 16, at = p0 + part * 32;
  uint8_t* q = p.q + (c0 + col) * p.q_stride + at;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (at + 16 * h < wide) *reinterpret_cast<uint4*>(q + 16 * h) = quantize16<QT>(v[h], s);
  if (part == 0) p.scales[(c0 + col) * ((P + 127) / 128) + p0 / 128] = s.scale;
}

// A workgroup takes a tile of 128 x 128; eight lanes take a row's 128, four rows a thread.
template <int DT, int QT>
__global__ __launch_bounds__(256) void quantize_tile_kernel(QuantizeParams p) {
  using T = typename Elem<DT>::T;
  __shared__ uint32_t waves[4];
  const int64_t nb = (p.n + 127) / 128, nc = (p.n + 15) / 16 * 16;
  const int64_t unit = p.unit0 + blockIdx.x, r0 = unit / nb * 128, b = unit % nb;
  const int64_t c = b * 128 + threadIdx.x % 8 * 16;
  float v[4][16];
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + i * 32 + threadIdx.x / 8;
    if (r < p.rows) {
      load16<DT>(static_cast<const T*>(p.x) + r * p.row_stride, c, p.n, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[i][e] = 0.0f;
    }
    most = max(most, most16(v[i]));
  }
  most = row_reduce<6>(most, [](uint32_t a, uint32_t q) { return max(a, q); });
  if (threadIdx.x % 64 == 0) waves[threadIdx.x / 64] = most;
  __syncthreads();
  most = max(max(waves[0], waves[1]), max(waves[2], waves[3]));
  const Scale s = scale_of<QT>(most);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + i * 32 + threadIdx.x / 8;
    if (r < p.rows && c < nc) *reinterpret_cast<uint4*>(p.q + r * p.q_stride + c) = quantize16<QT>(v[i], s);
  }
  if (threadIdx.x == 0) p.scales[unit] = s.scale;
}

template <int DT, int QT>
hipError_t quantize_of(int layout, QuantizeParams p, hipStream_t s) {
  const bool sorted = p.plan.place != nullptr;
  const int64_t nb = (p.n + 127) / 128;
  if (layout == DS_BLOCK_ROW) {
    p.pad_units =
        sorted ? static_cast<int64_t>(p.plan.experts) * ((p.plan.align - 1 + kPadRun - 1) / kPadRun) : 0;
    return launch_units(quantize_row_kernel<DT, QT>, p, p.pad_units + (p.rows * nb + 31) / 32, 256, s);
  }
  if (layout == DS_BLOCK_COLUMN) {
    const int64_t P = sorted ? p.plan.capacity : p.rows;
    return launch_units(quantize_column_kernel<DT, QT>, p, (P + 127) / 128 * ((p.n + 63) / 64), 256, s);
  }
  return launch_units(quantize_tile_kernel<DT, QT>, p, (p.rows + 127) / 128 * nb, 256, s);
}

}  // namespace

hipError_t launch_quantize(int dtype, int q_dtype, int layout, QuantizeParams p, hipStream_t s) {
  if (dtype == DS_BF16)
    return q_dtype == DS_E4M3 ? quantize_of<DS_BF16, DS_E4M3>(layout, p, s) : quantize_of<DS_BF16, DS_E5M2>(layout, p, s);
  return q_dtype == DS_E4M3 ? quantize_of<DS_FP32, DS_E4M3>(layout, p, s) : quantize_of<DS_FP32, DS_E5M2>(layout, p, s);
}

}  // namespace ds
