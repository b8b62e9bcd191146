// Blocks of 128 to 8-bit floats and their scales.
#include "ds_expert.h"
#include "ds_rows_device.h"

namespace ds {
namespace {

// scale = max(|block|, 2^-100) / largest; q = x / scale, rounded once. With inv the rounded reciprocal, q0 = x inv
// is within two steps of the quotient, its remainder x - q0 scale comes from one fused step, and q0 + remainder inv,
// before its rounding to fp32, is off by less than 2^-45 of the quotient (P. Markstein, 1990), as long as the
// remainder is no subnormal: blocks below 2^-60 are multiplied by 2^64 first (scale too), which is exact. A
// division takes three times the instructions.
// Rounded to 8 bits from there, a quotient would be off where fp32 made it a tie of 8-bit floats (one bf16 element
// in 1500, one of fp32 in 2^23), so its remainder decides between it and its odd neighbours first: five instructions
// more an element (8192 x 4096 bf16 16.7 to 19.0 us; only where a lane's quotient ends in 16 zeros, by fours or
// by sixteens, 20.8).
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
  float scale;         // as it is stored
  float by, inv, raise;  // raise scale, its reciprocal (0: the block is not finite), 1 or 2^64
};
template <int QT>
__device__ __forceinline__ Scale scale_of(uint32_t most) {
  if (most >= 0x7F800000u) return {__uint_as_float(0x7FC00000u), 0.0f, 0.0f, 0.0f};
  const float top = fmaxf(__uint_as_float(most), 0x1p-100f);
  const float scale = top / Eight<QT>::kLargest, raise = top < 0x1p-60f ? 0x1p64f : 1.0f;
  return {scale, scale * raise, 1.0f / (scale * raise), raise};
}

// x / scale from its rounding to fp32: it or the odd float next to it on the quotient's side, so that rounding that
// to fewer bits rounds the quotient itself.
__device__ __forceinline__ float settled(float q, float x, float by) {
  const uint32_t even = __float_as_uint(q) & 0x7FFFFFFEu;
  const float rest = __builtin_fmaf(-__uint_as_float(even), by, __builtin_fabsf(x));  // exact
  int32_t side;  // of its sign, 0 of 0
  asm("v_med3_i32 %0, %1, -1, 1" : "=v"(side) : "v"(rest));
  return __builtin_copysignf(__uint_as_float(even + side), q);
}

// Sixteen elements. A block without a scale is 0 (its infinities and NaN are not converted).
template <int QT, bool RAISE>
__device__ __forceinline__ uint4 quantize16_of(const float (&v)[16], const Scale& s) {
  const auto one = [&](int i) {
    const float x = RAISE ? v[i] * s.raise : v[i], q0 = x * s.inv;
    return settled(__builtin_fmaf(__builtin_fmaf(-q0, s.by, x), s.inv, q0), x, s.by);
  };
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int lo = Eight<QT>::template pack<false>(one(4 * i), one(4 * i + 1), 0);
    w[i] = static_cast<uint32_t>(Eight<QT>::template pack<true>(one(4 * i + 2), one(4 * i + 3), lo));
  }
  return s.inv == 0.0f ? uint4{0, 0, 0, 0} : uint4{w[0], w[1], w[2], w[3]};
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
  for (int i = 0; i < 16; i += 2) m = max(max(magnitude(v[i]), magnitude(v[i + 1])), m);  // (one instruction of three)
  return m;
}

template <int QT>
__device__ __forceinline__ uint4 quantize16(const float (&v)[16], const Scale& s) {
  return __any(s.raise != 1.0f) ? quantize16_of<QT, true>(v, s) : quantize16_of<QT, false>(v, s);
}

__device__ __forceinline__ int64_t plan_end(const Plan& q) {
  const int64_t end = q.offsets[q.experts];
  return end < 0 ? 0 : end < q.capacity ? end : q.capacity;
}

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
constexpr int kPadRun = 16;

// Eight lanes take a block of a row, sixteen elements each (16-byte stores of eight lanes make a line). With a
// plan the row is quantised once and written to all its slots' positions, past the caches. Bound by the stores:
// 8192 x 8 rows of 4096 bf16, 365 MB, 54 us on the GPU, 6.7 TB/s (gathering first and quantising then: 108 and more).
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
    if (c < nc) __builtin_nontemporal_store(v4u{q.x, q.y, q.z, q.w}, reinterpret_cast<v4u*>(p.q + at * p.q_stride + c));
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

// A workgroup takes 128 positions of 64 columns through LDS: rows are read in vectors (all of a thread's at
// once: first the rows' numbers, then the rows), and a thread takes 32 elements of one (fp32) or two (bf16)
// columns, four or eight lanes a column, whose 16-byte stores make whole lines. The rows' distance in LDS makes the
// reads down the columns meet every bank once. A position's row is quantised anew for every expert, since the blocks
// run over positions: 28000 positions of 2001 fp32 columns 38.8 us, bound by vector instructions (by the counters 17
// an element: nine make the quotient and its rounding, the rest are magnitudes, padding, addresses and the way
// through LDS), memory would take 20.
template <int DT, int QT>
__global__ __launch_bounds__(256, 4) void quantize_column_kernel(QuantizeParams p) {
  using T = typename Elem<DT>::T;
  constexpr int V = Elem<DT>::kPer16, kCols = 64, kPerRow = kCols / V, kRows = 256 / kPerRow, kEach = 128 / kRows;
  constexpr int kPairs = DT == DS_BF16 ? 2 : 1;  // columns a 32-bit word
  constexpr int kStep = kCols / kPairs + 1;      // words a row
  using Vt = Vec<DT, V>;
  __shared__ uint32_t tile[128 * kStep + 8];
  const auto word = [&](int row) { return row * kStep + (kPairs == 2 ? (row >> 6) * 8 : 0); };
  const bool sorted = p.plan.place != nullptr;
  const int64_t P = sorted ? p.plan.capacity : p.rows, end = sorted ? plan_end(p.plan) : P;
  // Neighbouring workgroups are on eight XCDs: each takes an eighth of the columns, so that a row's second and
  // later readings (a token's other experts) find it in that XCD's L2.
  const int64_t per = p.col_units, unit = p.unit0 + blockIdx.x, turn = unit / p.xcds;
  const int64_t p0 = turn / per * 128, c0 = (unit % p.xcds * per + turn % per) * kCols;
  if (p0 >= end || c0 >= p.n) return;
  const int tc = threadIdx.x % kPerRow * V, tr = threadIdx.x / kPerRow;
  // where the positions' rows begin (one division a position); padding is read from the first row and cleared
  const T* x = static_cast<const T*>(p.x);
  __shared__ int64_t rows[128];
  if (threadIdx.x < 128) {
    const int64_t at = p0 + threadIdx.x;
    int64_t from = -1;
    if (at < end) {
      from = at;
      if (sorted) {
        const int slot = p.plan.order[at];
        from = slot >= 0 && slot < p.plan.rows * p.plan.k ? slot / p.plan.k : -1;
      }
    }
    rows[threadIdx.x] = from < 0 ? -1 : from * p.row_stride;
  }
  __syncthreads();
  int64_t from[kEach];
  typename Vt::type d[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) from[i] = rows[tr + i * kRows];
  if (p.rows == 0) {  // a plan of no rows whose offsets are broken: all is padding, and there is no first row
#pragma unroll
    for (int i = 0; i < kEach; ++i) d[i] = typename Vt::type{};
  } else if (c0 + kCols <= p.n) {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      d[i] = *reinterpret_cast<const typename Vt::unaligned*>(x + (from[i] < 0 ? 0 : from[i]) + c0 + tc);
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int64_t c = c0 + tc + e;
        const T one = x[(from[i] < 0 ? 0 : from[i]) + (c < p.n ? c : p.n - 1)];
        d[i][e] = c < p.n ? one : T{0};
      }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (from[i] < 0) d[i] = typename Vt::type{};
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const auto w = __builtin_bit_cast(__attribute__((ext_vector_type(4))) uint32_t, d[i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) tile[word(tr + i * kRows) + tc / kPairs + e] = w[e];
  }
  __syncthreads();
  constexpr int kLanes = 4 * kPairs;  // a column
  const int part = threadIdx.x % kLanes, col = threadIdx.x / kLanes * kPairs;
  float v[2][16];  // bf16: of two columns; fp32: of rows 64 apart
#pragma unroll
  for (int i = 0; i < 32 / kPairs; ++i) {
    const uint32_t w = tile[word(i / 16 * 64 + part * 16 + i % 16) + col / kPairs];
    if constexpr (kPairs == 2) {
      v[0][i] = __uint_as_float(w << 16);
      v[1][i] = __uint_as_float(w & 0xFFFF0000u);
    } else {
      v[i / 16][i % 16] = __uint_as_float(w);
    }
  }
  const auto top = [](uint32_t a, uint32_t b) { return max(a, b); };
  Scale s[2];
  if constexpr (kPairs == 2) {
    s[0] = scale_of<QT>(row_reduce<3>(most16(v[0]), top));
    s[1] = scale_of<QT>(row_reduce<3>(most16(v[1]), top));
  } else {
    s[0] = s[1] = scale_of<QT>(row_reduce<2>(max(most16(v[0]), most16(v[1])), top));
  }
  const int64_t wide = (P + 15) / 16 * 16, blocks = (P + 127) / 128;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t c = c0 + col + (kPairs == 2 ? h : 0), at = p0 + part * 16 + (kPairs == 2 ? 0 : h * 64);
    if (c < p.n) {
      if (at < wide) *reinterpret_cast<uint4*>(p.q + c * p.q_stride + at) = quantize16<QT>(v[h], s[h]);
      if (part == 0 && (kPairs == 2 || h == 0)) p.scales[c * blocks + p0 / 128] = s[h].scale;
    }
  }
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
    const int64_t units = (p.n + 63) / 64;
    p.xcds = units >= 8 ? 8 : 1;
    p.col_units = (units + p.xcds - 1) / p.xcds;
    return launch_units(quantize_column_kernel<DT, QT>, p, (P + 127) / 128 * p.col_units * p.xcds, 256, s);
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
