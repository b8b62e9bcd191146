// Products of 8-bit operands with a scale for each block of 128 along the inner axis.
#include "ds_expert.h"
#include "ds_rows_device.h"

namespace ds {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

typedef __bf16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v2h __attribute__((ext_vector_type(2)));

// Eight 8-bit floats as bf16, exactly.
template <int ET>
__device__ __forceinline__ v8h widen8(int lo, int hi) {
  v2h p[4];
  if constexpr (ET == DS_E4M3) {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  } else {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, false);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, true);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, false);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, true);
  }
  return v8h{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

// One block of 128 of sixteen rows of each side: lane l gives 32 of row l % 16's bytes, the same ones on
// both sides (the sum's order is the hardware's), and gets elements (b row 4 (l / 16) + i, a row l % 16).
// As bf16 the products are exact and the sums fp32: the 8-bit unit itself adds eight products at a time
// aligned to the largest of them, and cuts what is below 2^-13 of it (measured: 1.5e-5 to 7e-5 of the
// result for normal data, where this way is exact to fp32's rounding).
template <int AT>
__device__ __forceinline__ v4f block_product(v8i b, v8i a) {
  v4f d{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<DS_E4M3>(b[i], b[i + 1]), widen8<AT>(a[i], a[i + 1]), d, 0, 0, 0);
  return d;
}

// What a workgroup works on.
struct Tile {
  int group;
  int64_t m0, m1;  // rows of a and out
  int64_t k0, k1;  // the inner range
};

__device__ __forceinline__ int64_t clamped(const ProductParams& p, int g, int64_t most) {
  const int64_t v = p.offsets[g];
  return v < 0 ? 0 : v < most ? v : most;
}

// The t-th tile of TM rows of the groups' segments, found by every wave for itself: 64 groups' tiles are
// counted at a time. False past the last.
template <int TM>
__device__ __forceinline__ bool find_rows(const ProductParams& p, int64_t t, Tile& tile) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int g0 = 0; g0 < p.groups; g0 += 64) {
    const int g = g0 + lane;
    int64_t lo = 0, hi = 0;
    if (g < p.groups) {
      lo = clamped(p, g, p.m);
      hi = clamped(p, g + 1, p.m);
    }
    const int tiles = hi > lo ? static_cast<int>((hi - lo + TM - 1) / TM) : 0;
    int incl = tiles;
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d);
      if (lane >= d) incl += v;
    }
    const uint64_t past = __ballot(t < before + incl);
    if (past) {
      const int at = __ffsll(static_cast<unsigned long long>(past)) - 1;
      const int64_t first = before + __shfl(incl - tiles, at);
      const int slo = __shfl(static_cast<int>(lo), at), shi = __shfl(static_cast<int>(hi), at);
      tile.group = __builtin_amdgcn_readfirstlane(g0 + at);
      tile.m0 = __builtin_amdgcn_readfirstlane(static_cast<int>(slo + (t - first) * TM));
      tile.m1 = __builtin_amdgcn_readfirstlane(shi);
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

template <int GROUP, int TM>
__device__ __forceinline__ bool find_tile(const ProductParams& p, int64_t mt, Tile& tile) {
  tile.k0 = 0;
  tile.k1 = p.k;
  if constexpr (GROUP == DS_GROUP_ROWS) return find_rows<TM>(p, mt, tile);
  const int64_t per = (p.m + TM - 1) / TM;
  tile.group = static_cast<int>(mt / per);
  tile.m0 = (mt - tile.group * per) * TM;
  tile.m1 = p.m;
  if constexpr (GROUP == DS_GROUP_INNER) {
    // whole blocks: other offsets count as the next multiple
    const int64_t lo = (clamped(p, tile.group, p.k) + 127) / 128 * 128, hi = (clamped(p, tile.group + 1, p.k) + 127) / 128 * 128;
    tile.k0 = lo < p.k ? lo : p.k;
    tile.k1 = hi < p.k ? hi : p.k;
  }
  return true;
}

// Sixteen bytes of a row's block, 0 past the end.
__device__ __forceinline__ v4i load_part(const uint8_t* row, int64_t k, int64_t k1) {
  return k < k1 ? *reinterpret_cast<const v4i*>(row + k) : v4i{0, 0, 0, 0};
}

template <int OT>
__device__ __forceinline__ void store4(typename Elem<OT>::T* out, int64_t n0, int64_t n, const float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n0 + i < n) out[n0 + i] = Elem<OT>::narrow(v[i]);
}

// Sixteen rows of a and 64 of b a workgroup; its four waves take every fourth block of the inner
// axis, and their sums are joined in LDS in the waves' order.
template <int AT, int BROWS, int GROUP, int OT>
__global__ __launch_bounds__(256) void product_small_kernel(ProductParams p) {
  __shared__ float part[4][64][16 + 1];
  const int64_t unit = p.unit0 + blockIdx.x;
  Tile t;
  if (!find_tile<GROUP, 16>(p, unit / p.n_tiles, t)) return;
  const int64_t n0 = unit % p.n_tiles * 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane & 15, quad = lane >> 4;
  const int64_t b0 = GROUP == DS_GROUP_ROWS ? t.group * p.n : 0;
  const int64_t b_blocks = (p.n + 127) / 128;
  const bool a_live = t.m0 + row < t.m1;
  const uint8_t* a = p.a + (t.m0 + row) * p.a_stride;
  float acc[4][4] = {};
  for (int64_t k = t.k0 + wave * 128; k < t.k1; k += 4 * 128) {
    const int64_t kb = k / 128;
    v4i a0{}, a1{};
    float sa = 0;
    if (a_live) {
      a0 = load_part(a, k + quad * 16, t.k1);
      a1 = load_part(a, k + 64 + quad * 16, t.k1);
      sa = p.sa[(t.m0 + row) * p.blocks + kb];
    }
    const v8i av = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int64_t n = n0 + f * 16 + row;
      v4i b0v{}, b1v{};
      if (n < p.n) {
        const uint8_t* b = p.b + (b0 + n) * p.b_stride;
        b0v = load_part(b, k + quad * 16, t.k1);
        b1v = load_part(b, k + 64 + quad * 16, t.k1);
      }
      const v4f d = block_product<AT>(__builtin_shufflevector(b0v, b1v, 0, 1, 2, 3, 4, 5, 6, 7), av);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t nn = n0 + f * 16 + quad * 4 + i;
        float sb = 0;
        if (nn < p.n)
          sb = BROWS == 1 ? p.sb[(b0 + nn) * p.blocks + kb]
                          : p.sb[((GROUP == DS_GROUP_ROWS ? t.group * b_blocks : 0) + nn / 128) * p.blocks + kb];
        acc[f][i] = __builtin_fmaf(sa * sb, d[i], acc[f][i]);
      }
    }
  }
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][lane][f * 4 + i] = acc[f][i];
  __syncthreads();
  // wave f stores b rows 16 f on
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = wave * 4 + i;
    v[i] = part[0][lane][at] + part[1][lane][at] + part[2][lane][at] + part[3][lane][at];
  }
  if (!a_live) return;
  const int64_t out_row = (GROUP == DS_GROUP_INNER ? t.group * p.m : 0) + t.m0 + row;
  store4<OT>(static_cast<typename Elem<OT>::T*>(p.out) + out_row * p.out_stride, n0 + wave * 16 + quad * 4, p.n, v);
}

template <int AT, int BROWS, int GROUP, int OT>
hipError_t product_of(ProductParams p, hipStream_t s) {
  constexpr int TM = 16, TN = 64;
  p.m_tiles = (p.m + TM - 1) / TM;
  if (GROUP == DS_GROUP_ROWS) p.m_tiles = p.m < p.m / TM + p.groups ? p.m : p.m / TM + p.groups;
  if (GROUP == DS_GROUP_INNER) p.m_tiles *= p.groups;
  p.n_tiles = (p.n + TN - 1) / TN;
  return launch_units(product_small_kernel<AT, BROWS, GROUP, OT>, p, p.m_tiles * p.n_tiles, 256, s);
}

template <int AT, int OT>
hipError_t product_by_group(int b_rows, int group, const ProductParams& p, hipStream_t s) {
  if (group == DS_GROUP_INNER) return product_of<AT, 1, DS_GROUP_INNER, OT>(p, s);
  if (group == DS_GROUP_ROWS)
    return b_rows == 1 ? product_of<AT, 1, DS_GROUP_ROWS, OT>(p, s) : product_of<AT, 128, DS_GROUP_ROWS, OT>(p, s);
  return b_rows == 1 ? product_of<AT, 1, DS_GROUP_NONE, OT>(p, s) : product_of<AT, 128, DS_GROUP_NONE, OT>(p, s);
}

}  // namespace

hipError_t launch_product(int a_dtype, int b_rows, int group, int out_dtype, ProductParams p, hipStream_t s) {
  if (a_dtype == DS_E4M3)
    return out_dtype == DS_BF16 ? product_by_group<DS_E4M3, DS_BF16>(b_rows, group, p, s)
                                : product_by_group<DS_E4M3, DS_FP32>(b_rows, group, p, s);
  return out_dtype == DS_BF16 ? product_by_group<DS_E5M2, DS_BF16>(b_rows, group, p, s)
                              : product_by_group<DS_E5M2, DS_FP32>(b_rows, group, p, s);
}

}  // namespace ds
