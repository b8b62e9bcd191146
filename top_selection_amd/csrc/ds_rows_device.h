#pragma once
// Device helpers shared by the row operators' kernels.
#include "ds_rows.h"

namespace ds {
namespace {

// The element types: bf16 as its 16 bits, fp32 as it is. Widening is exact; narrowing to bf16
// rounds to nearest even, once.
template <int DT>
struct Elem;
template <>
struct Elem<DS_FP32> {
  using T = float;
  static constexpr int kPer16 = 4;  // elements in 16 bytes
  static __device__ __forceinline__ float widen(T v) { return v; }
  static __device__ __forceinline__ T narrow(float v) { return v; }
};
template <>
struct Elem<DS_BF16> {
  using T = uint16_t;
  static constexpr int kPer16 = 8;
  static __device__ __forceinline__ float widen(T v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
  static __device__ __forceinline__ T narrow(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  }
};

// Sixteen bytes of elements at their own alignment: the hardware reads and writes vectors at
// any element's address, so rows of odd length need no peeling.
template <int DT, int N>
struct Vec {
  using T = typename Elem<DT>::T;
  typedef T type __attribute__((ext_vector_type(N)));
  typedef type unaligned __attribute__((aligned(sizeof(T))));
};

// The value of a lane of the other half of 2^(LEVEL + 1) lanes, where the lanes of a half hold
// equal values (a butterfly's do after LEVEL levels): by data-parallel moves, no LDS.
template <int LEVEL>
__device__ __forceinline__ uint32_t from_partner(uint32_t v) {
  if constexpr (LEVEL == 0) return __builtin_amdgcn_update_dpp(0u, v, 0xB1, 0xF, 0xF, false);   // xor 1
  if constexpr (LEVEL == 1) return __builtin_amdgcn_update_dpp(0u, v, 0x4E, 0xF, 0xF, false);   // xor 2
  if constexpr (LEVEL == 2) return __builtin_amdgcn_update_dpp(0u, v, 0x141, 0xF, 0xF, false);  // 8 lanes reversed
  if constexpr (LEVEL == 3) return __builtin_amdgcn_update_dpp(0u, v, 0x140, 0xF, 0xF, false);  // 16 lanes reversed
  if constexpr (LEVEL == 4) {
    const auto q = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (threadIdx.x & 16u) ? q[0] : q[1];
  }
  if constexpr (LEVEL == 5) {
    const auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (threadIdx.x & 32u) ? q[0] : q[1];
  }
}
template <int LEVEL>
__device__ __forceinline__ int from_partner(int v) {
  return static_cast<int>(from_partner<LEVEL>(static_cast<uint32_t>(v)));
}
template <int LEVEL>
__device__ __forceinline__ float from_partner(float v) {
  return __uint_as_float(from_partner<LEVEL>(__float_as_uint(v)));
}
template <int LEVEL>
__device__ __forceinline__ double from_partner(double v) {
  return __hiloint2double(from_partner<LEVEL>(__double2hiint(v)), from_partner<LEVEL>(__double2loint(v)));
}

// f over 2^LEVELS neighbouring lanes, in all of them.
template <int LEVELS, class T, class F>
__device__ __forceinline__ T row_reduce(T v, F f) {
  if constexpr (LEVELS > 0) v = f(v, from_partner<0>(v));
  if constexpr (LEVELS > 1) v = f(v, from_partner<1>(v));
  if constexpr (LEVELS > 2) v = f(v, from_partner<2>(v));
  if constexpr (LEVELS > 3) v = f(v, from_partner<3>(v));
  if constexpr (LEVELS > 4) v = f(v, from_partner<4>(v));
  if constexpr (LEVELS > 5) v = f(v, from_partner<5>(v));
  return v;
}

template <class T>
__device__ __forceinline__ T plus(T a, T b) { return a + b; }

__device__ __forceinline__ float wave_max(float v) {
  return row_reduce<6>(v, [](float a, float b) { return fmaxf(a, b); });
}

template <class T>
__device__ __forceinline__ T wave_sum(T v) {
  return row_reduce<6>(v, plus<T>);
}

// Orders a wave's LDS accesses: what its lanes wrote before is what they read after.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// One workgroup per unit, in launches of at most kMaxUnits.
template <class P, class K>
hipError_t launch_units(K kern, P p, int64_t units, int threads, hipStream_t s) {
  for (p.unit0 = 0; p.unit0 < units; p.unit0 += kMaxUnits) {
    const int64_t g = units - p.unit0 < kMaxUnits ? units - p.unit0 : kMaxUnits;
    hipLaunchKernelGGL(kern, dim3(static_cast<uint32_t>(g)), dim3(threads), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace
}  // namespace ds
