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

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// Orders a wave's LDS accesses: what its lanes wrote before is what they read after.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <class T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
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
