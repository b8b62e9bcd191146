// A sampler's probabilities: softmax of whole rows at a temperature, and of top-k lists.
#include "ds_rows_device.h"

namespace ds {
namespace {

constexpr int kSoftWaves = 8;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2E = 1.44269504088896341f;

// (v - m) * scale; by way of half the difference, which does not overflow for finite numbers, where the
// product might be small all the same (and not elsewhere: half of fp32's least number is 0).
__device__ __forceinline__ float apart(float v, float m, float scale) {
  const bool half = scale < 1.0f;
  const float h = half ? 0.5f : 1.0f;
  return fmaf(v, h, m * -h) * (half ? scale + scale : scale);
}

// exp((v - m) / t) with scale = log2(e) / t; exactly 1 at the maximum, infinities included.
__device__ __forceinline__ float soft_exp(float v, float m, float scale) {
  return v == m ? 1.0f : __builtin_amdgcn_exp2f(apart(v, m, scale));
}

// (maximum, sum) of two parts of a row. A part without any mass is (-inf, 0).
__device__ __forceinline__ float2 soft_join(float2 a, float2 b, float scale) {
  const float m = fmaxf(a.x, b.x);
  if (m == kNegInf) return make_float2(kNegInf, 0.0f);
  return make_float2(m, a.y * soft_exp(a.x, m, scale) + b.y * soft_exp(b.x, m, scale));
}

// A part of a greedy row: its maximum and the bits of the first index that holds it.
__device__ __forceinline__ float2 first_join(float2 a, float2 b) {
  const bool take = b.x > a.x || (b.x == a.x && __float_as_uint(b.y) < __float_as_uint(a.y));
  return take ? b : a;
}

__device__ __forceinline__ float2 wave_xor(float2 v, int o) {
  return make_float2(__shfl_xor(v.x, o), __shfl_xor(v.y, o));
}

__device__ __forceinline__ float row_scale(const float* temperature, int64_t r, bool* greedy) {
  const float t = temperature ? temperature[r] : 1.0f;
  *greedy = !(t > 0.0f);
  // at an infinite temperature fp32's least number: -inf keeps no mass, and the largest difference there is
  // moves an exponent by 1e-6
  return *greedy ? 0.0f : fmaxf(kLog2E / t, __uint_as_float(1u));
}

// One workgroup per (row, slice): the slice's maximum and sum.
template <int DT>
__global__ __launch_bounds__(kSoftWaves * 64) void softmax_stats_kernel(SoftmaxParams p) {
  using E = Elem<DT>;
  using V = Vec<DT, E::kPer16>;
  const int64_t unit = p.unit0 + blockIdx.x;
  const int64_t r = unit / p.slices;
  const int sl = static_cast<int>(unit - r * p.slices);
  const int64_t lo = sl * p.slice, hi = lo + p.slice < p.n ? lo + p.slice : p.n;
  const typename E::T* x = static_cast<const typename E::T*>(p.x) + r * p.row_stride;
  bool greedy;
  const float scale = row_scale(p.temperature, r, &greedy);
  constexpr int N = E::kPer16;
  float2 a = make_float2(kNegInf, greedy ? __uint_as_float(0xFFFFFFFFu) : 0.0f);
  double sum = 0.0;  // a thread's terms may be thousands: equal ones added in fp32 are all rounded to one side
  for (int64_t i = lo + static_cast<int64_t>(threadIdx.x) * N; i < hi; i += kSoftWaves * 64 * N) {
    float v[N];
    if (i + N <= hi) {
      const typename V::type q = *reinterpret_cast<const typename V::unaligned*>(x + i);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = E::widen(q[j]);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = i + j < hi ? E::widen(x[i + j]) : kNegInf;
    }
    if (greedy) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (v[j] > a.x) a = make_float2(v[j], __uint_as_float(static_cast<uint32_t>(i + j)));
    } else {
      float m = a.x;
#pragma unroll
      for (int j = 0; j < N; ++j) m = fmaxf(m, v[j]);
      if (m != kNegInf) {
        float z = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) z += soft_exp(v[j], m, scale);
        sum = sum * static_cast<double>(soft_exp(a.x, m, scale)) + static_cast<double>(z);
        a.x = m;
      }
    }
  }
  if (!greedy) a.y = static_cast<float>(sum);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float2 b = wave_xor(a, o);
    a = greedy ? first_join(a, b) : soft_join(a, b, scale);
  }
  __shared__ float2 of_wave[kSoftWaves];
  if ((threadIdx.x & 63) == 0) of_wave[threadIdx.x >> 6] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kSoftWaves; ++w) a = greedy ? first_join(a, of_wave[w]) : soft_join(a, of_wave[w], scale);
    p.part[unit] = a;
  }
}

// One workgroup per (row, slice): joins the row's parts and writes the slice.
template <int DT, int OT>
__global__ __launch_bounds__(kSoftWaves * 64) void softmax_write_kernel(SoftmaxParams p) {
  using E = Elem<DT>;
  using O = Elem<OT>;
  constexpr int N = E::kPer16;
  using V = Vec<DT, N>;
  using W = Vec<OT, N>;
  const int64_t unit = p.unit0 + blockIdx.x;
  const int64_t r = unit / p.slices;
  const int sl = static_cast<int>(unit - r * p.slices);
  const int64_t lo = sl * p.slice, hi = lo + p.slice < p.n ? lo + p.slice : p.n;
  const typename E::T* x = static_cast<const typename E::T*>(p.x) + r * p.row_stride;
  typename O::T* out = static_cast<typename O::T*>(p.out) + r * p.out_stride;
  bool greedy;
  const float scale = row_scale(p.temperature, r, &greedy);
  const float2* part = p.part + r * p.slices;
  const int lane = threadIdx.x & 63;
  float2 a = make_float2(kNegInf, greedy ? __uint_as_float(0xFFFFFFFFu) : 0.0f);
  for (int i = lane; i < p.slices; i += 64) a = greedy ? first_join(a, part[i]) : soft_join(a, part[i], scale);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float2 b = wave_xor(a, o);
    a = greedy ? first_join(a, b) : soft_join(a, b, scale);
  }
  // (the lanes' joins round differently: one lane's sum is everyone's)
  a.x = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(a.x)));
  a.y = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(a.y)));
  const bool empty = a.x == kNegInf;
  const int64_t first = greedy && !empty ? static_cast<int64_t>(__float_as_uint(a.y)) : -1;
  const float inv = greedy || empty ? 0.0f : 1.0f / a.y;
  for (int64_t i = lo + static_cast<int64_t>(threadIdx.x) * N; i < hi; i += kSoftWaves * 64 * N) {
    float v[N];
    const bool full = i + N <= hi;
    if (greedy || empty) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = i + j == first ? 1.0f : 0.0f;
    } else if (full) {
      const typename V::type q = *reinterpret_cast<const typename V::unaligned*>(x + i);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = soft_exp(E::widen(q[j]), a.x, scale) * inv;
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = i + j < hi ? soft_exp(E::widen(x[i + j]), a.x, scale) * inv : 0.0f;
    }
    if (full) {
      typename W::type q;
#pragma unroll
      for (int j = 0; j < N; ++j) q[j] = O::narrow(v[j]);
      *reinterpret_cast<typename W::unaligned*>(out + i) = q;
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (i + j < hi) out[i + j] = O::narrow(v[j]);
    }
  }
}

// A workgroup per row of at least N elements, which it reads from memory once where it can:
// each thread keeps R vectors in registers and LV in LDS, and only what is past them is read
// again for the output. Vector j of thread t holds elements (j * THREADS + t) * N on; a vector
// that would pass the row's end is moved back to end there (no branches around loads and
// stores: what it holds twice changes no maximum, is left out of the sum, and is written
// twice with the same value). 2^together workgroups may work out the same row and write each
// their part of the vectors.
template <int DT, int OT, int THREADS, int R, int LV>
__global__ __launch_bounds__(THREADS) void softmax_row_kernel(SoftmaxParams p) {
  using E = Elem<DT>;
  using O = Elem<OT>;
  using T = typename E::T;
  constexpr int N = E::kPer16, kWaves = THREADS / 64;
  constexpr uint32_t kStep = THREADS * N, kKept = (R + LV) * kStep;
  using V = Vec<DT, N>;
  using W = Vec<OT, N>;
  typedef typename V::type VT;
  __shared__ __attribute__((aligned(16))) VT kept[LV ? LV * THREADS : 1];
  __shared__ float of_wave[kWaves];
  __shared__ uint32_t first_of_wave[kWaves];
  const int64_t r = (p.unit0 + blockIdx.x) >> p.together;
  const int part = (p.unit0 + blockIdx.x) & ((1 << p.together) - 1);
  const auto ours = [&](int j) { return ((j ^ part) & ((1 << p.together) - 1)) == 0; };
  const T* x = static_cast<const T*>(p.x) + r * p.row_stride;
  typename O::T* out = static_cast<typename O::T*>(p.out) + r * p.out_stride;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  bool greedy;
  const float scale = row_scale(p.temperature, r, &greedy);
  // the kept vectors lie within 32 bits of the row's start
  const uint32_t n = p.n < 2 * static_cast<int64_t>(kKept) ? static_cast<uint32_t>(p.n) : 2 * kKept;
  uint32_t mine = threadIdx.x * N;
  const auto place = [&](uint32_t j) { return j * kStep + mine < n - N ? j * kStep + mine : n - N; };
  const auto load = [&](auto i) { return *reinterpret_cast<const typename V::unaligned*>(x + i); };
  const auto most = [](float m, VT v) {
#pragma unroll
    for (int j = 0; j < N; ++j) m = fmaxf(m, E::widen(v[j]));
    return m;
  };
  VT reg[R];
  float m = kNegInf, z = 0.0f;
  if constexpr (LV > 0) {
    // LDS vectors come first, B at a time: the registers' loads are under way meanwhile
    constexpr int B = LV % 4 == 0 ? 4 : 3;
    static_assert(LV % B == 0);
    VT ahead[B];
#pragma unroll
    for (int j = 0; j < B; ++j) ahead[j] = load(place(R + j));
#pragma unroll
    for (int j = 0; j < R; ++j) reg[j] = load(place(j));
#pragma unroll
    for (int b = 0; b < LV; b += B) {
#pragma unroll
      for (int j = 0; j < B; ++j) {
        kept[(b + j) * THREADS + threadIdx.x] = ahead[j];
        m = most(m, ahead[j]);
        if (b + B < LV) ahead[j] = load(place(R + b + B + j));
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < R; ++j) reg[j] = load(place(j));
  }
  // what is past the kept vectors: the running maximum and sum, four vectors at a time
  const int64_t past = kKept + static_cast<int64_t>(mine), end = p.n - N;
  const auto place64 = [&](int64_t i) { return i < end ? i : end; };
  // exp((v - top) / t) as exp2(v * scale - tops), tops = top * scale rounded once: what that is off by is
  // the same factor everywhere and divides out. Below 2^28 (kFar) it is off by at most 8, a factor that
  // takes no term or sum out of fp32's range; larger products are not used.
  constexpr float kFar = 0x1p28f;
  const auto term = [&](T v, float tops) { return __builtin_amdgcn_exp2f(fmaf(E::widen(v), scale, -tops)); };
  const auto sum_of = [&](VT v, int64_t back, float tops) {  // back: elements that another vector holds too
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) s += i >= back ? term(v[i], tops) : 0.0f;
    return s;
  };
  // A thread's running maximum may be any finite number (a mask), of which no product can be
  // rounded harmlessly: here the difference is taken first. (Infinite maxima and inverse
  // temperatures make NaN here; their rows are summed again below.)
  // The sum is kept in double: a thread of a very long row has thousands of terms, and equal ones
  // added in fp32 are all rounded to one side.
  double past_sum = 0.0;
  for (int64_t at = past; at - mine < p.n; at += 4 * kStep) {
    VT v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = load(place64(at + j * kStep));
    float top = m;
#pragma unroll
    for (int j = 0; j < 4; ++j) top = most(top, v[j]);
    if (top != kNegInf) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t back = at + j * kStep - place64(at + j * kStep);
#pragma unroll
        for (int i = 0; i < N; ++i)
          s += i >= back ? __builtin_amdgcn_exp2f(apart(E::widen(v[j][i]), top, scale)) : 0.0f;
      }
      past_sum = past_sum * static_cast<double>(__builtin_amdgcn_exp2f(apart(m, top, scale))) + static_cast<double>(s);
    }
    m = top;
  }
  const float own = m, own_sum = static_cast<float>(past_sum);
  // (places are worked out anew in each phase: kept, they would take a register per vector)
  asm volatile("" : "+v"(mine));
#pragma unroll
  for (int j = 0; j < R; ++j) m = most(m, reg[j]);
  m = wave_max(m);
  if (lane == 0) of_wave[wave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) m = fmaxf(m, of_wave[w]);
  __syncthreads();
  if (greedy || m == kNegInf) {  // one-hot at the first maximum, or nothing (n fits 31 bits)
    uint32_t hot = 0xFFFFFFFFu;
    if (m != kNegInf) {
      const auto look = [&](VT v, uint32_t a) {
        uint32_t in = N;
#pragma unroll
        for (int j = N - 1; j >= 0; --j) in = E::widen(v[j]) == m ? j : in;
        hot = in < N && a + in < hot ? a + in : hot;
      };
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (j * kStep < n) look(reg[j], place(j));
      if constexpr (LV > 0) {
        for (int j = 0; j < LV; ++j)
          if ((R + j) * kStep < n) look(kept[j * THREADS + threadIdx.x], place(R + j));
      }
      for (int64_t i = past; i - mine < p.n && hot == 0xFFFFFFFFu; i += 4 * kStep) {
        VT v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = load(place64(i + j * kStep));
#pragma unroll
        for (int j = 0; j < 4; ++j) look(v[j], static_cast<uint32_t>(place64(i + j * kStep)));
      }
      hot = row_reduce<6>(hot, [](uint32_t u, uint32_t w) { return u < w ? u : w; });
      if (lane == 0) first_of_wave[wave] = hot;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWaves; ++w) hot = first_of_wave[w] < hot ? first_of_wave[w] : hot;
    }
    for (int64_t i = mine + part * static_cast<int64_t>(kStep); i < p.n; i += static_cast<int64_t>(kStep) << p.together) {
      const int64_t a = place64(i);
      const uint32_t in = hot - static_cast<uint32_t>(a);
      typename W::type o;
#pragma unroll
      for (int j = 0; j < N; ++j) o[j] = O::narrow(in == static_cast<uint32_t>(j) ? 1.0f : 0.0f);
      *reinterpret_cast<typename W::unaligned*>(out + a) = o;
    }
    return;
  }
  const float ms = m * scale;
  const auto block_sum = [&](float v) {
    v = wave_sum(v);
    if (lane == 0) of_wave[wave] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += of_wave[w];
    return v;
  };
  if (!(fabsf(ms) < kFar)) {  // far logits, tiny temperatures, infinities: differences, element by element
    double sum = 0.0;
    for (int64_t i = mine; i < p.n; i += kStep) {
      const int64_t a = place64(i);
      const VT v = load(a);
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) s += a + j >= i ? soft_exp(E::widen(v[j]), m, scale) : 0.0f;
      sum += static_cast<double>(s);
    }
    const float inv = 1.0f / block_sum(static_cast<float>(sum));
    for (int64_t i = mine + part * static_cast<int64_t>(kStep); i < p.n; i += static_cast<int64_t>(kStep) << p.together) {
      const int64_t a = place64(i);
      const VT v = load(a);
      typename W::type o;
#pragma unroll
      for (int j = 0; j < N; ++j) o[j] = O::narrow(soft_exp(E::widen(v[j]), m, scale) * inv);
      *reinterpret_cast<typename W::unaligned*>(out + a) = o;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const bool whole = (j + 1) * kStep <= n;
    if constexpr (DT == DS_FP32) {  // the registers hold exp from here on (bf16 has no room for it)
#pragma unroll
      for (int i = 0; i < N; ++i) reg[j][i] = term(reg[j][i], ms);
      if (whole) {
#pragma unroll
        for (int i = 0; i < N; ++i) z += reg[j][i];
      } else {
        const uint32_t back = j * kStep + mine - place(j);
#pragma unroll
        for (int i = 0; i < N; ++i) z += i >= back ? reg[j][i] : 0.0f;
      }
    } else if (whole) {
#pragma unroll
      for (int i = 0; i < N; ++i) z += term(reg[j][i], ms);
    } else {
      z += sum_of(reg[j], j * kStep + mine - place(j), ms);
    }
    __builtin_amdgcn_sched_barrier(0);  // vector by vector: more at a time takes more registers than there are
  }
  if constexpr (LV > 0) {
#pragma unroll
    for (int j = 0; j < LV; ++j)
      z += sum_of(kept[j * THREADS + threadIdx.x], (R + j) * kStep + mine - place(R + j), ms);
  }
  z += own_sum * __builtin_amdgcn_exp2f(fmaf(own, scale, -ms));  // to what `term` gives
  const float inv = 1.0f / block_sum(z);
  asm volatile("" : "+v"(mine));
  const auto store = [&](auto i, const float* q) {
    typename W::type o;
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = O::narrow(q[j]);
    const auto to = reinterpret_cast<typename W::unaligned*>(out + i);
    // past the caches, which keep more of the logits (256 x 129280 fp32: a call after another into one
    // buffer 50.3 -> 48.4 us, from a graph into 15 in turn 56.5 -> 53.8), where a store writes whole lines (two stores of bf16 to fp32 share one: 26.9 -> 32.3 us at 128 rows)
    if constexpr (sizeof(o) <= 16) __builtin_nontemporal_store(o, to);
    else *to = o;
  };
#pragma unroll
  for (int j = 0; j < R; ++j)
    if (j * kStep < n && ours(j)) {
      float q[N];
#pragma unroll
      for (int i = 0; i < N; ++i)
        q[i] = (DT == DS_FP32 ? E::widen(reg[j][i]) : term(reg[j][i], ms)) * inv;
      store(place(j), q);
      __builtin_amdgcn_sched_barrier(0);
    }
  const auto finish = [&](auto i, VT v) {
    float q[N];
#pragma unroll
    for (int j = 0; j < N; ++j) q[j] = term(v[j], ms) * inv;
    store(i, q);
  };
  if constexpr (LV > 0) {
#pragma unroll
    for (int j = 0; j < LV; ++j)
      if ((R + j) * kStep < n) finish(place(R + j), kept[j * THREADS + threadIdx.x]);
  }
  for (int64_t at = past; at - mine < p.n; at += 4 * kStep) {
    VT v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = load(place64(at + j * kStep));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (at + j * kStep - mine < p.n) finish(place64(at + j * kStep), v[j]);
  }
}

// One workgroup per (row, slice of the output): every workgroup of a row works out the list's
// probabilities (in double: the prefix's end is exact), clears its slice and writes the
// entries that fall in it. Where a slice takes longer to clear than a short list takes one wave,
// one wave works on the list while the others clear (LW = 1: a wave's loads wait for its own
// earlier stores, so that all doing both took 22 us where the clearing of 256 x 129280 fp32
// takes 17.4; this way 19.0). Elsewhere all waves share the list and clear after it (one list
// of 512: 5.8 us, by one wave 7.4).
constexpr int kListWaves = 8;
constexpr int kListThreads = kListWaves * 64;
constexpr int kOneWaveList = 512;
constexpr int64_t kOneWaveBytes = 128 * 1024;

template <int DT, int OT, int LW>
__global__ __launch_bounds__(kListThreads) void list_softmax_kernel(ListSoftmaxParams p) {
  using E = Elem<DT>;
  using O = Elem<OT>;
  constexpr int kPer = (LW == 1 ? kOneWaveList : DS_MAX_K) / (LW * 64);  // entries per thread, consecutive
  __shared__ double of_wave[LW];
  __shared__ int first_of_wave[LW];
  const int64_t unit = p.unit0 + blockIdx.x;
  const int64_t r = unit / p.slices;
  const int sl = static_cast<int>(unit - r * p.slices);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t lo = sl * p.slice, hi = lo + p.slice < p.n ? lo + p.slice : p.n;
  typename O::T* out = static_cast<typename O::T*>(p.out) + r * p.out_stride;
  constexpr int N = O::kPer16;
  using W = Vec<OT, N>;
  const auto clear = [&](int thread, int threads) {
    for (int64_t i = lo + static_cast<int64_t>(thread) * N; i < hi; i += threads * N) {
      if (i + N <= hi) {
        *reinterpret_cast<typename W::unaligned*>(out + i) = typename W::type(0);
      } else {
        for (int j = 0; i + j < hi; ++j) out[i + j] = O::narrow(0.0f);
      }
    }
  };
  // sums and minima over the waves that have the list
  const auto all_sum = [&](double v) {
    v = wave_sum(v);
    if constexpr (LW > 1) {
      __syncthreads();
      if (lane == 0) of_wave[wave] = v;
      __syncthreads();
      v = 0.0;
      for (int w = 0; w < LW; ++w) v += of_wave[w];
    }
    return v;
  };
  double e[kPer];
  int at[kPer];
  double inv = 0.0;
  const int per = (p.k + LW * 64 - 1) / (LW * 64);
  const int base = threadIdx.x * per;
  if (LW > 1 || wave == 0) {
    const typename E::T* vals = static_cast<const typename E::T*>(p.vals) + r * p.k;
    const int32_t* idx = p.idx + r * p.k;
    const float t = p.temperature ? p.temperature[r] : 1.0f;
    const bool greedy = p.temperature && !(p.temperature[r] > 0.0f);
    const float top_p = p.top_p ? p.top_p[r] : 0.0f;
    int used = p.ks ? p.ks[r] : p.k;
    used = used < 1 ? 1 : (used > p.k ? p.k : used);
    float v[kPer];
    int first = p.k;  // the first entry that names an element: the list's maximum
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = base + j;
      const bool held = j < per && i < p.k;
      at[j] = held ? idx[i] : -1;
      v[j] = held ? E::widen(vals[i]) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (base + j >= used || at[j] < 0 || at[j] >= p.n) at[j] = -1;
      if (at[j] >= 0 && first == p.k) first = base + j;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const int b = __shfl_xor(first, o);
      first = b < first ? b : first;
    }
    if constexpr (LW > 1) {
      if (lane == 0) first_of_wave[wave] = first;
      __syncthreads();
      for (int w = 0; w < LW; ++w) first = first_of_wave[w] < first ? first_of_wave[w] : first;
    }
    const float m = first < p.k ? E::widen(vals[first]) : kNegInf;
    double mine = 0.0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool live = at[j] >= 0 && m != kNegInf && (!greedy || base + j == first);
      e[j] = 0.0;
      if (j < per)  // (the same in every thread)
        e[j] = !live || v[j] == kNegInf ? 0.0  // (at an infinite temperature too)
               : v[j] == m ? 1.0
                           : exp((static_cast<double>(v[j]) - static_cast<double>(m)) / static_cast<double>(t));
      mine += e[j];
    }
    double total = all_sum(mine);
    if (p.top_p) {
      // the mass before each entry: the waves before this one, the lanes before this one, then
      // this thread's own entries
      double before = mine;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double b = __shfl_up(before, o);
        if (lane >= o) before += b;
      }
      before -= mine;
      if constexpr (LW > 1) {
        for (int w = 0; w < wave; ++w) before += of_wave[w];
      }
      // (all of the mass is in the whole list only, also where a double no longer shows an entry's share)
      const double most = top_p >= 1.0f ? __builtin_huge_val() : static_cast<double>(top_p) * total;
      mine = 0.0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const double q = e[j];
        if (!(before < most) && base + j != first) e[j] = 0.0;
        before += q;
        mine += e[j];
      }
      total = all_sum(mine);
    }
    inv = total > 0.0 ? 1.0 / total : 0.0;
    if (p.out_list && sl == 0) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (j < per && base + j < p.k) p.out_list[r * p.k + base + j] = static_cast<float>(e[j] * inv);
    }
    if (LW > 1 && p.out) clear(threadIdx.x, kListThreads);
  } else if (p.out) {
    clear(threadIdx.x - 64, kListThreads - 64);
  }
  if (!p.out) return;
  __syncthreads();  // the zeros are written before the entries go over them
  if (LW > 1 || wave == 0) {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (at[j] >= lo && at[j] < hi && e[j] > 0.0) out[at[j]] = O::narrow(static_cast<float>(e[j] * inv));
  }
}

}  // namespace

static RowCut cut_rows(int64_t rows, int64_t n, int64_t per_cu) {
  if (rows < 1) rows = 1;
  constexpr int64_t step = kSoftWaves * 64 * 8;
  const int64_t most = (n + step - 1) / step, want = (kCus * per_cu + rows - 1) / rows;
  const int64_t slices = want < 1 ? 1 : (want > most ? most : want);
  const int64_t slice = ((n + slices - 1) / slices + step - 1) / step * step;
  return {slice, static_cast<int32_t>((n + slice - 1) / slice)};
}

// No slices (one workgroup per row, one launch) while a row is short or there are many; else
// slices and two launches. Both sides, in us, called one after the other from the host: 7 rows
// of 50001 bf16 7.9 and 11.6, 7 of 50001 fp32 11.4 and 12.0 (from a graph 11.6 and 8.2), 64 of
// 129280 fp32 19.9 and 21.1, 100 of them 24 and 33, one of 16384 fp32 7.8 and 12.
RowCut cut_softmax(int64_t rows, int64_t n, int dtype) {
  const int64_t bytes = n * (dtype == DS_BF16 ? 2 : 4);
  if (n >= 8 && (bytes <= 128 * 1024 || rows >= 48)) return {0, 0};  // (a row kernel's vectors hold up to 8)
  return cut_rows(rows, n, 4);
}

// Two workgroups a CU: each of a row's repeats the list (256 lists of 512 over 129280 fp32: one 19.6,
// two 19.0, four 23.4 us).
RowCut cut_list_softmax(int64_t rows, int64_t n) { return cut_rows(rows, n, 2); }

template <int DT, int OT>
static hipError_t softmax_out(SoftmaxParams p, hipStream_t s) {
  if (p.slices == 0) {
    // the fewest vectors a thread that hold the row: those past its end cost as much as others
    const int64_t vectors = (p.n + Elem<DT>::kPer16 - 1) / Elem<DT>::kPer16;
    if (vectors <= 256 * 4) return launch_units(softmax_row_kernel<DT, OT, 256, 4, 0>, p, p.rows, 256, s);
    if (vectors <= 256 * 8) return launch_units(softmax_row_kernel<DT, OT, 256, 8, 0>, p, p.rows, 256, s);
    // few rows: several workgroups per row, each with its share of the stores and of the second
    // exponentials, but not so many that reading each row that often costs more (8 workgroups for
    // each of 7 rows of 50001 bf16 10.0 -> 7.9 us; 2 for 32 of 32000 fp32 change nothing, 4 take
    // 7.0 us for 5.9), nor more than the vectors that a thread may hold: they would store nothing. (With
    // 5 to 7 of 8 vectors in the row, one to three of 8 workgroups store nothing: the other ones' single
    // vectors still make it faster than 4 with two, 8 rows of 40960 bf16 6.2 and 6.45 us.)
    if (vectors <= 1024 * 8) {
      const int most = vectors <= 1024 * 4 ? 4 : 8;
      while (2 << p.together <= most && p.rows << (p.together + 1) <= kCus / 4) ++p.together;
    }
    if (vectors <= 1024 * 4) return launch_units(softmax_row_kernel<DT, OT, 1024, 4, 0>, p, p.rows << p.together, 1024, s);
    if (vectors <= 1024 * 8) return launch_units(softmax_row_kernel<DT, OT, 1024, 8, 0>, p, p.rows << p.together, 1024, s);
    constexpr bool kTwo = DT == DS_BF16;  // (two bytes an element)
    return launch_units(softmax_row_kernel<DT, OT, 1024, kTwo ? 8 : 20, kTwo ? 8 : 9>, p, p.rows, 1024, s);
  }
  const int64_t units = p.rows * p.slices;
  const hipError_t e = launch_units(softmax_stats_kernel<DT>, p, units, kSoftWaves * 64, s);
  return e != hipSuccess ? e : launch_units(softmax_write_kernel<DT, OT>, p, units, kSoftWaves * 64, s);
}

template <int DT>
static hipError_t softmax_dt(int out_dtype, const SoftmaxParams& p, hipStream_t s) {
  return out_dtype == DS_BF16 ? softmax_out<DT, DS_BF16>(p, s) : softmax_out<DT, DS_FP32>(p, s);
}

hipError_t launch_softmax(int dtype, int out_dtype, const SoftmaxParams& p, hipStream_t s) {
  return dtype == DS_BF16 ? softmax_dt<DS_BF16>(out_dtype, p, s) : softmax_dt<DS_FP32>(out_dtype, p, s);
}

template <int DT, int OT>
static hipError_t list_softmax_out(const ListSoftmaxParams& p, hipStream_t s) {
  const int64_t units = p.rows * p.slices;
  const bool one = p.out && p.k <= kOneWaveList && p.slice * static_cast<int64_t>(sizeof(typename Elem<OT>::T)) >= kOneWaveBytes;
  return one ? launch_units(list_softmax_kernel<DT, OT, 1>, p, units, kListThreads, s)
                             : launch_units(list_softmax_kernel<DT, OT, kListWaves>, p, units, kListThreads, s);
}

hipError_t launch_list_softmax(int dtype, int out_dtype, const ListSoftmaxParams& p, hipStream_t s) {
  if (dtype == DS_BF16) return out_dtype == DS_BF16 ? list_softmax_out<DS_BF16, DS_BF16>(p, s) : list_softmax_out<DS_BF16, DS_FP32>(p, s);
  return out_dtype == DS_BF16 ? list_softmax_out<DS_FP32, DS_BF16>(p, s) : list_softmax_out<DS_FP32, DS_FP32>(p, s);
}

}  // namespace ds
