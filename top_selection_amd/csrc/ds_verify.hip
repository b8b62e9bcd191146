// Verification of drafted tokens against the target's probabilities.
#include "ds_rows_device.h"

namespace ds {
namespace {

constexpr int kVerifyWaves = 8;
constexpr int kVerifyThreads = kVerifyWaves * 64;

// What the acceptance tests of sequence b decide; the same in every lane. `refused` is the
// position of the next token: its target row, and its draft row when it is below `len`.
struct Verdict {
  int len;      // drafts of the sequence
  int next;     // accepted drafts, and the row the next token is drawn from
};

template <int DT>
__device__ __forceinline__ Verdict judge(const VerifyParams& p, int64_t b, int lane) {
  using E = Elem<DT>;
  const typename E::T* target = static_cast<const typename E::T*>(p.target);
  const typename E::T* draft = static_cast<const typename E::T*>(p.draft);
  int len = p.lens ? p.lens[b] : p.drafts;
  len = len < 0 ? 0 : (len > p.drafts ? p.drafts : len);
  bool fails = false;
  if (lane < len) {
    const int32_t t = p.tokens[b * p.drafts + lane];
    fails = true;
    if (t >= 0 && t < p.n) {
      // both factors have at most 24 significant bits: the product is exact in double
      const double pt = E::widen(target[(b * (p.drafts + 1) + lane) * p.target_stride + t]);
      const double qt = draft ? E::widen(draft[(b * p.drafts + lane) * p.draft_stride + t]) : 1.0f;
      fails = !(static_cast<double>(p.accept_u[b * p.drafts + lane]) * qt < pt);
    }
  }
  const uint64_t bad = __ballot(fails);
  return {len, bad ? __builtin_ctzll(bad) : len};
}

// The rows the next token is drawn from: element i has mass max(p - q, 0).
template <int DT>
struct Rows {
  using E = Elem<DT>;
  using T = typename E::T;
  const T* p;
  const T* q;       // NULL: no draft row
  int64_t without;  // an element without mass (a refused certain draft), or -1

  __device__ __forceinline__ Rows(const VerifyParams& v, int64_t b, Verdict d) {
    p = static_cast<const T*>(v.target) + (b * (v.drafts + 1) + d.next) * v.target_stride;
    const bool refused = d.next < d.len;
    q = refused && v.draft ? static_cast<const T*>(v.draft) + (b * v.drafts + d.next) * v.draft_stride : nullptr;
    without = refused && !v.draft ? v.tokens[b * v.drafts + d.next] : -1;
  }
  __device__ __forceinline__ double mass(int64_t i, float pv, float qv) const {
    const double m = static_cast<double>(pv) - static_cast<double>(qv);
    return i == without || !(m > 0.0) ? 0.0 : m;
  }
  __device__ __forceinline__ double mass_at(int64_t i) const {
    return mass(i, E::widen(p[i]), q ? E::widen(q[i]) : 0.0f);
  }
};

template <class T>
__device__ __forceinline__ T block_total(T v, T* of_wave) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) of_wave[threadIdx.x >> 6] = v;
  __syncthreads();
  T t = 0;
  for (int w = 0; w < kVerifyWaves; ++w) t += of_wave[w];
  return t;
}

// One workgroup per (sequence, slice): the slice's residual mass and the target's own.
template <int DT>
__global__ __launch_bounds__(kVerifyThreads) void verify_sums_kernel(VerifyParams p) {
  using E = Elem<DT>;
  constexpr int N = E::kPer16;
  using V = Vec<DT, N>;
  __shared__ double of_wave[kVerifyWaves];
  const int64_t unit = p.unit0 + blockIdx.x;
  const int64_t b = unit / p.slices;
  const int sl = static_cast<int>(unit - b * p.slices);
  const Verdict d = judge<DT>(p, b, threadIdx.x & 63);
  const Rows<DT> rows(p, b, d);
  const int64_t lo = sl * p.slice, hi = lo + p.slice < p.n ? lo + p.slice : p.n;
  double rest = 0.0, whole = 0.0;
  for (int64_t i = lo + static_cast<int64_t>(threadIdx.x) * N; i < hi; i += kVerifyThreads * N) {
    if (i + N <= hi) {
      const typename V::type pv = *reinterpret_cast<const typename V::unaligned*>(rows.p + i);
      typename V::type qv = typename V::type(0);
      if (rows.q) qv = *reinterpret_cast<const typename V::unaligned*>(rows.q + i);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        rest += rows.mass(i + j, E::widen(pv[j]), E::widen(qv[j]));
        whole += static_cast<double>(E::widen(pv[j]));
      }
    } else {
      for (int64_t j = i; j < hi; ++j) rest += rows.mass_at(j), whole += static_cast<double>(E::widen(rows.p[j]));
    }
  }
  rest = block_total(rest, of_wave);
  whole = block_total(whole, of_wave);
  if (threadIdx.x == 0) {
    p.part[2 * unit] = rest;
    p.part[2 * unit + 1] = whole;
  }
}

// One workgroup per sequence: finds the slice in which the running sum passes the drawn
// point, then the element in it.
template <int DT>
__global__ __launch_bounds__(kVerifyThreads) void verify_pick_kernel(VerifyParams p) {
  __shared__ double of_wave[kVerifyWaves];
  __shared__ int64_t found[kVerifyWaves], last[kVerifyWaves];
  const int64_t b = p.unit0 + blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Verdict d = judge<DT>(p, b, lane);
  Rows<DT> rows(p, b, d);
  const double* part = p.part + 2 * b * p.slices;
  double total = 0.0;
  int which = 0;
  for (int i = 0; i < p.slices; ++i) total += part[2 * i];
  if (!(total > 0.0)) {  // no residual: draw from the target's row itself
    which = 1;
    rows.q = nullptr;
    rows.without = -1;
    total = 0.0;
    for (int i = 0; i < p.slices; ++i) total += part[2 * i + 1];
  }
  int64_t token = -1;
  if (total > 0.0) {
    const double point = static_cast<double>(p.sample_u[b]) * total;
    double before = 0.0;
    int sl = -1, at = 0;
    for (; at < p.slices; ++at) {  // the first slice whose end passes the point
      const double m = part[2 * at + which];
      if (m > 0.0) sl = at;
      if (before + m > point) break;
      before += m;
    }
    if (at == p.slices) before -= part[2 * sl + which];  // rounding: the last slice with mass
    const int64_t lo = sl * p.slice, hi = lo + p.slice < p.n ? lo + p.slice : p.n;
    const int64_t per = (hi - lo + kVerifyThreads - 1) / kVerifyThreads;
    const int64_t my_lo = lo + threadIdx.x * per < hi ? lo + threadIdx.x * per : hi;
    const int64_t my_hi = my_lo + per < hi ? my_lo + per : hi;
    double mine = 0.0;
    int64_t my_last = -1, my_found = INT64_MAX;
    for (int64_t i = my_lo; i < my_hi; ++i) {
      const double m = rows.mass_at(i);
      mine += m;
      if (m > 0.0) my_last = i;
    }
    double sum = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double other = __shfl_up(sum, o);
      if (lane >= o) sum += other;
    }
    if (lane == 63) of_wave[wave] = sum;
    __syncthreads();
    sum -= mine;
    for (int w = 0; w < wave; ++w) sum += of_wave[w];
    sum += before;
    for (int64_t i = my_lo; i < my_hi; ++i) {
      const double m = rows.mass_at(i);
      sum += m;
      if (m > 0.0 && sum > point) {
        my_found = i;
        break;
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const int64_t f = __shfl_xor(my_found, o), l = __shfl_xor(my_last, o);
      my_found = f < my_found ? f : my_found;
      my_last = l > my_last ? l : my_last;
    }
    if (lane == 0) found[wave] = my_found, last[wave] = my_last;
    __syncthreads();
    for (int w = 0; w < kVerifyWaves; ++w) {
      my_found = found[w] < my_found ? found[w] : my_found;
      my_last = last[w] > my_last ? last[w] : my_last;
    }
    token = my_found != INT64_MAX ? my_found : my_last;
  }
  for (int j = threadIdx.x; j <= p.drafts; j += kVerifyThreads)
    p.out_tokens[b * (p.drafts + 1) + j] =
        j < d.next ? p.tokens[b * p.drafts + j] : (j == d.next ? static_cast<int32_t>(token) : -1);
  if (threadIdx.x == 0) p.out_accepted[b] = d.next;
}

template <int DT>
hipError_t verify_dt(const VerifyParams& p, hipStream_t s) {
  const hipError_t e = launch_units(verify_sums_kernel<DT>, p, p.batch * p.slices, kVerifyThreads, s);
  return e != hipSuccess ? e : launch_units(verify_pick_kernel<DT>, p, p.batch, kVerifyThreads, s);
}

}  // namespace

RowCut cut_verify(int64_t batch, int64_t n) { return cut_softmax(batch, n); }

hipError_t launch_verify(int dtype, const VerifyParams& p, hipStream_t s) {
  return dtype == DS_BF16 ? verify_dt<DS_BF16>(p, s) : verify_dt<DS_FP32>(p, s);
}

}  // namespace ds
