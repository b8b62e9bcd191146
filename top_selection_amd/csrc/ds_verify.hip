// Verification of drafted tokens against the target's probabilities.
#include "ds_rows_device.h"

namespace ds {
namespace {

constexpr int kVerifyWaves = 16;
constexpr int kVerifyThreads = kVerifyWaves * 64;
constexpr int kVerifyLoads = 4;  // 16-byte loads of each row that a lane has in flight

// Rows are summed in units of consecutive elements, one wave per unit; the drawn token is
// found from the units' sums and by reading one unit again.
template <int DT>
constexpr int kVerifyUnit = 64 * Elem<DT>::kPer16 * kVerifyLoads;  // 1024 fp32 or 2048 bf16 elements
constexpr int kVerifyShort = 32;       // units of a row that counts as short
constexpr int kVerifyLdsUnits = 2048;  // units of a row that one workgroup draws from alone

// What the acceptance tests of a sequence decide; the same in every lane.
struct Verdict {
  int len;        // drafts of the sequence
  int next;       // accepted drafts, and the row the next token is drawn from
  int32_t token;  // the draft that was refused (next < len)
};

// The drafts' tokens and numbers are asked for together with the length, and all rows' elements
// together: two waits for memory, whatever the number of drafts.
template <int DT>
__device__ __forceinline__ Verdict judge(const VerifyParams& p, int64_t b, int lane) {
  using E = Elem<DT>;
  const typename E::T* target = static_cast<const typename E::T*>(p.target);
  const typename E::T* draft = static_cast<const typename E::T*>(p.draft);
  const int j = lane < p.drafts ? lane : 0;
  int len = p.lens ? p.lens[b] : p.drafts;
  const int32_t t = p.drafts ? p.tokens[b * p.drafts + j] : 0;
  const float u = p.drafts ? p.accept_u[b * p.drafts + j] : 0.0f;
  len = len < 0 ? 0 : (len > p.drafts ? p.drafts : len);
  bool fails = false;
  if (lane < len) {
    fails = true;
    if (t >= 0 && t < p.n) {
      // both factors have at most 24 significant bits: the product is exact in double
      const double pt = E::widen(target[(b * (p.drafts + 1) + lane) * p.target_stride + t]);
      const double qt = draft ? E::widen(draft[(b * p.drafts + lane) * p.draft_stride + t]) : 1.0f;
      fails = !(static_cast<double>(u) * qt < pt);
    }
  }
  const uint64_t bad = __ballot(fails);
  const int next = bad ? __builtin_ctzll(bad) : len;
  return {len, next, __shfl(t, next & 63)};
}

// The rows the next token is drawn from: element i has mass max(p - q, 0).
template <int DT>
struct Rows {
  using E = Elem<DT>;
  using T = typename E::T;
  static constexpr int N = E::kPer16;
  using V = Vec<DT, N>;
  const T* p;
  const T* q;       // NULL: no draft row
  int64_t without;  // an element without mass (a refused certain draft), or -1

  __device__ __forceinline__ Rows(const VerifyParams& v, int64_t b, Verdict d) {
    p = static_cast<const T*>(v.target) + (b * (v.drafts + 1) + d.next) * v.target_stride;
    const bool refused = d.next < d.len;
    q = refused && v.draft ? static_cast<const T*>(v.draft) + (b * v.drafts + d.next) * v.draft_stride : nullptr;
    without = refused && !v.draft ? d.token : -1;
  }

  // kOnce: past the caches, for rows that are long and read once (256 x 129280 fp32 42.5 -> 37.9 us;
  // short rows are better kept for the draw, 48 x 32003 bf16 7.6 and 8.5 us).
  template <bool kOnce>
  static __device__ __forceinline__ typename V::type load(const T* from) {
    const auto at = reinterpret_cast<const typename V::unaligned*>(from);
    if constexpr (kOnce) return __builtin_nontemporal_load(at);
    else return *at;
  }

  // The mass of element i; none past the end. The difference of two fp32 is taken in double: the
  // sums' terms must not be rounded.
  __device__ __forceinline__ double mass(int64_t i, int64_t n) const {
    if (i >= n || i == without) return 0.0;
    const double d = E::widen(p[i]);
    return fmax(d - (q ? static_cast<double>(E::widen(q[i])) : 0.0), 0.0);
  }

  // The mass of the lane's elements of a unit: vectors `step` elements apart, the lanes' first ones
  // `first` apart. A vector that would pass the row's end is moved back to end there, and what it
  // then holds a second time is left out: loads one by one under guards, for the last unit alone,
  // made that unit's wave the last. And few instructions, as a wave runs them once or twice and
  // has to fetch them: without a draft row q is 0, not a case of its own, and the draw looks at
  // one run's elements in as many lanes. From 27 to 14 KB of code in all (bf16): 48 x 32003 10.9 ->
  // 7.7 us, one sequence of 129280 fp32 8.8 -> 7.4, 256 of them 41 -> 37.9.
  template <int kFirst, int kStep, bool kOnce = false>
  __device__ __forceinline__ double share(int64_t unit, int64_t n, int lane) const {
    double t = 0.0;
    if (n < N) {  // a row shorter than a vector
      if (lane == 0) {
#pragma unroll 1
        for (int i = 0; i < n; ++i) t += mass(i, n);
      }
      return t;
    }
    const int most = unit + kVerifyUnit<DT> <= n ? kVerifyUnit<DT> : static_cast<int>(n - unit) - N;
    const int64_t left = without - unit;
    const int gone = left >= 0 && left < kVerifyUnit<DT> ? static_cast<int>(left) : -1;
    typename V::type pv[kVerifyLoads], qv[kVerifyLoads] = {};
    int at[kVerifyLoads];
#pragma unroll
    for (int u = 0; u < kVerifyLoads; ++u) {
      at[u] = lane * kFirst + u * kStep < most ? lane * kFirst + u * kStep : most;
      pv[u] = load<kOnce>(p + unit + at[u]);
    }
    if (q) {
#pragma unroll
      for (int u = 0; u < kVerifyLoads; ++u) qv[u] = load<kOnce>(q + unit + at[u]);
    }
    if (gone >= 0 || most < kVerifyUnit<DT>) {  // (the same in every lane)
#pragma unroll
      for (int u = 0; u < kVerifyLoads; ++u) {
        const int twice = lane * kFirst + u * kStep - at[u], none = gone < 0 ? -1 : gone - at[u];
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (j < twice || j == none) pv[u][j] = T(0);
      }
    }
#pragma unroll
    for (int u = 0; u < kVerifyLoads; ++u)
#pragma unroll
      for (int j = 0; j < N; ++j)
        t += fmax(static_cast<double>(E::widen(pv[u][j])) - static_cast<double>(E::widen(qv[u][j])), 0.0);
    return t;
  }

  template <bool kOnce>
  __device__ __forceinline__ double sum(int64_t unit, int64_t n, int lane) const {
    return wave_sum(share<N, 64 * N, kOnce>(unit, n, lane));  // in memory's order
  }
};

// v moved by a data-parallel pattern; lanes that it does not reach, or that the row mask leaves
// out, get 0.
template <int PATTERN, int ROWS>
__device__ __forceinline__ double moved(double v) {
  return __hiloint2double(
      __builtin_amdgcn_update_dpp(0, __double2hiint(v), PATTERN, ROWS, 0xF, true),
      __builtin_amdgcn_update_dpp(0, __double2loint(v), PATTERN, ROWS, 0xF, true));
}

// The sum up to and with each lane: shifts within the rows of 16 lanes, then each row's last
// sum to the next row, and the second row's to the upper half.
__device__ __forceinline__ double scan_lanes(double v) {
  v += moved<0x111, 0xF>(v);  // by 1
  v += moved<0x112, 0xF>(v);  // by 2
  v += moved<0x114, 0xF>(v);  // by 4
  v += moved<0x118, 0xF>(v);  // by 8
  v += moved<0x142, 0xA>(v);  // lane 15 of rows 0 and 2 to rows 1 and 3
  v += moved<0x143, 0xC>(v);  // lane 31 to rows 2 and 3
  return v;
}

__device__ __forceinline__ double of_lane(double v, int lane) {  // lane: the same everywhere
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                          __builtin_amdgcn_readlane(__double2loint(v), lane));
}

// One wave: the element that the point share * total falls on. sums: the units' masses, total
// their (positive) sum.
template <int DT>
__device__ __forceinline__ int32_t draw(const Rows<DT>& rows, const double* sums, int units, int64_t n, double total,
                                        double share, int lane) {
  constexpr int N = Elem<DT>::kPer16, kRun = kVerifyLoads * N;
  const double point = share * total;
  // the first unit whose end passes the point; by rounding none may: the last one with mass
  int unit = -1;
  double before = 0.0, start = 0.0;
  for (int c = 0; c < units; c += 64) {
    const double s = c + lane < units ? sums[c + lane] : 0.0;
    const double end = start + scan_lanes(s);
    const uint64_t some = __ballot(s > 0.0), past = some & __ballot(end > point);
    if (some) {
      const int l = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(some);
      unit = c + l;
      before = of_lane(end, l) - of_lane(s, l);
    }
    if (past) break;
    start = of_lane(end, 63);
  }
  // within the unit each lane takes a run of elements, and then each an element of the run that
  // the point falls in; the last lane or element with mass where by rounding none is past it
  int64_t first = static_cast<int64_t>(unit) * kVerifyUnit<DT>;
  const auto pass = [&](double m) {
    const double end = before + scan_lanes(m);
    const uint64_t some = __ballot(m > 0.0), past = some & __ballot(end > point);
    const int l = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(some | 1);
    before = of_lane(end, l) - of_lane(m, l);
    return l;
  };
  first += pass(rows.template share<kRun, N>(first, n, lane)) * kRun;
  return static_cast<int32_t>(first + pass(lane < kRun ? rows.mass(first + lane, n) : 0.0));
}

// The sum of the units' masses, in every lane of every wave.
__device__ __forceinline__ double sum_units(const double* sums, int units, int lane) {
  double t = 0.0;
  for (int i = lane; i < units; i += 64) t += sums[i];
  return wave_sum(t);
}

__device__ __forceinline__ void answer(const VerifyParams& p, int64_t b, Verdict d, int32_t token, int lane) {
  for (int j = lane; j <= p.drafts; j += 64)
    p.out_tokens[b * (p.drafts + 1) + j] = j < d.next ? p.tokens[b * p.drafts + j] : (j == d.next ? token : -1);
  if (lane == 0) p.out_accepted[b] = d.next;
}

// A workgroup sums all units of a sequence and draws; a residual without mass is given up for
// the target's row, and a row without mass gives -1.
template <int DT>
__device__ __forceinline__ void draw_alone(const VerifyParams& p, int64_t b, Verdict d, Rows<DT> rows, double* sums) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int units = static_cast<int>((p.n + kVerifyUnit<DT> - 1) / kVerifyUnit<DT>);
  double total = 0.0;
  for (int turn = 0; turn < 2; ++turn) {
    if (units > kVerifyShort) {
      for (int i = wave; i < units; i += kVerifyWaves) {
        const double s = rows.template sum<true>(static_cast<int64_t>(i) * kVerifyUnit<DT>, p.n, lane);
        if (lane == 0) sums[i] = s;
      }
    } else {
      for (int i = wave; i < units; i += kVerifyWaves) {
        const double s = rows.template sum<false>(static_cast<int64_t>(i) * kVerifyUnit<DT>, p.n, lane);
        if (lane == 0) sums[i] = s;
      }
    }
    __syncthreads();
    total = sum_units(sums, units, lane);
    if (total > 0.0) break;  // (the same in every wave)
    __syncthreads();
    rows.q = nullptr;
    rows.without = -1;
  }
  if (wave == 0) {
    const int32_t token = total > 0.0 ? draw(rows, sums, units, p.n, total, static_cast<double>(p.sample_u[b]), lane) : -1;
    answer(p, b, d, token, lane);
  }
}

// One workgroup per sequence.
template <int DT>
__global__ __launch_bounds__(kVerifyThreads) void verify_kernel(VerifyParams p) {
  __shared__ double sums[kVerifyLdsUnits];
  const int64_t b = p.unit0 + blockIdx.x;
  const Verdict d = judge<DT>(p, b, threadIdx.x & 63);
  draw_alone<DT>(p, b, d, Rows<DT>(p, b, d), sums);
}

// Few sequences: one workgroup per (sequence, slice of units) leaves the units' sums in the
// workspace, then one workgroup per sequence draws.
template <int DT>
__global__ __launch_bounds__(kVerifyThreads) void verify_sums_kernel(VerifyParams p) {
  const int64_t at = p.unit0 + blockIdx.x;
  const int64_t b = at / p.slices;
  const int sl = static_cast<int>(at - b * p.slices);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Verdict d = judge<DT>(p, b, lane);
  const Rows<DT> rows(p, b, d);
  const int64_t units = (p.n + kVerifyUnit<DT> - 1) / kVerifyUnit<DT>;
  const int64_t lo = sl * p.slice, hi = lo + p.slice < units ? lo + p.slice : units;
  if (sl == 0 && threadIdx.x == 0) p.verdicts[b] = make_int2(d.len | d.next << 16, d.token);
  for (int64_t i = lo + wave; i < hi; i += kVerifyWaves) {
    const double s = rows.template sum<false>(i * kVerifyUnit<DT>, p.n, lane);
    if (lane == 0) p.part[b * units + i] = s;
  }
}

template <int DT>
__global__ __launch_bounds__(kVerifyThreads) void verify_draw_kernel(VerifyParams p) {
  __shared__ double near[kVerifyLdsUnits];
  const int64_t b = p.unit0 + blockIdx.x;
  const int lane = threadIdx.x & 63;
  const int units = static_cast<int>((p.n + kVerifyUnit<DT> - 1) / kVerifyUnit<DT>);
  double* const sums = p.part + b * units;
  const int2 v = p.verdicts[b];
  const Verdict d = {v.x & 0xFFFF, v.x >> 16, v.y};
  const Rows<DT> rows(p, b, d);
  const bool fits = units <= kVerifyLdsUnits;
  if (fits) {
    for (int i = threadIdx.x; i < units; i += kVerifyThreads) near[i] = sums[i];
    __syncthreads();
  }
  const double total = fits ? sum_units(near, units, lane) : sum_units(sums, units, lane);
  if (!(total > 0.0)) {  // (the same in every wave)
    __syncthreads();
    draw_alone<DT>(p, b, d, rows, sums);
  } else if (threadIdx.x < 64) {
    const double share = static_cast<double>(p.sample_u[b]);
    answer(p, b, d, fits ? draw(rows, near, units, p.n, total, share, lane)
                         : draw(rows, sums, units, p.n, total, share, lane), lane);
  }
}

template <int DT>
hipError_t verify_dt(const VerifyParams& p, hipStream_t s) {
  if (p.slices == 0) return launch_units(verify_kernel<DT>, p, p.batch, kVerifyThreads, s);
  const hipError_t e = launch_units(verify_sums_kernel<DT>, p, p.batch * p.slices, kVerifyThreads, s);
  return e != hipSuccess ? e : launch_units(verify_draw_kernel<DT>, p, p.batch, kVerifyThreads, s);
}

}  // namespace

// No slices (one workgroup per sequence, one launch) while a row is short or the sequences fill
// half the card by themselves; else slices of whole units. Both sides, fp32, drafts of 3: one
// sequence of 129280 in one workgroup 12.8 us, in slices 7.4; 64 sequences 28 and 18, 128 32 and 26,
// 192 35 and 40, 256 41 and 50.
VerifyCut cut_verify(int64_t batch, int64_t n, int dtype) {
  const int64_t unit = dtype == DS_BF16 ? kVerifyUnit<DS_BF16> : kVerifyUnit<DS_FP32>;
  const int64_t units = (n + unit - 1) / unit;
  if (units <= kVerifyShort || (batch > kCus / 2 && units <= kVerifyLdsUnits)) return {0, 0, 0};
  const int64_t want = batch >= kCus ? 1 : (kCus + batch - 1) / (batch < 1 ? 1 : batch);
  int64_t slice = (units + want - 1) / want;
  slice = (slice + kVerifyWaves - 1) / kVerifyWaves * kVerifyWaves;
  return {slice, static_cast<int32_t>((units + slice - 1) / slice),
          static_cast<size_t>(batch) * (units * sizeof(double) + sizeof(int2))};
}

hipError_t launch_verify(int dtype, VerifyParams p, hipStream_t s) {
  const int64_t unit = dtype == DS_BF16 ? kVerifyUnit<DS_BF16> : kVerifyUnit<DS_FP32>;
  if (p.slices) p.verdicts = reinterpret_cast<int2*>(p.part + p.batch * ((p.n + unit - 1) / unit));
  return dtype == DS_BF16 ? verify_dt<DS_BF16>(p, s) : verify_dt<DS_FP32>(p, s);
}

}  // namespace ds
