// Slots sorted by expert, rows gathered to their slots' positions and combined back, and the
// gradients of that.
#include "ds_expert.h"
#include "ds_rows_device.h"

namespace ds {
namespace {

// ------------------------------------------------------------------------------------- sort
// A stable counting sort: position = offsets[e] + slots of e in earlier chunks + in earlier
// waves of the chunk + in earlier lanes. A wave takes its slots in order, 64 at a time; lanes
// with equal experts find one another by ballots over the experts' bits, so no atomic decides a place.
// Up to 8192 slots one workgroup does it all (4 x 8 of 256 experts: 4.8 us, a chain of a dozen dependent LDS and
// memory accesses); above, a launch counts and one places (65536 x 8: 2.9 and 11.8 us, for 8 MB that take 2: the
// chain again. Neither the scattered 4-byte stores nor the sums over all chunks' counts show: with both confined to
// a few KB the time stays; chunks of half the size take as long with 16 waves and 1.5 us longer with eight).

__device__ __forceinline__ int expert_of(const SortParams& p, int64_t slot, int64_t end) {
  const int e = slot < end ? p.idx[slot] : -1;
  return static_cast<uint32_t>(e) < static_cast<uint32_t>(p.experts) ? e : -1;
}

constexpr int kTogether = 4;  // slots a lane loads at a time

// Counts of a chunk's slots by expert.
__global__ __launch_bounds__(1024) void sort_count_kernel(SortParams p) {
  __shared__ int hist[DS_MAX_EXPERTS];
  for (int e = threadIdx.x; e < p.experts; e += 1024) hist[e] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * p.chunk, hi = lo + p.chunk < p.slots ? lo + p.chunk : p.slots;
  for (int64_t s = lo + threadIdx.x; s < hi; s += 1024 * kTogether) {
    int e[kTogether];
#pragma unroll
    for (int i = 0; i < kTogether; ++i) e[i] = expert_of(p, s + i * 1024, hi);
#pragma unroll
    for (int i = 0; i < kTogether; ++i)
      if (e[i] >= 0) atomicAdd(&hist[e[i]], 1);
  }
  __syncthreads();
  const int wide = counts_wide(p.experts);
  for (int e = threadIdx.x; e < wide; e += 1024)
    p.counts[static_cast<int64_t>(blockIdx.x) * wide + e] = e < p.experts ? hist[e] : 0;
}

// Places of a chunk's slots. Every workgroup adds up all chunks' counts for itself (at most 256 chunks', from L2),
// which saves a launch.
template <int WAVES>
__global__ __launch_bounds__(WAVES * 64) void sort_place_kernel(SortParams p) {
  constexpr int T = WAVES * 64;
  extern __shared__ int lds[];
  const int E = p.experts, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int* mine = lds + wave * E;    // [WAVES][E]: the waves' counts, then their next positions
  int* total = lds + WAVES * E;  // [E]: slots of the expert
  int* before = total + E;       // [E]: of them in earlier chunks
  int* start = before + E;       // [E + 1]: offsets
  __shared__ int wave_sums[WAVES];
  for (int i = tid; i < (WAVES + 2) * E; i += T) lds[i] = 0;
  __syncthreads();

  const int64_t lo = blockIdx.x * p.chunk, hi = lo + p.chunk < p.slots ? lo + p.chunk : p.slots;
  const int64_t sub = ((hi - lo + WAVES - 1) / WAVES + 63) / 64 * 64;
  const int64_t wlo = lo + wave * sub < hi ? lo + wave * sub : hi, whi = wlo + sub < hi ? wlo + sub : hi;
  for (int64_t s = wlo + lane; s < whi; s += 64 * kTogether) {
    int e[kTogether];
#pragma unroll
    for (int i = 0; i < kTogether; ++i) e[i] = expert_of(p, s + i * 64, whi);
#pragma unroll
    for (int i = 0; i < kTogether; ++i)
      if (e[i] >= 0) atomicAdd(&mine[e[i]], 1);
  }
  if (p.chunks > 1) {
    // a thread adds up four experts' counts of every so many-th chunk
    const int quads = counts_wide(E) / 4, every = T / quads, from = tid / quads, e = (tid - from * quads) * 4;
    int all[4] = {}, early[4] = {};
    if (from < every) {
#pragma unroll 8
      for (int c = from; c < p.chunks; c += every) {
        const int4 v = *reinterpret_cast<const int4*>(p.counts + static_cast<int64_t>(c) * quads * 4 + e);
        const bool before_this = c < static_cast<int>(blockIdx.x);
        const int q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          all[i] += q[i];
          early[i] += before_this ? q[i] : 0;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e + i < E) {
          atomicAdd(&total[e + i], all[i]);
          atomicAdd(&before[e + i], early[i]);
        }
    }
    __syncthreads();
  } else {
    __syncthreads();
    for (int e = tid; e < E; e += T) {
      int t = 0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) t += lds[w * E + e];
      total[e] = t;
    }
    __syncthreads();
  }

  // offsets: an exclusive sum of the padded counts, a run of experts a thread
  const int per = (E + T - 1) / T, e0 = tid * per, e1 = e0 + per < E ? e0 + per : E;
  const auto room = [&](int n) { return p.align == 1 ? n : padded(n, p.align); };
  int run = 0;
  for (int e = e0; e < e1; ++e) run += room(total[e]);
  int incl = run;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 63) wave_sums[wave] = incl;
  __syncthreads();
  int at = incl - run;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) at += w < wave ? wave_sums[w] : 0;
  for (int e = e0; e < e1; ++e) {
    start[e] = at;
    at += room(total[e]);
    if (e == E - 1) start[E] = at;
  }
  __syncthreads();
  for (int e = tid; e < E; e += T) {
    int c[WAVES], next = start[e] + before[e];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) c[w] = lds[w * E + e];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      lds[w * E + e] = next;
      next += c[w];
    }
  }
  __syncthreads();

  // places
  const int bits = 32 - __clz(E);
  for (int64_t s0 = wlo + lane; s0 < wlo + sub && wlo < whi; s0 += 64 * kTogether) {
    int e[kTogether];
#pragma unroll
    for (int i = 0; i < kTogether; ++i) e[i] = expert_of(p, s0 + i * 64, whi);
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      const int64_t s = s0 + i * 64;
      uint64_t same = __ballot(e[i] >= 0);
      for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((e[i] >> b) & 1);
        same &= ((e[i] >> b) & 1) ? set : ~set;
      }
      int pos = -1;
      if (e[i] >= 0) pos = mine[e[i]] + __popcll(same & ((1ull << lane) - 1));
      wave_sync();
      if (e[i] >= 0 && (same >> lane) == 1) mine[e[i]] = pos + 1;  // the last of the equals
      wave_sync();
      if (s < whi) p.place[s] = pos;
      if (pos >= 0) p.order[pos] = static_cast<int>(s);
    }
  }

  // padding at the segments' ends, an expert a wave (a lane holds where one's padding lies), and what is
  // past the end
  if (p.align > 1) {
    const int step = p.chunks * WAVES;
    for (int first = blockIdx.x * WAVES + wave; first < E; first += step * 64) {
      const int e = first + lane * step;
      const int from = e < E ? start[e] + total[e] : 0, to = e < E ? start[e + 1] : 0;
      for (uint64_t left = __ballot(from < to); left; left &= left - 1) {
        const int l = __ffsll(static_cast<unsigned long long>(left)) - 1;
        const int64_t end = __builtin_amdgcn_readlane(to, l), begin = __builtin_amdgcn_readlane(from, l);
        for (int64_t i = begin + lane; i < end; i += 64) p.order[i] = -1;
      }
    }
  }
  for (int64_t i = start[E] + static_cast<int64_t>(blockIdx.x) * T + tid; i < p.capacity;
       i += static_cast<int64_t>(p.chunks) * T)
    p.order[i] = -1;
  if (blockIdx.x == 0)
    for (int e = tid; e <= E; e += T) p.offsets[e] = start[e];
}

// ----------------------------------------------------------------------------------- rows
// A team of LANES lanes takes a row; its lanes take the row's 16-byte vectors in turn and the
// elements past the last whole vector one each.

__device__ __forceinline__ int position(const Plan& q, int64_t slot) {
  const int pos = q.place[slot];
  return pos >= 0 && pos < q.capacity ? pos : -1;
}

// Clears the padding rows of 16 of the last align - 1 positions of a segment (unit: expert, then
// sixteenths), `bytes` long; `also(position)` runs for each with all threads.
constexpr int kPadRun = 16;
__device__ __forceinline__ int pad_parts(int align) { return (align - 1 + kPadRun - 1) / kPadRun; }

template <class F>
__device__ __forceinline__ void for_padding(const Plan& q, int64_t unit, F&& each) {
  const int parts = pad_parts(q.align), e = static_cast<int>(unit / parts), part = static_cast<int>(unit % parts);
  const int64_t cap = q.capacity;
  int64_t lo = q.offsets[e], hi = q.offsets[e + 1];
  lo = lo < 0 ? 0 : lo;
  hi = hi < cap ? hi : cap;
  const int64_t at = hi - (part + 1) * kPadRun + (threadIdx.x & (kPadRun - 1));
  bool pad = false;
  if (at >= lo && at >= hi - (q.align - 1)) {
    const int s = q.order[at];
    pad = s < 0 || s >= q.rows * q.k;
  }
  uint32_t mask = static_cast<uint32_t>(__ballot(pad)) & 0xFFFFu;
  while (mask) {
    const int i = __ffs(mask) - 1;
    mask &= mask - 1;
    each(hi - (part + 1) * kPadRun + i);
  }
}

template <int DT>
__device__ __forceinline__ void clear_row(typename Elem<DT>::T* row, int64_t n) {
  constexpr int V = Elem<DT>::kPer16;
  using Vt = Vec<DT, V>;
  const int64_t whole = n / V;
  typename Vt::type z = {};
  for (int64_t v = threadIdx.x; v < whole; v += 256) *reinterpret_cast<typename Vt::unaligned*>(row + v * V) = z;
  if (whole * V + threadIdx.x < n) row[whole * V + threadIdx.x] = 0;
}

// A team's row; of whole waves it is the same in all lanes, so that places and weights are read as scalars.
template <int LANES>
__device__ __forceinline__ int64_t team_row(int64_t unit) {
  const int64_t r = unit * (256 / LANES) + threadIdx.x / LANES;
  if constexpr (LANES < 64) return r;
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(r));
  return static_cast<int64_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(r >> 32))) << 32 | lo;
}

// A row is read once and written to all its slots' positions, a few vectors a lane at a time, past the caches.
// Bound by the stores: 8192 x 8 rows of 4096 bf16, 640 MB, 108 us on the GPU, 5.9 TB/s of both ways (ordinary
// stores: 6 us more; walking order instead would read each row k times).
constexpr int kHeld = 4;
template <int DT, int LANES>
__global__ __launch_bounds__(256) void gather_kernel(MoveParams p) {
  using T = typename Elem<DT>::T;
  constexpr int V = Elem<DT>::kPer16;
  using Vt = Vec<DT, V>;
  const int64_t unit = p.unit0 + blockIdx.x;
  T* out = static_cast<T*>(p.out);
  if (unit < p.pad_units) {
    for_padding(p.plan, unit, [&](int64_t at) { clear_row<DT>(out + at * p.out_stride, p.n); });
    return;
  }
  const int64_t r = team_row<LANES>(unit - p.pad_units);
  if (r >= p.plan.rows) return;
  const int lane = threadIdx.x % LANES, k = p.plan.k;
  const T* x = static_cast<const T*>(p.x) + r * p.x_stride;
  const int64_t whole = p.n / V, slot = r * k;
  for (int64_t v0 = lane; v0 < whole; v0 += LANES * kHeld) {
    typename Vt::type d[kHeld];
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (v0 + h * LANES < whole) d[h] = *reinterpret_cast<const typename Vt::unaligned*>(x + (v0 + h * LANES) * V);
    for (int j = 0; j < k; ++j) {
      const int64_t at = position(p.plan, slot + j);
      if (at < 0) continue;
      T* to = out + at * p.out_stride;
#pragma unroll
      for (int h = 0; h < kHeld; ++h)
        if (v0 + h * LANES < whole)
          __builtin_nontemporal_store(d[h], reinterpret_cast<typename Vt::unaligned*>(to + (v0 + h * LANES) * V));
    }
  }
  for (int64_t i = whole * V + lane; i < p.n; i += LANES) {
    const T d = x[i];
    for (int j = 0; j < k; ++j) {
      const int64_t at = position(p.plan, slot + j);
      if (at >= 0) out[at * p.out_stride + i] = d;
    }
  }
}

// Rows of y are read once, past the caches (ordinary loads: 11 us more): eight slots' at a time, so that their
// loads wait together (one at a time: 13 us more). Bound by the reading: 8192 x 8 rows of 4096 bf16, 605 MB, 111 us,
// 5.5 TB/s.
constexpr int kSlots = 8;
template <int DT, int LANES>
__global__ __launch_bounds__(256) void combine_kernel(MoveParams p) {
  using T = typename Elem<DT>::T;
  constexpr int V = Elem<DT>::kPer16;
  using Vt = Vec<DT, V>;
  const int64_t r = team_row<LANES>(p.unit0 + blockIdx.x);
  if (r >= p.plan.rows) return;
  const int lane = threadIdx.x % LANES, k = p.plan.k;
  const T* y = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out) + r * p.out_stride;
  const int64_t whole = p.n / V, slot = r * k;
  const auto weight = [&](int j) { return p.weights ? p.weights[slot + j] : 1.0f; };
  for (int64_t v = lane; v < whole; v += LANES) {
    float acc[V] = {};
    for (int j0 = 0; j0 < k; j0 += kSlots) {
      typename Vt::type d[kSlots];
      float w[kSlots];
      int64_t at[kSlots];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        at[j] = j0 + j < k ? position(p.plan, slot + j0 + j) : -1;
        w[j] = at[j] >= 0 ? weight(j0 + j) : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (at[j] >= 0)
          d[j] = __builtin_nontemporal_load(reinterpret_cast<const typename Vt::unaligned*>(y + at[j] * p.x_stride + v * V));
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (at[j] >= 0)
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(w[j], Elem<DT>::widen(d[j][i]), acc[i]);
    }
    typename Vt::type o;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = Elem<DT>::narrow(acc[i]);
    __builtin_nontemporal_store(o, reinterpret_cast<typename Vt::unaligned*>(out + v * V));
  }
  for (int64_t i = whole * V + lane; i < p.n; i += LANES) {
    float acc = 0;
    for (int j = 0; j < k; ++j) {
      const int64_t at = position(p.plan, slot + j);
      if (at >= 0) acc = __builtin_fmaf(weight(j), Elem<DT>::widen(y[at * p.x_stride + i]), acc);
    }
    out[i] = Elem<DT>::narrow(acc);
  }
}

// One wave a row: it holds up to 8 vectors a lane of g while it goes through the slots (a longer row's parts
// one after another), reads y's row, adds their products, and writes the gradient's. So g is read once and no
// barrier is met. Bound by memory both ways: 8192 x 8 rows of 4096 bf16, 1.18 GB, 232 us, 5.1 TB/s (a copy
// reaches as much).
template <int DT, int NV>
__global__ __launch_bounds__(256) void combine_grad_kernel(MoveParams p) {
  using T = typename Elem<DT>::T;
  constexpr int V = Elem<DT>::kPer16;
  using Vt = Vec<DT, V>;
  const int64_t unit = p.unit0 + blockIdx.x;
  T* out = static_cast<T*>(p.out);
  if (unit < p.pad_units) {
    for_padding(p.plan, unit, [&](int64_t at) { clear_row<DT>(out + at * p.out_stride, p.n); });
    return;
  }
  const int64_t r = team_row<64>(unit - p.pad_units);
  if (r >= p.plan.rows) return;
  const int lane = threadIdx.x % 64, k = p.plan.k;
  const T* g = static_cast<const T*>(p.g) + r * p.g_stride;
  const T* y = static_cast<const T*>(p.x);
  const int64_t whole = p.n / V, slot = r * k;
  float mine = 0;  // lane j: the gradient of slot j's weight
  for (int64_t v0 = lane;; v0 += 64 * NV) {
    typename Vt::type d[NV];
#pragma unroll
    for (int h = 0; h < NV; ++h)
      if (v0 + h * 64 < whole) d[h] = *reinterpret_cast<const typename Vt::unaligned*>(g + (v0 + h * 64) * V);
    const bool last = v0 - lane + 64 * NV >= whole;  // the elements past the last whole vector go with it
    const int64_t tail = whole * V + lane;
    const bool one = last && tail < p.n;
    const float gt = one ? Elem<DT>::widen(g[tail]) : 0.0f;
    for (int j = 0; j < k; ++j) {
      const int64_t at = position(p.plan, slot + j);
      if (at < 0) continue;
      if (p.out_weights) {
        const T* from = y + at * p.x_stride;
        typename Vt::type e[NV];
#pragma unroll
        for (int h = 0; h < NV; ++h)
          if (v0 + h * 64 < whole)
            e[h] = __builtin_nontemporal_load(reinterpret_cast<const typename Vt::unaligned*>(from + (v0 + h * 64) * V));
        float dot = one ? gt * Elem<DT>::widen(from[tail]) : 0.0f;
#pragma unroll
        for (int h = 0; h < NV; ++h)
          if (v0 + h * 64 < whole)
#pragma unroll
            for (int i = 0; i < V; ++i) dot = __builtin_fmaf(Elem<DT>::widen(d[h][i]), Elem<DT>::widen(e[h][i]), dot);
        const float sum = wave_sum(dot);
        if (lane == j) mine += sum;
      }
      if (out) {
        const float w = p.weights ? p.weights[slot + j] : 1.0f;
        T* to = out + at * p.out_stride;
#pragma unroll
        for (int h = 0; h < NV; ++h)
          if (v0 + h * 64 < whole) {
            typename Vt::type o;
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = Elem<DT>::narrow(w * Elem<DT>::widen(d[h][i]));
            __builtin_nontemporal_store(o, reinterpret_cast<typename Vt::unaligned*>(to + (v0 + h * 64) * V));
          }
        if (one) to[tail] = Elem<DT>::narrow(w * gt);
      }
    }
    if (last) break;
  }
  if (p.out_weights && lane < k) p.out_weights[slot + lane] = mine;
}

// Lanes of a team: what a row's vectors fill, up to a workgroup.
template <int DT>
int lanes_for(int64_t n) {
  const int64_t v = n / Elem<DT>::kPer16;
  return v <= 32 ? 16 : v <= 128 ? 64 : 256;
}

}  // namespace

SortCut cut_sort(int64_t slots) {
  // one workgroup up to 8192 slots; from there chunks of 4096, and at most 256 of them
  if (slots <= 8192) return {slots, 1};
  int64_t chunk = 4096;
  while ((slots + chunk - 1) / chunk > kCus) chunk *= 2;
  return {chunk, static_cast<int32_t>((slots + chunk - 1) / chunk)};
}

hipError_t launch_sort(const SortParams& p, hipStream_t s) {
  if (p.chunks > 1) {
    hipLaunchKernelGGL(sort_count_kernel, dim3(p.chunks), dim3(1024), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const auto bytes = [&](int waves) { return static_cast<size_t>((waves + 3) * p.experts + 1) * sizeof(int); };
  if (p.chunk <= 1024)
    hipLaunchKernelGGL(sort_place_kernel<4>, dim3(p.chunks), dim3(256), bytes(4), s, p);
  else if (p.experts > 512)  // the waves' counts within 64 KiB of LDS
    hipLaunchKernelGGL(sort_place_kernel<8>, dim3(p.chunks), dim3(512), bytes(8), s, p);
  else
    hipLaunchKernelGGL(sort_place_kernel<16>, dim3(p.chunks), dim3(1024), bytes(16), s, p);
  return hipGetLastError();
}

namespace {
int64_t pad_units_of(const Plan& q) {
  return static_cast<int64_t>(q.experts) * ((q.align - 1 + kPadRun - 1) / kPadRun);
}
int64_t teams(int64_t rows, int lanes) { return (rows + 256 / lanes - 1) / (256 / lanes); }

template <int DT>
hipError_t gather_of(MoveParams p, hipStream_t s) {
  const int lanes = lanes_for<DT>(p.n);
  p.pad_units = pad_units_of(p.plan);
  const int64_t units = p.pad_units + teams(p.plan.rows, lanes);
  return lanes == 16   ? launch_units(gather_kernel<DT, 16>, p, units, 256, s)
         : lanes == 64 ? launch_units(gather_kernel<DT, 64>, p, units, 256, s)
                       : launch_units(gather_kernel<DT, 256>, p, units, 256, s);
}

template <int DT>
hipError_t combine_of(MoveParams p, hipStream_t s) {
  const int lanes = lanes_for<DT>(p.n);
  const int64_t units = teams(p.plan.rows, lanes);
  return lanes == 16   ? launch_units(combine_kernel<DT, 16>, p, units, 256, s)
         : lanes == 64 ? launch_units(combine_kernel<DT, 64>, p, units, 256, s)
                       : launch_units(combine_kernel<DT, 256>, p, units, 256, s);
}

template <int DT>
hipError_t grad_of(const MoveParams& p, int64_t units, hipStream_t s) {
  const int64_t v = p.n / Elem<DT>::kPer16;  // vectors of a row
  return v <= 64    ? launch_units(combine_grad_kernel<DT, 1>, p, units, 256, s)
         : v <= 128 ? launch_units(combine_grad_kernel<DT, 2>, p, units, 256, s)
         : v <= 256 ? launch_units(combine_grad_kernel<DT, 4>, p, units, 256, s)
                    : launch_units(combine_grad_kernel<DT, 8>, p, units, 256, s);
}
}  // namespace

hipError_t launch_gather(int dtype, MoveParams p, hipStream_t s) {
  return dtype == DS_BF16 ? gather_of<DS_BF16>(p, s) : gather_of<DS_FP32>(p, s);
}

hipError_t launch_combine(int dtype, MoveParams p, hipStream_t s) {
  return dtype == DS_BF16 ? combine_of<DS_BF16>(p, s) : combine_of<DS_FP32>(p, s);
}

hipError_t launch_combine_grad(int dtype, MoveParams p, hipStream_t s) {
  p.pad_units = p.out ? pad_units_of(p.plan) : 0;
  const int64_t units = p.pad_units + teams(p.plan.rows, 64);
  return dtype == DS_BF16 ? grad_of<DS_BF16>(p, units, s) : grad_of<DS_FP32>(p, units, s);
}

}  // namespace ds
