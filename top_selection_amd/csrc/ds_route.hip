// Routing to experts and its gradient.
#include <cmath>
#include <type_traits>

#include "ds_rows_device.h"

namespace ds {
namespace {

constexpr int kRouteWaves = 4;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr double kNone = -__builtin_huge_val();  // the selection score of a masked or taken expert
constexpr float kLog2E = 1.44269504088896341f;

__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// ------------------------------------------------------------------ the exact choice of a row
// A whole wave chooses for one row with everything that decides in double; expert e is in lane
// e % 64, lds: exact_room(64 V) bytes of LDS, the wave's own. groups_kept: 0, or the chosen
// groups where they are known (group g's bit is g << groups_step). Rows that the fast kernel cannot
// decide come here, and every row where no fast kernel fits. Out of line: its registers would
// otherwise count against the fast kernel's, which seldom calls it. It reads the parameters
// where the launch left them (a kernel's only argument), with scalar loads. A lone wave waits
// for every one of its instructions, so what is done per row is kept short: a row's time is
// the tail of a launch in which any row comes here.
__device__ __forceinline__ const void* params_of_launch() {
  return (const void*)__builtin_amdgcn_kernarg_segment_ptr();
}

__device__ __forceinline__ uint64_t uniform(uint64_t v) {
  return static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32)))) << 32 |
         static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v)));
}

// LDS bytes of a row with room for n experts: their scores, their indices, the lanes' best.
__host__ __device__ constexpr int exact_room(int n) { return n * 12 + 64 * 4; }

// The two largest of a group's selection scores.
struct Top2 {
  double a, b;
};
__device__ __forceinline__ Top2 join(Top2 u, Top2 v) {
  const double lo = u.a > v.a ? v.a : u.a, next = u.b > v.b ? u.b : v.b;
  return {u.a > v.a ? u.a : v.a, lo > next ? lo : next};
}
template <int LEVEL>
__device__ __forceinline__ Top2 from_partner(Top2 v) {
  return {from_partner<LEVEL>(v.a), from_partner<LEVEL>(v.b)};
}

template <int DT, int SCORE, int V>
__device__ __noinline__ void route_row_exact(const void* params, int64_t row, uint8_t* lds, uint64_t groups_kept,
                                             int groups_step) {
  using E = Elem<DT>;
  typedef const __attribute__((address_space(4))) RouteParams* ScalarParams;
  const ScalarParams p = (ScalarParams)uniform(reinterpret_cast<uint64_t>(params));
  const int64_t r = static_cast<int64_t>(uniform(static_cast<uint64_t>(row)));
  const typename E::T* x = static_cast<const typename E::T*>(p->x) + r * p->row_stride;
  const float* const biases = p->bias;
  const int experts = p->experts, k = p->k, groups = p->groups, size = p->group_size, topk_groups = p->topk_groups;
  const bool two = p->group_top > 1, renorm = p->renorm != 0;
  const float scale = p->scale;
  float* const out_weights = p->out_weights;
  int32_t* const out_idx = p->out_idx;
  // (as LDS addresses: a generic pointer's accesses take longer)
  const auto room = (__attribute__((address_space(3))) double*)reinterpret_cast<double*>(lds);
  const auto room_at = (__attribute__((address_space(3))) int32_t*)(room + 64 * V);
  const auto lane_best = (__attribute__((address_space(3))) float*)(room_at + 64 * V);
  const int lane = threadIdx.x & 63;
  float xv[V], bias[V];
  double s[V], c[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 64 + lane;
    xv[v] = e < experts ? E::widen(x[e]) : kNegInf;
    bias[v] = biases && e < experts ? biases[e] : 0.0f;
  }
  if constexpr (SCORE == DS_SCORE_SOFTMAX) {
    float m = kNegInf;
#pragma unroll
    for (int v = 0; v < V; ++v) m = fmaxf(m, xv[v]);
    m = row_reduce<6>(m, [](float a, float b) { return larger(a, b); });
    double z = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] = xv[v] == kNegInf ? 0.0 : xv[v] == m ? 1.0 : exp(static_cast<double>(xv[v]) - static_cast<double>(m));
      z += s[v];
      if (V > 4) __builtin_amdgcn_sched_barrier(0);  // one exp at a time: the registers of many cost more
    }
    z = row_reduce<6>(z, plus<double>);
    const double inv = z > 0.0 ? 1.0 / z : 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] *= inv;
  } else {
    float least = xv[0];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] = 1.0 / (1.0 + exp(-static_cast<double>(xv[v])));
      least = fminf(least, xv[v]);
      if (V > 4) __builtin_amdgcn_sched_barrier(0);
    }
    if (__any(least < -700.0f)) {  // exp(-x) overflows at 709: far below zero the score is exp(x)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (xv[v] < -700.0f) s[v] = exp(static_cast<double>(xv[v]));
        if (V > 4) __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  const bool limited = topk_groups < groups;
  // without a bias the order is that of the logits; sums of scores for the groups are not
  const bool sums = limited && !biases && two;
#pragma unroll
  for (int v = 0; v < V; ++v)
    c[v] = xv[v] == kNegInf ? kNone
           : biases         ? s[v] + static_cast<double>(bias[v])
                            : static_cast<double>(xv[v]);
  uint64_t keep = uniform(groups_kept);
  int levels = __builtin_amdgcn_readfirstlane(groups_step);
  if (limited && keep == 0) {
    wave_sync();
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * 64 + lane < experts) room[v * 64 + lane] = sums && c[v] != kNone ? s[v] : c[v];
    wave_sync();
    levels = 6;  // 2^levels lanes share a group
    while ((64 >> levels) < groups) --levels;
    const int group = lane >> levels, part = lane & ((1 << levels) - 1);
    Top2 top = {kNone, kNone};
    if (group < groups)
      for (int j = part; j < size; j += 1 << levels)
        top = join(top, Top2{room[group * size + j], kNone});
    if (levels > 0) top = join(top, from_partner<0>(top));
    if (levels > 1) top = join(top, from_partner<1>(top));
    if (levels > 2) top = join(top, from_partner<2>(top));
    if (levels > 3) top = join(top, from_partner<3>(top));
    if (levels > 4) top = join(top, from_partner<4>(top));
    if (levels > 5) top = join(top, from_partner<5>(top));
    const double score = two && top.b != kNone ? top.a + top.b : top.a;
    int rank = 0;
    for (int o0 = 0; o0 < groups; o0 += 8)
#pragma unroll
      for (int o = o0; o < o0 + 8; ++o) {
        const double other = __shfl(score, (o << levels) & 63);
        rank += (o < groups) & ((other > score) | ((other == score) & (o < group)));
      }
    keep = __ballot(group < groups && rank < topk_groups);
  }
  if (limited) {
    const float per_group = 1.0f / static_cast<float>(size);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int g = static_cast<int>((static_cast<float>(v * 64 + lane) + 0.5f) * per_group);
      if (!((keep >> ((g << levels) & 63)) & 1)) c[v] = kNone;
    }
  }
  // A bound that at least k experts reach, the k-th largest of the lanes' best (everything, if
  // fewer lanes hold any); rounded to fp32, as what is compared with it. The experts that reach
  // it are listed and ranked by counting.
  float best = kNegInf;
#pragma unroll
  for (int v = 0; v < V; ++v) best = fmaxf(best, static_cast<float>(c[v]));
  wave_sync();
  lane_best[lane] = best;
  wave_sync();
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  const auto four_best = (const __attribute__((address_space(3))) f32x4*)lane_best;
  int above = 0;
#pragma unroll
  for (int o = 0; o < 16; ++o) {
    const f32x4 q = four_best[o];
#pragma unroll
    for (int j = 0; j < 4; ++j) above += q[j] > best;
  }
  const float bound = -row_reduce<6>(above < k ? -best : kNegInf, [](float a, float b) { return larger(a, b); });
  int listed = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool in = c[v] > kNone && static_cast<float>(c[v]) >= bound;
    const uint64_t mask = __ballot(in);
    if (in) {
      const int at = listed + __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                                        __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0u));
      room[at] = c[v];
      room_at[at] = v * 64 + lane;
    }
    listed += __builtin_popcountll(mask);
  }
  wave_sync();
  int rank[V];
#pragma unroll
  for (int v = 0; v < V; ++v) rank[v] = 0;
#pragma unroll 2
  for (int o = 0; o < listed; ++o) {
    const double other = room[o];
    const int at = room_at[o];
#pragma unroll
    for (int v = 0; v < V; ++v) rank[v] += (other > c[v]) | ((other == c[v]) & (at < v * 64 + lane));
  }
  double total = 0.0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool in = c[v] > kNone && static_cast<float>(c[v]) >= bound;
    rank[v] = in ? rank[v] : k;
    total += rank[v] < k ? s[v] : 0.0;
  }
  total = row_reduce<6>(total, plus<double>);
  const double factor = static_cast<double>(scale);
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (rank[v] < k) {
      const double w = !renorm ? s[v] : total > 0.0 ? s[v] / total : 0.0;
      if (out_weights) out_weights[r * k + rank[v]] = static_cast<float>(w * factor);
      if (out_idx) out_idx[r * k + rank[v]] = v * 64 + lane;
    }
  if (lane >= listed && lane < k) {  // slots that no expert is left for
    if (out_weights) out_weights[r * k + lane] = 0.0f;
    if (out_idx) out_idx[r * k + lane] = -1;
  }
  wave_sync();
}

template <int DT, int SCORE, int V>
__global__ __launch_bounds__(kRouteWaves * 64) void route_exact_kernel(RouteParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t room[kRouteWaves][exact_room(64 * V)];
  const int wave = threadIdx.x >> 6;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRouteWaves + wave; r < p.rows;
       r += static_cast<int64_t>(gridDim.x) * kRouteWaves)
    route_row_exact<DT, SCORE, V>(params_of_launch(), r, room[wave], 0, 0);
}

// ------------------------------------------------------------------------- the fast kernel
// L lanes of a wave take a row (64 / L rows a wave) and hold up to V consecutive experts each;
// a group is the experts of p.lanes consecutive lanes. Every expert becomes one 32-bit key,
//   (quantised selection score) << IB | (L V - 1 - position),
// so larger keys are better and equal scores go to the smaller expert. A lane sorts its keys to
// its KP best with a network of unsigned maxima and minima, and lanes merge their lists
// pairwise (the elementwise maximum of one list and the reversed other is the KP best of both,
// bitonic). Groups are ranked when the merges reach p.lanes lanes.
//
// The scores are fp32 and the keys hold 32 - IB bits of them, so two keys whose scores differ
// by at most `slack` steps may be in the wrong order. A row in which two neighbours of the
// result, the last chosen and the first left out, or the last chosen group and the first left
// out are that close goes to route_row_exact: the choice is always the exact one.
// What slack covers, in steps of 2^-24 of the keys' range (at least 1, so a step is at least
// 2^-24): a sigmoid's error is at most 4 steps (the exponent's rounding 0.84, exp2, 1 + y,
// rcp), a softmax's 64 (its sum's terms and their V + log2 L additions); the bias and the
// conversion add 2. Two keys: 2 * 6 + 1 and 2 * 66 + 1. Logits themselves: the subtraction and the
// conversion, 2 * 1.5. bf16 logits are keys without loss.
enum RouteMode { kBySigmoid, kBySoftmax, kByLogit };

__device__ __forceinline__ void order2(uint32_t& a, uint32_t& b) {  // a >= b
  const uint32_t hi = a > b ? a : b, lo = a > b ? b : a;
  a = hi, b = lo;
}

// Batcher's odd-even merge sort, largest first.
template <int N>
__device__ __forceinline__ void sort_down(uint32_t* a) {
#pragma unroll
  for (int q = 1; q < N; q *= 2)
#pragma unroll
    for (int d = q; d >= 1; d /= 2)
#pragma unroll
      for (int j = d % q; j + d < N; j += 2 * d)
#pragma unroll
        for (int i = 0; i < d; ++i)
          if (i + j + d < N && (i + j) / (2 * q) == (i + j + d) / (2 * q)) order2(a[i + j], a[i + j + d]);
}

// Sorts a bitonic sequence, largest first.
template <int N>
__device__ __forceinline__ void clean_down(uint32_t* a) {
#pragma unroll
  for (int d = N / 2; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & d) == 0) order2(a[i], a[i + d]);
}

// The KP best of a sorted list and another's (given reversed: o[i] is its entry KP - 1 - i);
// `dropped` keeps the best key that was not among them.
template <int KP>
__device__ __forceinline__ void merge_down(uint32_t* list, const uint32_t* o, uint32_t& dropped) {
#pragma unroll
  for (int i = 0; i < KP; ++i) {
    const uint32_t hi = larger(list[i], o[i]);
    dropped = larger(dropped, list[i] < o[i] ? list[i] : o[i]);
    list[i] = hi;
  }
  clean_down<KP>(list);
}

template <int LEVEL, int KP>
__device__ __forceinline__ void merge_partner(uint32_t* list, uint32_t& dropped) {
  uint32_t o[KP];
#pragma unroll
  for (int i = 0; i < KP; ++i) o[i] = from_partner<LEVEL>(list[KP - 1 - i]);
  dropped = larger(dropped, from_partner<LEVEL>(dropped));
  merge_down<KP>(list, o, dropped);
}

// Waves a SIMD, and workgroups a CU: with 32 experts a lane, three waves' registers hold what
// four spill (65536 x 256 fp32, k = 8: 26.5 and 29.9 us).
template <int V, int KP>
constexpr int kRouteOccupancy = V < 32 ? 4 : KP == 16 ? 2 : 3;

template <int DT, int SCORE, int MODE, int L, int V, int KP>
__global__ __launch_bounds__(kRouteWaves * 64, (kRouteOccupancy<V, KP>)) void route_kernel(RouteParams p) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int N = E::kPer16;
  static_assert(V % N == 0, "a lane's experts are whole vectors");
  constexpr int LEVELS = __builtin_ctz(L), IB = __builtin_ctz(L * V), QB = 32 - IB;
  constexpr uint32_t kFirst = 1u << IB;  // the smallest key of an expert that can be chosen
  constexpr float kTop = static_cast<float>((1 << (QB < 24 ? QB : 24)) - 64);  // whole numbers of fp32
  constexpr bool kExactKeys = MODE == kByLogit && DT == DS_BF16;
  constexpr int kSlack = MODE == kBySigmoid ? 13 : MODE == kBySoftmax ? 133 : kExactKeys ? -1 : 4;
  constexpr bool kSteps = MODE != kByLogit;
  constexpr int kPad = V + 4;  // (lanes read their V steps by 16 bytes: no two in the same banks)
  constexpr int kLane = V * static_cast<int>(sizeof(T)) + 16;  // a lane's experts in LDS; the 16 bytes spread the banks
  constexpr int kTile = 64 * kLane, kExact = exact_room(L * V);
  // a wave's rows on their way to the lanes that take them, or route_row_exact's room
  __shared__ __attribute__((aligned(16))) uint8_t room[kRouteWaves][kTile > kExact ? kTile : kExact];
  __shared__ __attribute__((aligned(16))) float steps[kSteps ? L * kPad : 4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, sub = lane & (L - 1);
  const int group = sub >> p.lanes_log2, part = sub & ((1 << p.lanes_log2) - 1);
  const int first = group * p.run + part * p.per_lane;  // the lane's first expert
  const bool limited = p.topk_groups < p.groups;
  int have = p.run - part * p.per_lane;  // and how many it holds
  have = have > p.per_lane ? p.per_lane : have;
  if (group >= p.experts / p.run || have < 0) have = 0;
  const bool full = __ballot(have != V) == 0;
  uint32_t apart = 0;  // vectors of which a lane holds only a part (or that a row is too short for)
#pragma unroll
  for (int v = 0; v < V; v += N)
    if (p.experts < N || __any(v < have && have < v + N)) apart |= 1u << (v / N);

  // c = s + b as a key: (s + b - least b) * per_unit + 1; `steps` holds the bias' part by
  // position, and -inf (key 0) where there is no expert
  float per_unit = kTop;
  bool undecided = false;  // no key can hold the biases' range
  bool flat = false;       // the order is that of bf16 logits through a sigmoid, whatever the bias
  if constexpr (kSteps) {
    float lo = 0.0f, hi = 0.0f;
    if (p.bias) {
      lo = __builtin_huge_valf(), hi = kNegInf;
      for (int e = lane; e < p.experts; e += 64) {
        const float b = p.bias[e];
        hi = fmaxf(hi, b);
        if (b != kNegInf) lo = fminf(lo, b);
      }
      hi = wave_max(hi);
      lo = -wave_max(-lo);
    }
    flat = MODE == kBySigmoid && DT == DS_BF16 && lo == hi;
    const float range = hi - lo + 1.0f;
    // (beyond, the sums' own rounding to double would count, and at last the keys' range)
    undecided = !(fmaxf(fabsf(lo), fabsf(hi)) <= 1e6f);
    per_unit = kTop / range;
    for (int i = threadIdx.x; i < L * V; i += kRouteWaves * 64) {
      const int of = i / V, v = i % V, run_at = (of & ((1 << p.lanes_log2) - 1)) * p.per_lane + v;
      const int e = (of >> p.lanes_log2) * p.run + run_at;
      float q = kNegInf;
      if (v < p.per_lane && run_at < p.run && e < p.experts)
        q = p.bias ? fmaf(p.bias[e] - lo, per_unit, 1.0f) : 1.0f;
      steps[of * kPad + v] = q;
    }
    __syncthreads();
  }

  const T* xs = static_cast<const T*>(p.x);
  constexpr int kRows = 64 / L;
  const int64_t first_row = (static_cast<int64_t>(blockIdx.x) * kRouteWaves + wave) * kRows;
  const int64_t row_step = static_cast<int64_t>(gridDim.x) * kRouteWaves * kRows;
  // the rows of the next turn are loaded while this turn's are worked on
  typename Vec<DT, N>::type ahead[V / N];
  const auto fetch = [&](int64_t r0) {
    if (full) {  // 64 vectors in memory's order at a time
#pragma unroll
      for (int i = 0; i < V / N; ++i) {
        const int at = i * 64 + lane, of = at / (L * V / N);
        const int64_t r = r0 + of < p.rows ? r0 + of : p.rows - 1;
        ahead[i] = *reinterpret_cast<const typename Vec<DT, N>::unaligned*>(xs + r * p.row_stride +
                                                                           at % (L * V / N) * N);
      }
    } else {
      const int64_t r = r0 + lane / L < p.rows ? r0 + lane / L : p.rows - 1;
      const T* row = xs + r * p.row_stride;
      int last = have > 0 ? first + have - 1 : 0;  // slots past the lane's experts load its last one
      asm("" : "+v"(last));                        // (not kept as one address per slot)
#pragma unroll
      for (int v = 0; v < V; v += N) {
        if (apart >> (v / N) & 1) {
#pragma unroll
          for (int j = 0; j < N; ++j) ahead[v / N][j] = row[first + v + j < last ? first + v + j : last];
        } else {
          ahead[v / N] = *reinterpret_cast<const typename Vec<DT, N>::unaligned*>(row + (first + v < last ? first + v : 0));
        }
      }
    }
  };
  // Turns are taken 64 at a time; lane i keeps which rows of turn i need the exact choice.
  for (int64_t turn0 = first_row; turn0 < p.rows; turn0 += 64 * row_step) {
  fetch(turn0);
  uint64_t left = 0, left_kept = 0, left_open = 0;
  int turn = 0;
  for (int64_t r0 = turn0; turn < 64 && r0 < p.rows; r0 += row_step, ++turn) {
    const int64_t r = r0 + lane / L < p.rows ? r0 + lane / L : p.rows - 1;
    const T* row = xs + r * p.row_stride;
    float x[V];
    if (full) {  // through LDS, so that each lane has its run of experts
      typedef typename Vec<DT, N>::type VT;
      wave_sync();
#pragma unroll
      for (int i = 0; i < V / N; ++i) {
        const int at = i * 64 + lane;
        *reinterpret_cast<VT*>(room[wave] + at / (V / N) * kLane + at % (V / N) * 16) = ahead[i];
      }
      wave_sync();
#pragma unroll
      for (int i = 0; i < V / N; ++i) ahead[i] = *reinterpret_cast<const VT*>(room[wave] + lane * kLane + i * 16);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = E::widen(ahead[v / N][v % N]);
    if (!full) {
      int n = have;
      asm volatile("" : "+v"(n));  // compared in every turn, not kept as one mask per slot
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = v < n ? x[v] : kNegInf;
    }
    if (r0 + row_step < p.rows) fetch(r0 + row_step);
    // the softmax's maximum and sum
    float m = 0.0f, inv = 1.0f;
    const bool soft = SCORE == DS_SCORE_SOFTMAX;
    if (MODE != kBySigmoid) {
      m = x[0];
#pragma unroll
      for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
      m = row_reduce<LEVELS>(m, [](float a, float b) { return fmaxf(a, b); });
    }
    float e[V];
    if (MODE == kBySoftmax || (soft && !p.renorm)) {
      float z = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        e[v] = x[v] == m ? 1.0f : __builtin_amdgcn_exp2f((x[v] - m) * kLog2E);
        z += e[v];
      }
      z = row_reduce<LEVELS>(z, [](float a, float b) { return a + b; });
      inv = 1.0f / z;  // at least one term is 1
    }
    uint32_t key[V];
    const uint32_t place = static_cast<uint32_t>(L * V - 1 - sub * V);  // (its low bits are ones: place - v is place ^ v)
    float least = x[0];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      uint32_t q;
      const float step = kSteps ? steps[sub * kPad + v] : 0.0f;
      if constexpr (MODE == kBySigmoid) {
        const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x[v] * -kLog2E));
        q = static_cast<uint32_t>(fmaf(s, per_unit, step));
      } else if constexpr (MODE == kBySoftmax) {
        q = static_cast<uint32_t>(fmaf(e[v] * inv, per_unit, step));
      } else if constexpr (DT == DS_BF16) {
        const uint32_t u = __float_as_uint(x[v] + 0.0f);  // -0 as +0
        q = ((u ^ (static_cast<int32_t>(u) < 0 ? 0xFFFFFFFFu : 0x80000000u)) >> 16) + 1u;
      } else {
        q = static_cast<uint32_t>(fmaf(fmaxf(x[v] - m, -32.0f), kTop / 32.0f, kTop + 1.0f));
      }
      key[v] = (q << IB) | (place ^ static_cast<uint32_t>(v));
      least = fminf(least, x[v]);
    }
    if (__any(least == kNegInf)) {  // masked logits
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = x[v] == kNegInf ? 0u : key[v];
    }
    // a lane's KP best; the barriers keep one block's network from being mixed with the next's,
    // which takes more registers than it gains
    uint32_t list[KP], dropped = 0u;
#pragma unroll
    for (int i = 0; i < KP; ++i) list[i] = i < V ? key[i] : 0u;
    sort_down<(V < KP ? V : KP)>(list);
#pragma unroll
    for (int b = KP; b < V; b += KP) {
      __builtin_amdgcn_sched_barrier(0);
      uint32_t t[KP], o[KP];
#pragma unroll
      for (int i = 0; i < KP; ++i) t[i] = key[b + i];
      sort_down<KP>(t);
#pragma unroll
      for (int i = 0; i < KP; ++i) o[i] = t[KP - 1 - i];
      merge_down<KP>(list, o, dropped);
    }
    bool close = undecided || (MODE == kByLogit && m == __builtin_huge_valf());
    bool unsure = undecided;  // the choice of groups is close, or not to be taken from keys at all
    uint64_t kept = 0;    // lanes whose group was chosen
    const auto rank_groups = [&](auto level) {  // of the lists of 2^level lanes
      const uint32_t a = list[0] >> IB, b = list[1] >> IB;
      unsure |= p.group_top > 1 && a != 0u && b == 0u;  // a sum of one: not comparable in steps
      const uint32_t sum = p.group_top > 1 ? a + b : a;
      const uint32_t mine = (sum << 6) | static_cast<uint32_t>(63 - group);
      int rank = 0;  // (lanes without a group have the smallest keys)
#pragma unroll
      for (int o = 0; o < (L >> level()); ++o)
        rank += static_cast<uint32_t>(__shfl(static_cast<int>(mine), (lane & ~(L - 1)) + (o << level()))) > mine;
      const bool out = rank >= p.topk_groups;
      const auto least = [](uint32_t u, uint32_t w) { return u < w ? u : w; };
      const uint32_t in = row_reduce<LEVELS>(out ? 0xFFFFFFFFu : sum, least);
      const uint32_t over = row_reduce<LEVELS>(out ? sum : 0u, [](uint32_t u, uint32_t w) { return larger(u, w); });
      unsure |= over != 0u && static_cast<int>(in - over) <= (p.group_top > 1 ? 2 * kSlack : kSlack);
      close |= unsure;
      kept = __ballot(!out);
      dropped = out ? 0u : dropped;
#pragma unroll
      for (int i = 0; i < KP; ++i) list[i] = out ? 0u : list[i];
    };
#define DS_LEVEL(n)                                        \
  if constexpr (LEVELS > n) {                              \
    if (limited && p.lanes_log2 == n) rank_groups(std::integral_constant<int, n>()); \
    merge_partner<n, KP>(list, dropped);                   \
  }
    DS_LEVEL(0) DS_LEVEL(1) DS_LEVEL(2) DS_LEVEL(3) DS_LEVEL(4)
#undef DS_LEVEL
    // Neighbours of the list (the last one's is the best key left out) too close to be told
    // apart. A list may go on past k: its later neighbours only send a row to the exact choice
    // for nothing.
    if constexpr (!kExactKeys) {
      constexpr uint32_t kNear = static_cast<uint32_t>(kSlack + 1) << IB;  // a gap of at most kSlack steps is below
      uint32_t gap = list[KP - 1] - dropped;
#pragma unroll
      for (int i = 0; i + 1 < KP; ++i) gap = list[i] - list[i + 1] < gap ? list[i] - list[i + 1] : gap;
      if (__any(gap < kNear)) {  // (or there is nothing at these places)
        bool near = (list[KP - 1] - dropped < kNear) & (dropped >= kFirst);
#pragma unroll
        for (int i = 0; i + 1 < KP; ++i) near |= (list[i] - list[i + 1] < kNear) & (list[i + 1] >= kFirst);
        // Equal bf16 logits are common, and with one bias for all (zeros, before any balancing) they
        // tie. Between 2^-8 and 8 different ones give scores at least 7e-6 apart, 30 steps of the
        // coarsest keys: there only equal logits are near, and the smaller expert is right.
        if (flat) {
          const uint32_t high = static_cast<uint32_t>(fmaf(0.99966465f, per_unit, 1.0f)) << IB,
                         low = static_cast<uint32_t>(fmaf(0.50097656f, per_unit, 2.0f)) << IB;
          near &= !(list[0] < high && dropped >= low);
        }
        close |= near;
      }
    }
    close = row_reduce<LEVELS>(close ? 1u : 0u, [](uint32_t a, uint32_t b) { return a | b; }) != 0u;
    // slot j in lane j % L: the weights
    constexpr int kSlots = KP > L ? KP / L : 1;
    float s[kSlots];
    int at[kSlots];
    float total = 0.0f;
#pragma unroll
    for (int t = 0; t < kSlots; ++t) {
      uint32_t mine;
      if constexpr (KP >= L) {  // slots t L to t L + L - 1, by the bits of the lane
        uint32_t of[L];
#pragma unroll
        for (int i = 0; i < L; ++i) of[i] = list[t * L + i];
#pragma unroll
        for (int b = L / 2; b >= 1; b /= 2)
#pragma unroll
          for (int i = 0; i < b; ++i) of[i] = (sub & b) ? of[i + b] : of[i];
        mine = of[0];
      } else {
        mine = 0u;
#pragma unroll
        for (int i = 0; i < KP; ++i) mine = i == sub ? list[i] : mine;
      }
      const uint32_t pos = static_cast<uint32_t>(L * V - 1) - (mine & (kFirst - 1u));
      const int owner = static_cast<int>(pos / V);
      at[t] = mine >= kFirst && t * L + sub < p.k
                  ? (owner >> p.lanes_log2) * p.run + (owner & ((1 << p.lanes_log2) - 1)) * p.per_lane +
                        static_cast<int>(pos % V)
                  : -1;
      const float v = at[t] >= 0 ? E::widen(row[at[t]]) : kNegInf;
      if (soft) {
        s[t] = v == kNegInf ? 0.0f : v == m ? inv : __builtin_amdgcn_exp2f((v - m) * kLog2E) * inv;
      } else {
        s[t] = 1.0f / (1.0f + __builtin_amdgcn_exp2f(v * -kLog2E));
      }
      total += s[t];
    }
    total = row_reduce<LEVELS>(total, [](float a, float b) { return a + b; });
    // scores that fp32 holds with too few bits to be divided
    close |= p.renorm && list[0] >= kFirst && !(total > 1e-30f);
    const bool mine = r0 + lane / L < p.rows;
    const float factor = p.renorm ? (total > 0.0f ? p.scale / total : 0.0f) : p.scale;
#pragma unroll
    for (int t = 0; t < kSlots; ++t) {
      const int j = t * L + sub;
      if (mine && !close && j < p.k) {
        if (p.out_weights) p.out_weights[r * p.k + j] = s[t] * factor;
        if (p.out_idx) p.out_idx[r * p.k + j] = at[t];
      }
    }
    const uint64_t rest = __ballot(mine && close && sub == 0), open = __ballot(unsure);
    if (lane == turn) left = rest, left_kept = kept, left_open = open;
  }
  if (__any(left != 0)) {
    for (int t = 0; t < turn; ++t) {
      uint64_t rest = __shfl(left, t);
      const uint64_t kept = __shfl(left_kept, t), open = __shfl(left_open, t);
      while (rest) {
        const int l = __builtin_ctzll(rest);
        rest &= rest - 1;
        constexpr uint64_t kLanes = (uint64_t{1} << L) - 1;
        const bool known = (open >> l & kLanes) == 0;
        route_row_exact<DT, SCORE, L * V / 64>(params_of_launch(), turn0 + t * row_step + l / L, room[wave],
                                               known ? kept >> l & kLanes : 0, p.lanes_log2);
      }
    }
  }
  }
}

// The experts' loads, from the chosen indices: few workgroups count in LDS and add once an expert
// each. (Adding from the routing itself, 524288 atomics on 256 counters, took 320 us: an
// address takes one add every 0.17 us or so from the card's several L2 caches.)
constexpr int kCountThreads = 1024, kCountGroups = 32;

__global__ __launch_bounds__(kCountThreads) void route_counts_kernel(const int32_t* idx, int64_t n, int32_t* counts,
                                                                     int32_t experts) {
  __shared__ int32_t of_expert[DS_MAX_EXPERTS];
  for (int e = threadIdx.x; e < experts; e += kCountThreads) of_expert[e] = 0;
  __syncthreads();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kCountThreads;
#pragma unroll 4
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCountThreads + threadIdx.x; i < n; i += step) {
    const int32_t e = idx[i];
    if (e >= 0) atomicAdd(&of_expert[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < experts; e += kCountThreads)
    if (of_expert[e]) atomicAdd(counts + e, of_expert[e]);
}

// ------------------------------------------------------------------------------ the gradient
// A wave keeps a tile of rows in LDS, all zero between turns: slots are added at their
// experts, lanes read the tile in memory's order and the slots clear what they added. Indices
// are checked before they are used as places.
constexpr int kGradTile = 1024;  // floats of a wave's tile (twice as many: 17.0 -> 17.6 us for 65536 x 256 fp32)

// The chosen experts' gradients only (all others are zero): KL lanes a row, slot j in lane
// j % KL; x is read at the chosen experts.
//   slot j adds c_j = ds_j * ds/dx at its expert, with f_j = scale * g_j and, renormalised,
//   ds_j = (f_j - sum f s / S) / S. The softmax renormalised is a softmax over the chosen
//   experts alone: it needs no other logits, s is exp(x - the chosen ones' maximum).
template <int DT, int SCORE, int KL>
__global__ __launch_bounds__(kRouteWaves * 64) void route_grad_chosen_kernel(RouteGradParams p) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int N = E::kPer16, LEVELS = __builtin_ctz(KL);
  __shared__ __attribute__((aligned(16))) float tiles[kRouteWaves][kGradTile];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, slot = lane % KL;
  float* const tile = tiles[wave];
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out);
  const int per_row = (p.experts + N - 1) / N, pitch = per_row * N;  // vectors of a row; floats of its tile
  int rows = kGradTile / pitch;
  rows = rows > 64 / KL ? 64 / KL : rows;
  const float inv_per_row = 1.0f / static_cast<float>(per_row);
#pragma unroll
  for (int i = 0; i < kGradTile; i += 256) *reinterpret_cast<float4*>(tile + i + lane * 4) = make_float4(0, 0, 0, 0);
  wave_sync();
  for (int64_t r0 = (static_cast<int64_t>(blockIdx.x) * kRouteWaves + wave) * rows; r0 < p.rows;
       r0 += static_cast<int64_t>(gridDim.x) * kRouteWaves * rows) {
    const int here = p.rows - r0 < rows ? static_cast<int>(p.rows - r0) : rows;
    const int row = lane / KL;
    const bool live = row < here && slot < p.k;
    int e = -1;
    float f = 0.0f, v = kNegInf;
    if (live) {
      const int64_t at = (r0 + row) * p.k + slot;
      e = p.idx[at];
      f = p.grad[at] * p.scale;
      if (e < 0 || e >= p.experts) e = -1;
      if (e >= 0) v = E::widen(x[(r0 + row) * p.row_stride + e]);
    }
    f = e >= 0 ? f : 0.0f;
    float s, slope;
    bool none = false;  // no chosen expert has a score in double: there are no weights either
    if constexpr (SCORE == DS_SCORE_SOFTMAX) {
      const float m = row_reduce<LEVELS>(v, [](float a, float b) { return larger(a, b); });
      s = v == kNegInf ? 0.0f : v == m ? 1.0f : __builtin_amdgcn_exp2f((v - m) * kLog2E);
      slope = s;
    } else {
      // scores far below 1 in units of the largest, which divides out of s / S: with
      // u = exp(-|x|), s = exp(min(x, 0)) / (1 + u) and 1 - s = exp(min(-x, 0)) / (1 + u)
      float unit = 0.0f;
      if (p.renorm) {
        unit = row_reduce<LEVELS>(v, [](float a, float b) { return larger(a, b); });
        none = unit < -745.1332f;
        unit = unit < 0.0f && unit > kNegInf ? unit : 0.0f;
      }
      const float part = 1.0f / (1.0f + __builtin_amdgcn_exp2f(fabsf(v) * -kLog2E));
      s = part * __builtin_amdgcn_exp2f((fminf(v, 0.0f) - unit) * kLog2E);
      slope = s * part * __builtin_amdgcn_exp2f(fminf(-v, 0.0f) * kLog2E);
    }
    float d = f;
    if (p.renorm) {
      const float S = row_reduce<LEVELS>(s, plus<float>), fs = row_reduce<LEVELS>(f * s, plus<float>);
      d = S > 0.0f && !none ? (f - fs / S) / S : 0.0f;
    }
    const int place = e >= 0 ? row * pitch + e : -1;
    if (place >= 0) atomicAdd(tile + place, d * slope);
    wave_sync();
    for (int i = lane; i < here * per_row; i += 64) {
      const int of = static_cast<int>((static_cast<float>(i) + 0.5f) * inv_per_row), at = (i - of * per_row) * N;
      const float* from = tile + of * pitch + at;
      T* to = out + (r0 + of) * p.out_stride + at;
      if (at + N <= p.experts) {
        typename Vec<DT, N>::type q;
#pragma unroll
        for (int j = 0; j < N; ++j) q[j] = E::narrow(from[j]);
        // (past the caches: 19.2 -> 17.4 us for 65536 x 256 fp32, 25.6 -> 17.9 from a graph)
        __builtin_nontemporal_store(q, reinterpret_cast<typename Vec<DT, N>::unaligned*>(to));
      } else {
        for (int j = 0; at + j < p.experts; ++j) to[j] = E::narrow(from[j]);
      }
    }
    wave_sync();
    if (place >= 0) tile[place] = 0.0f;
    wave_sync();
  }
}

// The softmax without renormalisation has a gradient at every expert: one wave per row, V
// vectors of N consecutive experts a lane.
template <int DT, int V>
__global__ __launch_bounds__(kRouteWaves * 64) void route_grad_softmax_kernel(RouteGradParams p) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int N = E::kPer16;
  typedef typename Vec<DT, N>::type VT;
  __shared__ __attribute__((aligned(16))) float tiles[kRouteWaves][V * 64 * N];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  float* const tile = tiles[wave];
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out);
#pragma unroll
  for (int i = 0; i < V * 64 * N; i += 256)
    *reinterpret_cast<float4*>(tile + i + lane * 4) = make_float4(0, 0, 0, 0);
  wave_sync();
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRouteWaves + wave; r < p.rows;
       r += static_cast<int64_t>(gridDim.x) * kRouteWaves) {
    int e = -1;
    float f = 0.0f;
    if (lane < p.k) {
      e = p.idx[r * p.k + lane];
      f = p.grad[r * p.k + lane] * p.scale;
      if (e < 0 || e >= p.experts) e = -1;
    }
    const T* row = x + r * p.row_stride;
    float s[V][N], m = kNegInf, z = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int at = (v * 64 + lane) * N;
      if (at + N <= p.experts) {
        const VT q = *reinterpret_cast<const typename Vec<DT, N>::unaligned*>(row + at);
#pragma unroll
        for (int j = 0; j < N; ++j) s[v][j] = E::widen(q[j]);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) s[v][j] = at + j < p.experts ? E::widen(row[at + j]) : kNegInf;
      }
#pragma unroll
      for (int j = 0; j < N; ++j) m = fmaxf(m, s[v][j]);
    }
    if (e >= 0) atomicAdd(tile + e, f);
    m = wave_max(m);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        s[v][j] = s[v][j] == kNegInf ? 0.0f : s[v][j] == m ? 1.0f : __builtin_amdgcn_exp2f((s[v][j] - m) * kLog2E);
        z += s[v][j];
      }
    z = wave_sum(z);
    wave_sync();
    const float inv = z > 0.0f ? 1.0f / z : 0.0f;
    float h[V][N], dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        h[v][j] = tile[(v * 64 + lane) * N + j];
        s[v][j] *= inv;
        dot += h[v][j] * s[v][j];
      }
    dot = wave_sum(dot);
    wave_sync();
    if (e >= 0) tile[e] = 0.0f;
    T* to = out + r * p.out_stride;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int at = (v * 64 + lane) * N;
      VT q;
#pragma unroll
      for (int j = 0; j < N; ++j) q[j] = E::narrow(s[v][j] * (h[v][j] - dot));
      if (at + N <= p.experts) {
        *reinterpret_cast<typename Vec<DT, N>::unaligned*>(to + at) = q;
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (at + j < p.experts) to[at + j] = q[j];
      }
    }
    wave_sync();
  }
}

uint32_t route_grid(int64_t rows, int64_t rows_per_group, int64_t per_cu) {
  const int64_t need = (rows + rows_per_group - 1) / rows_per_group, most = kCus * per_cu;
  return static_cast<uint32_t>(need < most ? need : most);
}

template <int DT, int SCORE, int MODE, int L, int V>
hipError_t route_shape(const RouteParams& p, hipStream_t s) {
  const auto go = [&](auto kern, int per_cu) {
    const dim3 g(route_grid(p.rows, kRouteWaves * (64 / L), per_cu)), b(kRouteWaves * 64);
    hipLaunchKernelGGL(kern, g, b, 0, s, p);
    return hipGetLastError();
  };
  if (p.k <= 8) return go(route_kernel<DT, SCORE, MODE, L, V, 8>, kRouteOccupancy<V, 8>);
  return go(route_kernel<DT, SCORE, MODE, L, V, 16>, kRouteOccupancy<V, 16>);
}

template <int DT, int SCORE, int MODE>
hipError_t route_mode(RouteParams p, hipStream_t s) {
  // the fewest lanes a row (more rows a wave) whose lists hold at most 32 experts each
  const bool limited = p.topk_groups < p.groups;
  const int groups = limited ? p.groups : 1;
  p.run = p.experts / groups;
  int need = 1;
  while (need < groups) need *= 2;
  // (a k that no list holds is left to the exact kernel; and scales past 1e8: the weights are
  // s * (scale / total) with totals down to 1e-30, and the quotient would leave fp32)
  const bool fast = p.k <= 16 && !(p.renorm && std::fabs(p.scale) > 1e8f);
  for (int lanes = 8; lanes <= 32 && fast; lanes *= 2) {
    if (lanes < need) continue;
    const int of_group = lanes / need;
    p.per_lane = (p.run + of_group - 1) / of_group;
    p.lanes_log2 = __builtin_ctz(of_group);
    if (p.per_lane > 32) continue;
    if (lanes == 8) {
      if (p.per_lane <= 8) return route_shape<DT, SCORE, MODE, 8, 8>(p, s);
      if (p.per_lane <= 16) return route_shape<DT, SCORE, MODE, 8, 16>(p, s);
      return route_shape<DT, SCORE, MODE, 8, 32>(p, s);
    }
    if (lanes == 16) {
      if (p.per_lane <= 16) return route_shape<DT, SCORE, MODE, 16, 16>(p, s);
      return route_shape<DT, SCORE, MODE, 16, 32>(p, s);
    }
    return route_shape<DT, SCORE, MODE, 32, 32>(p, s);
  }
  const dim3 g(route_grid(p.rows, kRouteWaves, 4)), b(kRouteWaves * 64);
  if (p.experts <= 256) hipLaunchKernelGGL((route_exact_kernel<DT, SCORE, 4>), g, b, 0, s, p);
  else hipLaunchKernelGGL((route_exact_kernel<DT, SCORE, DS_MAX_EXPERTS / 64>), g, b, 0, s, p);
  return hipGetLastError();
}

template <int DT>
hipError_t route_dt(int score, const RouteParams& p, hipStream_t s) {
  const bool by_score = p.bias || (p.topk_groups < p.groups && p.group_top > 1);
  if (score == DS_SCORE_SOFTMAX)
    return by_score ? route_mode<DT, DS_SCORE_SOFTMAX, kBySoftmax>(p, s) : route_mode<DT, DS_SCORE_SOFTMAX, kByLogit>(p, s);
  return by_score ? route_mode<DT, DS_SCORE_SIGMOID, kBySigmoid>(p, s) : route_mode<DT, DS_SCORE_SIGMOID, kByLogit>(p, s);
}

template <int DT, int SCORE>
hipError_t grad_chosen(const RouteGradParams& p, hipStream_t s) {
  const int pitch = (p.experts + Elem<DT>::kPer16 - 1) / Elem<DT>::kPer16 * Elem<DT>::kPer16;
  const int fit = kGradTile / pitch;
  const auto go = [&](auto kern, int kl) {
    const int rows = fit < 64 / kl ? fit : 64 / kl;
    hipLaunchKernelGGL(kern, dim3(route_grid(p.rows, kRouteWaves * rows, 16)), dim3(kRouteWaves * 64), 0, s, p);
    return hipGetLastError();
  };
  if (p.k <= 2) return go(route_grad_chosen_kernel<DT, SCORE, 2>, 2);
  if (p.k <= 4) return go(route_grad_chosen_kernel<DT, SCORE, 4>, 4);
  if (p.k <= 8) return go(route_grad_chosen_kernel<DT, SCORE, 8>, 8);
  if (p.k <= 16) return go(route_grad_chosen_kernel<DT, SCORE, 16>, 16);
  return go(route_grad_chosen_kernel<DT, SCORE, 64>, 64);
}

template <int DT>
hipError_t grad_softmax(const RouteGradParams& p, hipStream_t s) {
  constexpr int kOne = 64 * Elem<DT>::kPer16;  // experts of one vector a lane
  const dim3 g(route_grid(p.rows, kRouteWaves, 16)), b(kRouteWaves * 64);
  if (p.experts <= kOne) hipLaunchKernelGGL((route_grad_softmax_kernel<DT, 1>), g, b, 0, s, p);
  else if (p.experts <= 2 * kOne) hipLaunchKernelGGL((route_grad_softmax_kernel<DT, 2>), g, b, 0, s, p);
  else hipLaunchKernelGGL((route_grad_softmax_kernel<DT, DS_MAX_EXPERTS / kOne>), g, b, 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(int dtype, int score, const RouteParams& p, hipStream_t s) {
  const hipError_t e = dtype == DS_BF16 ? route_dt<DS_BF16>(score, p, s) : route_dt<DS_FP32>(score, p, s);
  if (e != hipSuccess || !p.counts) return e;
  const int64_t n = p.rows * p.k, need = (n + 4 * kCountThreads - 1) / (4 * kCountThreads);
  hipLaunchKernelGGL(route_counts_kernel, dim3(static_cast<uint32_t>(need < kCountGroups ? need : kCountGroups)),
                     dim3(kCountThreads), 0, s, p.out_idx, n, p.counts, p.experts);
  return hipGetLastError();
}

hipError_t launch_route_grad(int dtype, int score, const RouteGradParams& p, hipStream_t s) {
  if (score == DS_SCORE_SOFTMAX && !p.renorm) return dtype == DS_BF16 ? grad_softmax<DS_BF16>(p, s) : grad_softmax<DS_FP32>(p, s);
  if (score == DS_SCORE_SOFTMAX)
    return dtype == DS_BF16 ? grad_chosen<DS_BF16, DS_SCORE_SOFTMAX>(p, s) : grad_chosen<DS_FP32, DS_SCORE_SOFTMAX>(p, s);
  return dtype == DS_BF16 ? grad_chosen<DS_BF16, DS_SCORE_SIGMOID>(p, s) : grad_chosen<DS_FP32, DS_SCORE_SIGMOID>(p, s);
}

}  // namespace ds
