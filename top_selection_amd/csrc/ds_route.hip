// Routing to experts and its gradient.
#include "ds_rows_device.h"

namespace ds {
namespace {

constexpr int kRouteWaves = 4;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr double kNone = -__builtin_huge_val();  // the selection score of a masked or taken expert
constexpr float kLog2E = 1.44269504088896341f;

// ------------------------------------------------------------------ the exact choice of a row
// A whole wave chooses for one row with everything that decides in double; c: LDS room of
// p.experts doubles that is the wave's own. Rows that the fast kernel cannot decide come here,
// and every row where no fast kernel fits.
template <int DT, int SCORE>
__device__ __forceinline__ void route_row_exact(const RouteParams& p, int64_t r, double* c) {
  using E = Elem<DT>;
  const int lane = threadIdx.x & 63;
  const typename E::T* x = static_cast<const typename E::T*>(p.x) + r * p.row_stride;
  float m = kNegInf;
  double inv = 1.0;
  if constexpr (SCORE == DS_SCORE_SOFTMAX) {
    for (int e = lane; e < p.experts; e += 64) m = fmaxf(m, E::widen(x[e]));
    m = wave_max(m);
  }
  const auto term = [&](float v) {  // the score, the softmax's without its division
    if constexpr (SCORE == DS_SCORE_SOFTMAX)
      return v == kNegInf ? 0.0 : v == m ? 1.0 : exp(static_cast<double>(v) - static_cast<double>(m));
    else
      return 1.0 / (1.0 + exp(-static_cast<double>(v)));
  };
  if constexpr (SCORE == DS_SCORE_SOFTMAX) {
    double z = 0.0;
    for (int e = lane; e < p.experts; e += 64) z += term(E::widen(x[e]));
    z = wave_sum(z);
    inv = z > 0.0 ? 1.0 / z : 0.0;
  }
  const bool limited = p.topk_groups < p.groups;
  // without a bias the order is that of the logits; sums of scores for the groups are not
  const bool sums = limited && !p.bias && p.group_top > 1;
  const auto choice = [&](int e, bool score) {
    const float v = E::widen(x[e]);
    if (v == kNegInf) return kNone;
    if (p.bias) return term(v) * inv + static_cast<double>(p.bias[e]);
    return score ? term(v) * inv : static_cast<double>(v);
  };
  for (int e = lane; e < p.experts; e += 64) c[e] = choice(e, sums);
  __builtin_amdgcn_wave_barrier();
  if (limited) {
    double top = kNone, second = kNone;
    if (lane < p.groups)
      for (int j = 0; j < p.group_size; ++j) {
        const double q = c[lane * p.group_size + j];
        second = q > top ? top : (q > second ? q : second);
        top = q > top ? q : top;
      }
    const double score = p.group_top > 1 && second != kNone ? top + second : top;
    int rank = 0;
    for (int o = 0; o < p.groups; ++o) {
      const double other = __shfl(score, o);
      rank += other > score || (other == score && o < lane);
    }
    const uint64_t keep = __ballot(lane < p.groups && rank < p.topk_groups);
    __builtin_amdgcn_wave_barrier();
    for (int e = lane; e < p.experts; e += 64) {
      if (!((keep >> (e / p.group_size)) & 1)) c[e] = kNone;
      else if (sums) c[e] = choice(e, false);
    }
    __builtin_amdgcn_wave_barrier();
  }
  int my_e = -1;
  for (int j = 0; j < p.k; ++j) {
    double best = kNone;
    int at = 0x7FFFFFFF;
    for (int e = lane; e < p.experts; e += 64)
      if (c[e] > best) best = c[e], at = e;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const double ob = __shfl_xor(best, o);
      const int oa = __shfl_xor(at, o);
      if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
    }
    if (at == 0x7FFFFFFF) break;  // nothing left
    if ((at & 63) == lane) c[at] = kNone;
    if (lane == j) my_e = at;
  }
  const double s = my_e >= 0 ? term(E::widen(x[my_e])) * inv : 0.0;
  const double total = wave_sum(s);
  if (lane < p.k) {
    const double w = !p.renorm ? s : total > 0.0 ? s / total : 0.0;
    if (p.out_weights) p.out_weights[r * p.k + lane] = static_cast<float>(w * static_cast<double>(p.scale));
    if (p.out_idx) p.out_idx[r * p.k + lane] = my_e;
    if (p.counts && my_e >= 0) atomicAdd(p.counts + my_e, 1);
  }
  __builtin_amdgcn_wave_barrier();
}

template <int DT, int SCORE>
__global__ __launch_bounds__(kRouteWaves * 64) void route_exact_kernel(RouteParams p) {
  __shared__ double c[kRouteWaves][DS_MAX_EXPERTS];
  const int wave = threadIdx.x >> 6;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRouteWaves + wave; r < p.rows;
       r += static_cast<int64_t>(gridDim.x) * kRouteWaves)
    route_row_exact<DT, SCORE>(p, r, c[wave]);
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

template <int LEVEL>
__device__ __forceinline__ uint32_t from_partner(uint32_t v) {
  // a lane of the other half of 2^(LEVEL + 1) lanes, whose values within a half are equal
  if constexpr (LEVEL == 0) return __builtin_amdgcn_update_dpp(0u, v, 0xB1, 0xF, 0xF, false);   // xor 1
  if constexpr (LEVEL == 1) return __builtin_amdgcn_update_dpp(0u, v, 0x4E, 0xF, 0xF, false);   // xor 2
  if constexpr (LEVEL == 2) return __builtin_amdgcn_update_dpp(0u, v, 0x141, 0xF, 0xF, false);  // 8 lanes reversed
  if constexpr (LEVEL == 3) return __builtin_amdgcn_update_dpp(0u, v, 0x140, 0xF, 0xF, false);  // 16 lanes reversed
  if constexpr (LEVEL == 4) {
    const auto q = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (threadIdx.x & 16u) ? q[0] : q[1];
  }
}
template <int LEVEL>
__device__ __forceinline__ float from_partner(float v) {
  return __uint_as_float(from_partner<LEVEL>(__float_as_uint(v)));
}

template <int LEVELS, class T, class F>
__device__ __forceinline__ T row_reduce(T v, F f) {
  if constexpr (LEVELS > 0) v = f(v, from_partner<0>(v));
  if constexpr (LEVELS > 1) v = f(v, from_partner<1>(v));
  if constexpr (LEVELS > 2) v = f(v, from_partner<2>(v));
  if constexpr (LEVELS > 3) v = f(v, from_partner<3>(v));
  if constexpr (LEVELS > 4) v = f(v, from_partner<4>(v));
  return v;
}

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

template <int LEVEL, int KP>
__device__ __forceinline__ void merge_partner(uint32_t* list) {
  uint32_t t[KP];
#pragma unroll
  for (int i = 0; i < KP; ++i) {
    const uint32_t o = from_partner<LEVEL>(list[KP - 1 - i]);
    t[i] = list[i] > o ? list[i] : o;
  }
#pragma unroll
  for (int i = 0; i < KP; ++i) list[i] = t[i];
  clean_down<KP>(list);
}

template <int DT, int SCORE, int MODE, int L, int V, int KP>
__global__ __launch_bounds__(kRouteWaves * 64) void route_kernel(RouteParams p) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int N = E::kPer16 < V ? E::kPer16 : V;
  constexpr int LEVELS = __builtin_ctz(L), IB = __builtin_ctz(L * V), QB = 32 - IB;
  constexpr uint32_t kFirst = 1u << IB;  // the smallest key of an expert that can be chosen
  constexpr float kTop = static_cast<float>((1 << (QB < 24 ? QB : 24)) - 64);  // whole numbers of fp32
  constexpr bool kExactKeys = MODE == kByLogit && DT == DS_BF16;
  constexpr int kSlack = MODE == kBySigmoid ? 13 : MODE == kBySoftmax ? 133 : kExactKeys ? -1 : 4;
  __shared__ double room[kRouteWaves][L * V];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, sub = lane & (L - 1);
  const int group = sub >> p.lanes_log2, part = sub & ((1 << p.lanes_log2) - 1);
  const int first = group * p.run + part * p.per_lane;  // the lane's first expert
  const bool limited = p.topk_groups < p.groups;
  int have = p.run - part * p.per_lane;  // and how many it holds
  have = have > p.per_lane ? p.per_lane : have;
  if (group >= p.experts / p.run || have < 0) have = 0;
  const bool full = __ballot(have != V) == 0;

  // c = s + b as a key: (s + b - least b) * per_unit, plus one
  float step[V];
  float per_unit = kTop;
  bool undecided = false;  // no key can hold the biases' range
  if constexpr (MODE != kByLogit) {
    float lo = __builtin_huge_valf(), hi = kNegInf;
    if (p.bias) {
      for (int e = lane; e < p.experts; e += 64) {
        const float b = p.bias[e];
        hi = fmaxf(hi, b);
        if (b != kNegInf) lo = fminf(lo, b);
      }
      hi = wave_max(hi);
      lo = -wave_max(-lo);
    } else {
      lo = hi = 0.0f;
    }
    const float range = hi - lo + 1.0f;
    undecided = !(range < 1e30f);
    per_unit = kTop / range;
#pragma unroll
    for (int v = 0; v < V; ++v)
      step[v] = p.bias && v < have ? fmaf(p.bias[first + v] - lo, per_unit, 1.0f) : 1.0f;
  }

  const T* xs = static_cast<const T*>(p.x);
  constexpr int kRows = 64 / L;
  for (int64_t r0 = (static_cast<int64_t>(blockIdx.x) * kRouteWaves + wave) * kRows; r0 < p.rows;
       r0 += static_cast<int64_t>(gridDim.x) * kRouteWaves * kRows) {
    const int64_t r = r0 + lane / L < p.rows ? r0 + lane / L : p.rows - 1;
    const T* row = xs + r * p.row_stride;
    float x[V];
    if (full) {
#pragma unroll
      for (int v = 0; v < V; v += N) {
        const typename Vec<DT, N>::type q = *reinterpret_cast<const typename Vec<DT, N>::unaligned*>(row + first + v);
#pragma unroll
        for (int j = 0; j < N; ++j) x[v + j] = E::widen(q[j]);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = v < have ? E::widen(row[first + v]) : kNegInf;
    }
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
#pragma unroll
    for (int v = 0; v < V; ++v) {
      uint32_t q;
      if constexpr (MODE == kBySigmoid) {
        const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x[v] * -kLog2E));
        q = static_cast<uint32_t>(fmaf(s, per_unit, step[v]));
      } else if constexpr (MODE == kBySoftmax) {
        q = static_cast<uint32_t>(fmaf(e[v] * inv, per_unit, step[v]));
      } else if constexpr (DT == DS_BF16) {
        const uint32_t u = __float_as_uint(x[v] + 0.0f);  // -0 as +0
        q = ((u ^ (static_cast<int32_t>(u) < 0 ? 0xFFFFFFFFu : 0x80000000u)) >> 16) + 1u;
      } else {
        q = static_cast<uint32_t>(fmaf(fmaxf(x[v] - m, -32.0f), kTop / 32.0f, kTop + 1.0f));
      }
      q = x[v] == kNegInf ? 0u : q;
      key[v] = (q << IB) | static_cast<uint32_t>(L * V - 1 - (sub * V + v));
    }
    // a lane's KP best
    uint32_t list[KP];
#pragma unroll
    for (int i = 0; i < KP; ++i) list[i] = i < V ? key[i] : 0u;
    sort_down<(V < KP ? V : KP)>(list);
#pragma unroll
    for (int b = KP; b < V; b += KP) {
      uint32_t t[KP];
#pragma unroll
      for (int i = 0; i < KP; ++i) t[i] = key[b + i];
      sort_down<KP>(t);
#pragma unroll
      for (int i = 0; i < KP; ++i) list[i] = list[i] > t[KP - 1 - i] ? list[i] : t[KP - 1 - i];
      clean_down<KP>(list);
    }
    bool close = undecided || (MODE == kByLogit && m == __builtin_huge_valf());
    bool out = false;  // the lane's group is left out
    const auto rank_groups = [&] {
      const uint32_t a = list[0] >> IB, b = list[1] >> IB;
      close |= p.group_top > 1 && a != 0u && b == 0u;  // a sum of one: not comparable in steps
      const uint32_t sum = p.group_top > 1 ? a + b : a;
      const uint32_t mine = (sum << 6) | static_cast<uint32_t>(63 - group);
      int rank = 0;
      for (int o = 0; o < p.groups; ++o)
        rank += static_cast<uint32_t>(__shfl(static_cast<int>(mine), (lane & ~(L - 1)) + (o << p.lanes_log2))) > mine;
      out = rank >= p.topk_groups;
      const auto least = [](uint32_t u, uint32_t w) { return u < w ? u : w; };
      const auto most = [](uint32_t u, uint32_t w) { return u > w ? u : w; };
      const uint32_t in = row_reduce<LEVELS>(out ? 0xFFFFFFFFu : sum, least);
      const uint32_t over = row_reduce<LEVELS>(out ? sum : 0u, most);
      close |= over != 0u && static_cast<int>(in - over) <= (p.group_top > 1 ? 2 * kSlack : kSlack);
      if (out) {
#pragma unroll
        for (int i = 0; i < KP; ++i) list[i] = 0u;
      }
    };
#define DS_LEVEL(n)                                        \
  if constexpr (LEVELS > n) {                              \
    if (limited && p.lanes_log2 == n) rank_groups();       \
    merge_partner<n, KP>(list);                            \
  }
    DS_LEVEL(0) DS_LEVEL(1) DS_LEVEL(2) DS_LEVEL(3) DS_LEVEL(4)
#undef DS_LEVEL
    // the first expert left out
    uint32_t last = 0u;
#pragma unroll
    for (int i = 0; i < KP; ++i) last = i == p.k - 1 ? list[i] : last;
    uint32_t next = 0u;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t q = key[v] < last ? key[v] : 0u;
      next = next > q ? next : q;
    }
    next = row_reduce<LEVELS>(out ? 0u : next, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
    close |= next >= kFirst && static_cast<int>((last >> IB) - (next >> IB)) <= kSlack;
#pragma unroll
    for (int i = 0; i + 1 < KP; ++i)
      close |= i + 1 < p.k && list[i + 1] >= kFirst &&
               static_cast<int>((list[i] >> IB) - (list[i + 1] >> IB)) <= kSlack;
    close = row_reduce<LEVELS>(close ? 1u : 0u, [](uint32_t a, uint32_t b) { return a | b; }) != 0u;
    // slot j in lane j % L: the weights
    constexpr int kSlots = KP > L ? KP / L : 1;
    float s[kSlots];
    int at[kSlots];
    float total = 0.0f;
#pragma unroll
    for (int t = 0; t < kSlots; ++t) {
      uint32_t mine = 0u;
#pragma unroll
      for (int i = t * L; i < KP && i < (t + 1) * L; ++i) mine = i == t * L + sub ? list[i] : mine;
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
        if (p.counts && at[t] >= 0) atomicAdd(p.counts + at[t], 1);
      }
    }
    uint64_t rest = __ballot(mine && close && sub == 0);
    while (rest) {
      const int l = __builtin_ctzll(rest);
      rest &= rest - 1;
      route_row_exact<DT, SCORE>(p, r0 + l / L, room[wave]);
    }
  }
}

// One wave per row, expert e in lane e % 64; each slot is given to its expert by comparing
// indices, so no index is ever used as an address.
template <int DT, int SCORE, int V>
__global__ __launch_bounds__(kRouteWaves * 64) void route_grad_kernel(RouteGradParams p) {
  using E = Elem<DT>;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const typename E::T* x = static_cast<const typename E::T*>(p.x);
  typename E::T* out = static_cast<typename E::T*>(p.out);
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRouteWaves + wave; r < p.rows;
       r += static_cast<int64_t>(gridDim.x) * kRouteWaves) {
    float xv[V], s[V], h[V], hits[V];
    float m = -__builtin_huge_valf();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 64 + lane;
      xv[v] = e < p.experts ? E::widen(x[r * p.row_stride + e]) : -__builtin_huge_valf();
      m = fmaxf(m, xv[v]);
      h[v] = hits[v] = 0.0f;
    }
    if constexpr (SCORE == DS_SCORE_SOFTMAX) {
      m = wave_max(m);
      float z = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[v] = xv[v] == -__builtin_huge_valf() ? 0.0f : xv[v] == m ? 1.0f : expf(xv[v] - m);
        z += s[v];
      }
      z = wave_sum(z);
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = z > 0.0f ? s[v] / z : 0.0f;
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = 1.0f / (1.0f + expf(-xv[v]));
    }
    for (int j = 0; j < p.k; ++j) {
      const int e = p.idx[r * p.k + j];
      const float g = p.grad[r * p.k + j] * p.scale;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (e == v * 64 + lane) h[v] += g, hits[v] += 1.0f;
    }
    if (p.renorm) {
      float S = 0.0f, hs = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) S += hits[v] * s[v], hs += h[v] * s[v];
      S = wave_sum(S), hs = wave_sum(hs);
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = S > 0.0f ? (h[v] - hits[v] * (hs / S)) / S : 0.0f;
    }
    float dot = 0.0f;  // with renormalised weights sum ds s is zero
    if (SCORE == DS_SCORE_SOFTMAX && !p.renorm) {
#pragma unroll
      for (int v = 0; v < V; ++v) dot += h[v] * s[v];
      dot = wave_sum(dot);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 64 + lane;
      const float d = SCORE == DS_SCORE_SOFTMAX ? s[v] * (h[v] - dot) : h[v] * s[v] * (1.0f - s[v]);
      if (e < p.experts) out[r * p.out_stride + e] = E::narrow(d);
    }
  }
}

uint32_t route_grid(int64_t rows, int64_t rows_per_group) {
  const int64_t need = (rows + rows_per_group - 1) / rows_per_group, most = kCus * 8;
  return static_cast<uint32_t>(need < most ? need : most);
}

template <int DT, int SCORE, int MODE, int L, int V>
hipError_t route_shape(const RouteParams& p, hipStream_t s) {
  const dim3 g(route_grid(p.rows, kRouteWaves * (64 / L))), b(kRouteWaves * 64);
  if (p.k <= 8) hipLaunchKernelGGL((route_kernel<DT, SCORE, MODE, L, V, 8>), g, b, 0, s, p);
  else hipLaunchKernelGGL((route_kernel<DT, SCORE, MODE, L, V, 16>), g, b, 0, s, p);
  return hipGetLastError();
}

template <int DT, int SCORE, int MODE>
hipError_t route_mode(RouteParams p, hipStream_t s) {
  // the fewest lanes a row (more rows a wave) whose lists hold at most 32 experts each
  const bool limited = p.topk_groups < p.groups;
  const int groups = limited ? p.groups : 1;
  p.run = p.experts / groups;
  int need = 1;
  while (need < groups) need *= 2;
  for (int lanes = 8; lanes <= 32 && p.k <= 16; lanes *= 2) {
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
  hipLaunchKernelGGL((route_exact_kernel<DT, SCORE>), dim3(route_grid(p.rows, kRouteWaves)), dim3(kRouteWaves * 64), 0, s, p);
  return hipGetLastError();
}

template <int DT>
hipError_t route_dt(int score, const RouteParams& p, hipStream_t s) {
  const bool by_score = p.bias || (p.topk_groups < p.groups && p.group_top > 1);
  if (score == DS_SCORE_SOFTMAX)
    return by_score ? route_mode<DT, DS_SCORE_SOFTMAX, kBySoftmax>(p, s) : route_mode<DT, DS_SCORE_SOFTMAX, kByLogit>(p, s);
  return by_score ? route_mode<DT, DS_SCORE_SIGMOID, kBySigmoid>(p, s) : route_mode<DT, DS_SCORE_SIGMOID, kByLogit>(p, s);
}

#define DS_ROUTE_V(KERN, DT, SCORE)                                                                              \
  do {                                                                                                           \
    const dim3 g(route_grid(p.rows, kRouteWaves)), b(kRouteWaves * 64);                                          \
    if (p.experts <= 64) hipLaunchKernelGGL((KERN<DT, SCORE, 1>), g, b, 0, s, p);                                \
    else if (p.experts <= 128) hipLaunchKernelGGL((KERN<DT, SCORE, 2>), g, b, 0, s, p);                          \
    else if (p.experts <= 256) hipLaunchKernelGGL((KERN<DT, SCORE, 4>), g, b, 0, s, p);                          \
    else if (p.experts <= 512) hipLaunchKernelGGL((KERN<DT, SCORE, 8>), g, b, 0, s, p);                          \
    else hipLaunchKernelGGL((KERN<DT, SCORE, 16>), g, b, 0, s, p);                                               \
  } while (0)

}  // namespace

hipError_t launch_route(int dtype, int score, const RouteParams& p, hipStream_t s) {
  return dtype == DS_BF16 ? route_dt<DS_BF16>(score, p, s) : route_dt<DS_FP32>(score, p, s);
}

hipError_t launch_route_grad(int dtype, int score, const RouteGradParams& p, hipStream_t s) {
  if (dtype == DS_BF16) {
    if (score == DS_SCORE_SOFTMAX) DS_ROUTE_V(route_grad_kernel, DS_BF16, DS_SCORE_SOFTMAX);
    else DS_ROUTE_V(route_grad_kernel, DS_BF16, DS_SCORE_SIGMOID);
  } else {
    if (score == DS_SCORE_SOFTMAX) DS_ROUTE_V(route_grad_kernel, DS_FP32, DS_SCORE_SOFTMAX);
    else DS_ROUTE_V(route_grad_kernel, DS_FP32, DS_SCORE_SIGMOID);
  }
  return hipGetLastError();
}

}  // namespace ds
