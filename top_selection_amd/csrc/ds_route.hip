// Routing to experts and its gradient.
#include "ds_rows_device.h"

namespace ds {
namespace {

constexpr int kRouteWaves = 4;
constexpr double kNone = -__builtin_huge_val();  // the selection score of a masked or taken expert

// One wave per row, expert e in lane e % 64. Everything that decides the choice is in double.
template <int DT, int SCORE, int V>
__global__ __launch_bounds__(kRouteWaves * 64) void route_kernel(RouteParams p) {
  using E = Elem<DT>;
  __shared__ double of_group[kRouteWaves][64 * V];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const typename E::T* x = static_cast<const typename E::T*>(p.x);
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRouteWaves + wave; r < p.rows;
       r += static_cast<int64_t>(gridDim.x) * kRouteWaves) {
    float xv[V];
    double s[V], c[V];
    float m = -__builtin_huge_valf();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 64 + lane;
      xv[v] = e < p.experts ? E::widen(x[r * p.row_stride + e]) : -__builtin_huge_valf();
      m = fmaxf(m, xv[v]);
    }
    double inv = 1.0;
    if constexpr (SCORE == DS_SCORE_SOFTMAX) {
      m = wave_max(m);
      double z = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[v] = xv[v] == -__builtin_huge_valf() ? 0.0
               : xv[v] == m                    ? 1.0
                                               : exp(static_cast<double>(xv[v]) - static_cast<double>(m));
        z += s[v];
      }
      z = wave_sum(z);
      inv = z > 0.0 ? 1.0 / z : 0.0;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 64 + lane;
      if constexpr (SCORE == DS_SCORE_SOFTMAX) s[v] *= inv;
      else s[v] = 1.0 / (1.0 + exp(-static_cast<double>(xv[v])));
      c[v] = xv[v] == -__builtin_huge_valf() ? kNone
             : p.bias                        ? s[v] + static_cast<double>(p.bias[e])
                                             : static_cast<double>(xv[v]);
    }
    if (p.topk_groups < p.groups) {
      double* g = of_group[wave];
#pragma unroll
      for (int v = 0; v < V; ++v)  // group scores add scores: without a bias those are not the order's logits
        g[v * 64 + lane] = (!p.bias && p.group_top > 1 && c[v] != kNone) ? s[v] : c[v];
      __builtin_amdgcn_wave_barrier();
      double top = kNone, second = kNone;
      if (lane < p.groups)
        for (int j = 0; j < p.group_size; ++j) {
          const double q = g[lane * p.group_size + j];
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
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = v * 64 + lane;
        if (e < p.experts && !((keep >> (e / p.group_size)) & 1)) c[v] = kNone;
      }
      __builtin_amdgcn_wave_barrier();
    }
    int my_e = -1;
    double my_s = 0.0, total = 0.0;
    for (int j = 0; j < p.k; ++j) {
      double best = kNone, bs = 0.0;
      int at = 0x7FFFFFFF;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (c[v] > best) best = c[v], bs = s[v], at = v * 64 + lane;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) {
        const double ob = __shfl_xor(best, o), os = __shfl_xor(bs, o);
        const int oa = __shfl_xor(at, o);
        if (ob > best || (ob == best && oa < at)) best = ob, bs = os, at = oa;
      }
      if (at == 0x7FFFFFFF) break;  // nothing left
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v * 64 + lane == at) c[v] = kNone;
      if (lane == j) my_e = at, my_s = bs;
      total += bs;
    }
    if (lane < p.k) {
      const double w = !p.renorm ? my_s : total > 0.0 ? my_s / total : 0.0;
      if (p.out_weights) p.out_weights[r * p.k + lane] = static_cast<float>(w * static_cast<double>(p.scale));
      if (p.out_idx) p.out_idx[r * p.k + lane] = my_e;
      if (p.counts && my_e >= 0) atomicAdd(p.counts + my_e, 1);
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

template <class P>
uint32_t route_grid(const P& p) {
  const int64_t need = (p.rows + kRouteWaves - 1) / kRouteWaves, most = kCus * 16;
  return static_cast<uint32_t>(need < most ? need : most);
}

#define DS_ROUTE_V(KERN, DT, SCORE)                                                                              \
  do {                                                                                                           \
    const dim3 g(route_grid(p)), b(kRouteWaves * 64);                                                       \
    if (p.experts <= 64) hipLaunchKernelGGL((KERN<DT, SCORE, 1>), g, b, 0, s, p);                                \
    else if (p.experts <= 128) hipLaunchKernelGGL((KERN<DT, SCORE, 2>), g, b, 0, s, p);                          \
    else if (p.experts <= 256) hipLaunchKernelGGL((KERN<DT, SCORE, 4>), g, b, 0, s, p);                          \
    else if (p.experts <= 512) hipLaunchKernelGGL((KERN<DT, SCORE, 8>), g, b, 0, s, p);                          \
    else hipLaunchKernelGGL((KERN<DT, SCORE, 16>), g, b, 0, s, p);                                               \
  } while (0)

#define DS_ROUTE_PICK(KERN)                                                    \
  do {                                                                         \
    if (dtype == DS_BF16) {                                                    \
      if (score == DS_SCORE_SOFTMAX) DS_ROUTE_V(KERN, DS_BF16, DS_SCORE_SOFTMAX); \
      else DS_ROUTE_V(KERN, DS_BF16, DS_SCORE_SIGMOID);                        \
    } else {                                                                   \
      if (score == DS_SCORE_SOFTMAX) DS_ROUTE_V(KERN, DS_FP32, DS_SCORE_SOFTMAX); \
      else DS_ROUTE_V(KERN, DS_FP32, DS_SCORE_SIGMOID);                        \
    }                                                                          \
  } while (0)

}  // namespace

hipError_t launch_route(int dtype, int score, const RouteParams& p, hipStream_t s) {
  DS_ROUTE_PICK(route_kernel);
  return hipGetLastError();
}

hipError_t launch_route_grad(int dtype, int score, const RouteGradParams& p, hipStream_t s) {
  DS_ROUTE_PICK(route_grad_kernel);
  return hipGetLastError();
}

}  // namespace ds
