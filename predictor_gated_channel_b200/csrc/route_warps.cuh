// route_warps.cuh -- routing (route.cuh) with a warp per row; built for one type
// each by route_f32.cu and route_bf16.cu.
#pragma once

#include "route.cuh"

namespace sfn {
namespace {

// One warp per row.
template <bool kBf16, int V, bool kBlocked, bool kByLogit, bool kGroups>
__global__ void __launch_bounds__(32 * kWarps, (route_blocks<V, kByLogit>()))
    k_route(const RouteParams p) {
  extern __shared__ double route_smem[];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float bias[kByLogit ? 1 : V];
  if constexpr (!kByLogit) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = expert_of<V, kBlocked>(j);
      bias[j] = (p.bias != nullptr && e < p.E) ? __ldg(p.bias + e) : 0.f;
    }
  }
  const int64_t stride = (int64_t)gridDim.x * kWarps;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < p.T; t += stride) {
    float l[V];
    load_row<kBf16, V, kBlocked>(p.logits, t, p.E, l);
    const bool nan = row_has_nan<V>(l);
    // softmax statistics, where something needs every score: z_fast for the
    // choice, z for what is written
    float m = 0.f, z = 1.f, z_fast = 1.f;
    const bool exact_z = !p.sigmoid && (p.scores != nullptr || !p.renorm);
    if (!p.sigmoid && (!kByLogit || exact_z)) {
      m = row_max<V>(l, nan);
      if (!kByLogit) z_fast = row_sum<V, true>(l, m);
      if (exact_z) z = row_sum<V, false>(l, m);
    }
    if (p.scores != nullptr) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (expert_of<V, kBlocked>(j) < p.E)
          p.scores[t * p.E + expert_of<V, kBlocked>(j)] = score_of<float>(l[j], p.sigmoid, m, z);
    }
    float lp, bp;
    const int pick = select_row<kBf16, V, kBlocked, kByLogit, kGroups>(
        p, t, l, bias, nan, m, z_fast, route_smem + (size_t)warp * (kGroups ? p.E : 0), lp, bp);
    const bool slot = lane < p.k;
    if (!slot || bp == -INFINITY) lp = -INFINITY;  // (the choice may leave more than k)
    const bool empty = lp == -INFINITY;
    float w;
    if (p.renorm) {
      const float top = key_value(__reduce_max_sync(kFull, empty ? 0u : order_key(lp)));
      // (ranked by logits, a softmax row's largest is among the chosen)
      const bool none = shares_vanish(p.sigmoid, top, kByLogit ? top : m);
      w = empty || none ? 0.f : share_of(lp, p.sigmoid, top);
    } else {
      w = empty ? 0.f : score_of<float>(lp, p.sigmoid, m, z);
    }
    if (p.renorm) {
      const float sum = warp_add(slot ? w : 0.f);
      w = sum == 0.f ? 0.f : w / sum;
    }
    if (slot) {
      // a NaN or +inf anywhere makes the softmax, and with it every weight, NaN
      const bool bad = !p.sigmoid && (nan || m == INFINITY);
      p.experts[t * p.k + lane] = empty ? -1 : pick;
      p.weights[t * p.k + lane] =
          empty ? 0.f : (bad ? __int_as_float(0x7fc00000) : w * p.scale);
    }
  }
}

}  // namespace

// The kernels of one type: a warp per row.
template <bool kBf16>
cudaError_t launch_route_warps(const RouteParams &p, bool by_logit, int num_sms, cudaStream_t st) {
  const bool groups = p.groups > 1;
  const size_t smem = groups ? (size_t)kWarps * p.E * sizeof(double) : 0;
  return with_layout(p.E, aligned16({p.logits}), groups, [&](auto v, auto blocked) {
    constexpr int V = decltype(v)::value;
    constexpr bool kB = decltype(blocked)::value;
    auto go = [&](auto logit, auto grouped) {
      // (not reached, and not built)
      if constexpr (kB && !vector_part<V>() && !decltype(grouped)::value)
        return cudaErrorInvalidValue;
      else
        return launch_rows(k_route<kBf16, V, kB, decltype(logit)::value, decltype(grouped)::value>,
                           p.T, route_blocks<V, decltype(logit)::value>(), smem, num_sms, st, p);
    };
    auto with_groups = [&](auto logit) {
      return groups ? go(logit, std::true_type{}) : go(logit, std::false_type{});
    };
    return by_logit ? with_groups(std::true_type{}) : with_groups(std::false_type{});
  });
}

}  // namespace sfn
