// route_lanes.cu -- routing (route.cuh) with eight lanes per row, for many rows.
#include "route.cuh"

namespace sfn {
namespace {

// As select_row(), on its own: for the few rows that k_route_lanes leaves.
template <bool kBf16, int V, bool kBlocked, bool kByLogit, bool kGroups>
__device__ __noinline__ int select_left_row(const RouteParams &p, int64_t t, double *row64) {
  float l[V], bias[kByLogit ? 1 : V];
  load_row<kBf16, V, kBlocked>(p.logits, t, p.E, l);
  const bool nan = row_has_nan<V>(l);
  float m = 0.f, z = 1.f, lp, bp;
  if constexpr (!kByLogit) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = expert_of<V, kBlocked>(j);
      bias[j] = (p.bias != nullptr && e < p.E) ? __ldg(p.bias + e) : 0.f;
    }
    if (!p.sigmoid) {
      m = row_max<V>(l, nan);
      z = row_sum<V, true>(l, m);
    }
  }
  return select_row<kBf16, V, kBlocked, kByLogit, kGroups>(p, t, l, bias, nan, m, z, row64, lp, bp);
}

// The eight largest of V words, in descending order: blocks of eight sorted
// and merged, the larger of a pair from both ends being the upper half of a
// merge.
template <int V>
__device__ __forceinline__ void top8(const uint32_t (&w)[V], uint32_t (&top)[8]) {
#pragma unroll
  for (int b = 0; b < V; b += 8) {
    uint32_t s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = b + i < V ? w[b + i] : 0u;
    sort_descending<8>(s);
    if (b == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top[i] = s[i];
      continue;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) top[i] = max(top[i], s[7 - i]);
#pragma unroll
    for (int q = 4; q >= 1; q /= 2)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((i & q) == 0) cex_desc(top[i], top[i + q]);
  }
}

template <bool kByLogit>
constexpr Lanes route_kind() {
  return kByLogit ? Lanes::kByLogit : Lanes::kByScore;
}

// Eight lanes per row, four rows a warp, k <= 8: for many rows, where the
// instructions that do not depend on E (picks, weights, stores, loop) count;
// four rows share them.  V = E / 8 values a lane, neighbours with kGroups (8
// lanes are then a whole number for each group; by logit only), else every eighth.  A row with
// anything to settle (a NaN, neighbours or a k-th place within the words or the
// error bound, more than eight of one lane) is left to the whole warp.
template <bool kBf16, int V, bool kByLogit, bool kGroups>
__global__ void __launch_bounds__(32 * kWarps, (lanes_blocks<V, route_kind<kByLogit>()>()))
    k_route_lanes(const RouteParams p) {
  static_assert(kByLogit || !kGroups, "groups are ranked by their largest logit here");
  extern __shared__ double route_smem[];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % kRowLanes, first = lane - sub;
  const uint32_t row_mask = 0xffu << first;
  const int per = kGroups ? kRowLanes / p.groups : kRowLanes;
  const uint32_t none = order_key(-INFINITY);
  constexpr bool kWhole = kByLogit && kBf16;
  constexpr uint32_t kPlaces = places<V>();
  const uint32_t low = kWhole ? p.low : kPlaces;
  auto expert = [&](int owner, int j) { return kGroups ? owner * V + j : owner + kRowLanes * j; };
  float bias[kByLogit ? 1 : V];
  if constexpr (!kByLogit) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      bias[j] = (p.bias != nullptr && expert(sub, j) < p.E) ? __ldg(p.bias + expert(sub, j)) : 0.f;
  }
  const int64_t stride = (int64_t)gridDim.x * kWarps * 4;
  for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * 4; t0 < p.T; t0 += stride) {
    const bool live = t0 + first / kRowLanes < p.T;
    const int64_t t = live ? t0 + first / kRowLanes : p.T - 1;
    float l[V];
    load_row<kBf16, V, kGroups, kRowLanes>(p.logits, t, p.E, l);
    bool nan = false;
#pragma unroll
    for (int j = 0; j < V; ++j) nan |= l[j] != l[j];
    nan = (__ballot_sync(kFull, nan) & row_mask) != 0u;
    float m = 0.f, z = 1.f, z_fast = 1.f;
    if (!p.sigmoid && (!kByLogit || !p.renorm)) {
      m = l[0];
#pragma unroll
      for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
      const uint32_t key = lanes_max(order_key(m));
      m = key == 0u ? -INFINITY : key_value(key);
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (!kByLogit) a += __expf(l[j] - m);
        if (!p.renorm) b += expf(l[j] - m);
      }
      // the sums by all lanes: the rows of a warp differ in m
      a = lanes_add(a);
      b = lanes_add(b);
      z_fast = m == -INFINITY ? 0.f : a;
      z = m == -INFINITY ? 0.f : b;
    }
    float c[V];
    bool number = true;  // the words have no room for a NaN (of a bias, of exp(inf - inf))
#pragma unroll
    for (int j = 0; j < V; ++j) {
      c[j] = kByLogit ? l[j]
                      : select_score(score_fast(l[j], p.sigmoid, m, z_fast), l[j], bias[j]);
      if (!kByLogit) number &= c[j] == c[j];
    }
    const float most = p.sigmoid || kByLogit ? 1.f : (z_fast > 0.f ? __fdividef(1.f, z_fast) : 0.f);
    auto bound = [&](float x) { return score_error(most, x, p.sigmoid); };
    bool unsure = nan || (!kByLogit && !number), in = true;
    if (kGroups) {  // by their largest logit
      float gs = -INFINITY;
#pragma unroll
      for (int j = 0; j < V; ++j) gs = fmaxf(gs, c[j]);
      for (int o = per >> 1; o > 0; o >>= 1) gs = fmaxf(gs, __shfl_xor_sync(kFull, gs, o));
      int rank = 0;
      for (int o = per; o < kRowLanes; o += per) {
        const float other = __shfl_xor_sync(kFull, gs, o);
        rank += other > gs || (other == gs && (sub ^ o) / per < sub / per);
      }
      in = rank < p.top_groups;
    }
    uint32_t w[V], top[8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = expert(sub, j);
      const uint32_t place = kWhole ? p.low - (uint32_t)e : kPlaces - (uint32_t)j;
      w[j] = (in && (kGroups || e < p.E)) ? (number_key(c[j]) & ~low) | place : 0u;
    }
    const bool any = w[0] != 0u;  // the lane's lowest index: it has values
    top8<V>(w, top);
    uint32_t mine = 0u;
    int winner = 0;
    for (int i = 0; i < p.k; ++i) {
      const uint32_t best = lanes_max(top[0]);
      bool won = top[0] == best;
      if constexpr (!kWhole) {
        const int at = __ffs(__ballot_sync(kFull, won) & row_mask) - 1;
        won = lane == at;
        if (sub == i) winner = at - first;
      }
      if (sub == i) mine = best;
      if (won) {
#pragma unroll
        for (int j = 0; j < 7; ++j) top[j] = top[j + 1];
        top[7] = 0u;
      }
    }
    // eight of one lane's: its ninth is not known
    unsure |= V > 8 && any && top[0] == 0u;
    const bool slot = sub < p.k;
    int pick = -1;
    float lp = -INFINITY, bp = 0.f;
    if constexpr (kWhole) {
      if (slot) {
        pick = (int)(p.low - (mine & p.low));
        const uint32_t kept = mine & ~low;
        lp = __uint_as_float((kept & 0x80000000u) ? kept & 0x7fff0000u : ~kept & 0xffff0000u);
      }
    } else {
      float cp = -INFINITY;
      if (slot) {
        pick = expert(winner, (int)(kPlaces - (mine & kPlaces)));
        lp = load_logit<kBf16>(p.logits, t * p.E + pick);
        if (!kByLogit && p.bias != nullptr) bp = __ldg(p.bias + pick);
        cp = kByLogit ? lp : select_score(score_fast(lp, p.sigmoid, m, z_fast), lp, bp);
      }
      float c1 = __shfl_down_sync(kFull, cp, 1);
      int e1 = __shfl_down_sync(kFull, pick, 1);
      if (__any_sync(kFull, sub < p.k - 1 && before(c1, e1, cp, pick))) {
        exchange_sort(p.k, sub, first, cp, pick, lp, bp);
        c1 = __shfl_down_sync(kFull, cp, 1);
      }
      const uint32_t left = lanes_max(top[0]);
      const bool rest = left != 0u && (left & ~low) != (none & ~low);
      const float hi = key_value(left | low);
      if constexpr (kByLogit) {
        unsure |= sub == p.k - 1 && rest && !(cp > hi);
      } else {
        const float l1 = __shfl_down_sync(kFull, lp, 1), b1 = __shfl_down_sync(kFull, bp, 1);
        if (slot && cp > -INFINITY) {
          if (sub == p.k - 1)
            unsure |= rest && !(cp - hi > bound(cp) + bound(hi));
          else
            unsure |= c1 > -INFINITY && !(lp == l1 && bp == b1) &&
                      !(cp - c1 > bound(cp) + bound(c1));
        }
      }
    }
    uint32_t left_rows = __ballot_sync(kFull, unsure && live);
    while (left_rows != 0u) {  // one row after the other, by the whole warp
      const int at = (__ffs(left_rows) - 1) & ~(kRowLanes - 1);
      left_rows &= ~(0xffu << at);
      constexpr int kV = V < 16 ? 2 : V / 4;  // values a lane of 32
      const int r = select_left_row<kBf16, kV, kGroups && kV * 4 == V, kByLogit, kGroups>(
          p, t0 + at / kRowLanes, route_smem + (size_t)warp * (kGroups ? p.E : 0));
      const int mine_now = __shfl_sync(kFull, r, sub);
      if (first == at && slot) {
        pick = mine_now;
        lp = -INFINITY;
        bp = 0.f;
        if (pick >= 0 && pick < p.E) {
          lp = load_logit<kBf16>(p.logits, t * p.E + pick);
          if (!kByLogit && p.bias != nullptr) bp = __ldg(p.bias + pick);
        }
      }
    }
    if (bp == -INFINITY) lp = -INFINITY;
    const bool empty = lp == -INFINITY;
    float weight;
    if (p.renorm) {  // as in k_route
      const float most_l = key_value(lanes_max(empty ? 0u : order_key(lp)));
      const bool none_left = shares_vanish(p.sigmoid, most_l, kByLogit ? most_l : m);
      weight = empty || none_left ? 0.f : share_of(lp, p.sigmoid, most_l);
    } else {
      weight = empty ? 0.f : score_of<float>(lp, p.sigmoid, m, z);
    }
    if (p.renorm) {
      const float sum = lanes_add(slot ? weight : 0.f);
      weight = sum == 0.f ? 0.f : weight / sum;
    }
    if (slot && live) {
      const bool bad = !p.sigmoid && (nan || m == INFINITY);  // as in k_route
      p.experts[t * p.k + sub] = empty ? -1 : pick;
      p.weights[t * p.k + sub] =
          empty ? 0.f : (bad ? __int_as_float(0x7fc00000) : weight * p.scale);
    }
  }
}

}  // namespace

template <bool kBf16>
cudaError_t launch_route_lanes(const RouteParams &p, bool by_logit, int num_sms, cudaStream_t st) {
  const bool groups = p.groups > 1;
  const size_t smem = groups ? (size_t)kWarps * p.E * sizeof(double) : 0;
  auto go = [&](auto v) {
    constexpr int V = decltype(v)::value;
    auto launch = [&](auto logit, auto grouped) {
      return launch_rows(
          k_route_lanes<kBf16, V, decltype(logit)::value, decltype(grouped)::value>,
          (p.T + 3) / 4, lanes_blocks<V, route_kind<decltype(logit)::value>()>(), smem, num_sms,
          st, p);
    };
    if (groups) return launch(std::true_type{}, std::true_type{});
    return by_logit ? launch(std::true_type{}, std::false_type{})
                    : launch(std::false_type{}, std::false_type{});
  };
  const int v = (p.E + kRowLanes - 1) / kRowLanes;
  if (v <= 8) return go(std::integral_constant<int, 8>{});
  if (v <= 16) return go(std::integral_constant<int, 16>{});
  if (v <= 20) return go(std::integral_constant<int, 20>{});
  return go(std::integral_constant<int, 32>{});
}
template cudaError_t launch_route_lanes<false>(const RouteParams &, bool, int, cudaStream_t);
template cudaError_t launch_route_lanes<true>(const RouteParams &, bool, int, cudaStream_t);

}  // namespace sfn
