// route.cu -- routing of tokens to experts: scores, balance biases, groups,
// top-k and its weights, and their gradient.
//
// For a row of E logits l (one token):
//   s = softmax(l) or sigma(l)
//   c = s + b, and -inf where l or b is -inf: the selection score
//   a group's score is its largest c, or the sum of its two largest (those at
//   -inf left out); the best top_groups groups stay
//   the k largest c of what stays, in descending order, equal ones to the
//   lower index; w_i = scale s_i / sum_j s_j, or scale s_i
// A slot whose c is -inf is empty: expert -1, weight 0.
//
// The choice does not depend on rounding.  Without a bias the ranking of c is
// the ranking of l and is done on l itself.  With one, c is computed in
// float32 and every decision the row took (between neighbours in the order,
// at the k-th place, between groups) is checked against a bound on the error
// of c; a row with a decision inside that bound is done again in float64.
//
// One warp per row.  Lane l holds the experts l, l + 32, ...: loads are
// coalesced for any E, and each of the k picks is two warp reductions (the
// largest key, then the lowest index that has it).
//
// The gradient: with n_i = s_i / sum_j s_j,
//   ds_i = scale (dw_i - sum_j dw_j n_j) / sum_j s_j (renormalised), or
//   ds_i = scale dw_i; plus a dense ds (a balance loss on the scores)
//   softmax: dl = s (ds - sum_e s_e ds_e);  sigmoid: dl = s (1 - s) ds
#include <cmath>

#include "async_util.cuh"
#include "experts.cuh"

namespace sfn {
namespace {

constexpr int kWarps = 4;  // rows in flight per block
constexpr int kNone = 0x7fffffff;

struct RouteParams {
  const void *logits;
  const float *bias;
  int32_t *experts;
  float *weights;
  float *scores;
  int64_t T;
  int E, k, groups, group_size, top_groups, group_top;
  bool sigmoid, renorm;
  float scale;
};

template <bool kBf16>
__device__ __forceinline__ float load_logit(const void *p, int64_t i) {
  if (kBf16) return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(p) + i) << 16);
  return __ldg(static_cast<const float *>(p) + i);
}

// Order keys: larger score, larger key; NaN 0, below -inf; +0 = -0.
__device__ __forceinline__ uint32_t key_of(float c) { return order_key(c); }
__device__ __forceinline__ uint64_t key_of(double c) {
  uint64_t b = (uint64_t)__double_as_longlong(c);
  if ((b & 0x7fffffffffffffffull) > 0x7ff0000000000000ull) return 0ull;
  if ((b << 1) == 0ull) b = 0ull;
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
__device__ __forceinline__ uint32_t warp_max_key(uint32_t k) { return __reduce_max_sync(kFull, k); }
__device__ __forceinline__ uint64_t warp_max_key(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(kFull, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(kFull, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ float warp_max(float v) {  // NaN is ignored
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
template <class R>
__device__ __forceinline__ R warp_add(R v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

// One score from its logit; m and z are the row's maximum and sum of
// exponentials (softmax only; z = 0 for a row of -inf, whose scores are 0).
template <class R>
__device__ __forceinline__ R score_of(float l, bool sigmoid, float m, R z) {
  if (sigmoid) return R(1) / (R(1) + exp_of(-(R)l));
  return z == R(0) ? R(0) : exp_of((R)l - (R)m) / z;
}

template <class R>
__device__ __forceinline__ R select_score(R s, float l, float b) {
  return (l == -INFINITY || b == -INFINITY) ? (R)-INFINITY : s + (R)b;
}

// The k experts of one row, from the selection scores c of this lane's
// experts lane + 32 j (those past E are never looked at).  Lane i returns slot
// i's expert.  `next`: the best expert left over (kNone: none).  gap_lo and
// gap_hi: the worst score of a kept group and the best of a dropped one.
template <int V, class R>
__device__ int choose(const R (&c)[V], const RouteParams &p, R *row_smem, int &next, R &gap_lo,
                      R &gap_hi) {
  using Key = decltype(key_of(R(0)));
  const int lane = threadIdx.x & 31;
  uint32_t gone = 0u;  // bit j: expert lane + 32 j is out
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (lane + 32 * j >= p.E) gone |= 1u << j;
  gap_lo = (R)INFINITY;
  gap_hi = (R)-INFINITY;
  if (p.groups > 1) {
    // all scores to shared memory; 32 / (groups rounded up to a power of two)
    // lanes per group find its two largest
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane + 32 * j < p.E) row_smem[lane + 32 * j] = c[j];
    __syncwarp();
    int per = 32;
    while (32 / per < p.groups) per >>= 1;
    const int g = lane / per;
    const bool have = g < p.groups;
    const R none = (R)-INFINITY;
    R a = none, b = none;  // the two largest (NaN: below -inf, so never kept over it)
    if (have)
      for (int i = lane % per; i < p.group_size; i += per) {
        const R v = row_smem[g * p.group_size + i];
        if (key_of(v) > key_of(a)) {
          b = a;
          a = v;
        } else if (key_of(v) > key_of(b)) {
          b = v;
        }
      }
    for (int o = per >> 1; o > 0; o >>= 1) {
      const R a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
      if (key_of(a2) > key_of(a)) {
        b = key_of(a) > key_of(b2) ? a : b2;
        a = a2;
      } else {
        b = key_of(a2) > key_of(b) ? a2 : b;
      }
    }
    const R gs = (p.group_top == 2 && b != none) ? a + b : a;
    const Key gk = key_of(gs);
    int rank = 0;
    for (int h = 0; h < p.groups; ++h) {
      const Key hk = __shfl_sync(kFull, gk, h * per);
      rank += (hk > gk) | ((hk == gk) & (h < g));
    }
    const bool kept = have && rank < p.top_groups;
    const uint32_t kept_lanes = __ballot_sync(kFull, kept);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = lane + 32 * j;
      if (e < p.E && !((kept_lanes >> ((e / p.group_size) * per)) & 1u)) gone |= 1u << j;
    }
    R lo = kept ? gs : (R)INFINITY, hi = (have && !kept) ? gs : none;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const R l2 = __shfl_xor_sync(kFull, lo, o), h2 = __shfl_xor_sync(kFull, hi, o);
      lo = l2 < lo ? l2 : lo;
      hi = h2 > hi ? h2 : hi;
    }
    gap_lo = lo;
    gap_hi = hi;
    __syncwarp();
  }
  int mine = -1;
  Key bk = 0;
  int bi = kNone;
  auto local_best = [&] {
    bk = 0;
    bi = kNone;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Key kj = key_of(c[j]);
      if (!((gone >> j) & 1u) && (bi == kNone || kj > bk)) {
        bk = kj;
        bi = lane + 32 * j;
      }
    }
  };
  local_best();
  for (int i = 0;; ++i) {
    const Key top = warp_max_key(bk);
    const int at = (int)__reduce_min_sync(kFull, (unsigned)(bk == top ? bi : kNone));
    if (i == p.k) {
      next = at;
      break;
    }
    if (lane == i) mine = at;
    if (bi == at) {
      gone |= 1u << (at >> 5);
      local_best();
    }
  }
  return mine;
}

// Bounds on the error of a float32 score: expf is within 2 units in the last
// place, and each operation within half of one (u = 2^-24).
//   sigmoid: 4u from expf, u from the sum, u from the quotient: 6u s
//   softmax: the argument l - m is off by u |l - m|, which costs the score at
//   most u / e; expf 4u; the sum of up to 1024 terms (32 in a lane, then five
//   levels) 4u + 37u; the quotient u: below 48u s + u
// and c = s + b adds u |c|.
constexpr float kUlp = 5.9604645e-8f;
__device__ __forceinline__ float score_error(float s, float c, bool sigmoid) {
  return kUlp * ((sigmoid ? 6.f : 48.f) * s + 1.f + fabsf(c));
}

// kByLogit: no bias, and groups (if any) scored by their largest: the logits
// themselves are ranked.
template <bool kBf16, int V, bool kByLogit>
__global__ void __launch_bounds__(32 * kWarps) k_route(const RouteParams p) {
  extern __shared__ double route_smem[];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double *row64 = route_smem + (size_t)warp * (p.groups > 1 ? p.E : 0);
  float *row32 = reinterpret_cast<float *>(row64);
  const int64_t stride = (int64_t)gridDim.x * kWarps;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < p.T; t += stride) {
    float l[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = lane + 32 * j;
      l[j] = e < p.E ? load_logit<kBf16>(p.logits, t * p.E + e) : -INFINITY;
    }
    // softmax statistics and scores, where something needs all of them
    float m = 0.f, z = 1.f;
    const bool all = !kByLogit || p.scores != nullptr || !p.renorm;
    if (!p.sigmoid && all) {
      m = l[0];
#pragma unroll
      for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
      m = warp_max(m);
      z = 0.f;
      if (m != -INFINITY) {
#pragma unroll
        for (int j = 0; j < V; ++j) z += expf(l[j] - m);
        z = warp_add(z);
      }
    }
    if (p.scores != nullptr) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (lane + 32 * j < p.E)
          p.scores[t * p.E + lane + 32 * j] = score_of<float>(l[j], p.sigmoid, m, z);
    }
    int pick, next;
    if (kByLogit) {
      float lo, hi;
      pick = choose<V, float>(l, p, row32, next, lo, hi);
    } else {
      float c[V], lo, hi;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = lane + 32 * j;
        const float b = (p.bias != nullptr && e < p.E) ? __ldg(p.bias + e) : 0.f;
        c[j] = select_score(score_of<float>(l[j], p.sigmoid, m, z), l[j], b);
      }
      pick = choose<V, float>(c, p, row32, next, lo, hi);
      // Is every decision outside the error of c?  Lane i < k compares slot i
      // with slot i + 1, the last slot with the best expert left over.  Equal
      // logits with equal biases are true ties, which the index decides.
      auto score_at = [&](int e, float &le, float &be, float &se, float &ce) {
        le = -INFINITY;
        be = 0.f;
        se = 0.f;
        ce = -INFINITY;
        if (e >= 0 && e < p.E) {
          le = load_logit<kBf16>(p.logits, t * p.E + e);
          if (p.bias != nullptr) be = __ldg(p.bias + e);
          se = score_of<float>(le, p.sigmoid, m, z);
          ce = select_score(se, le, be);
        }
      };
      float l0, b0, s0, c0, l1, b1, s1, c1;
      score_at(pick, l0, b0, s0, c0);
      int after = __shfl_down_sync(kFull, pick, 1);
      if (lane == p.k - 1) after = next;
      score_at(after, l1, b1, s1, c1);
      bool unsure = false;
      if (lane < p.k && c0 > -INFINITY && c1 > -INFINITY && !(l0 == l1 && b0 == b1))
        unsure = c0 - c1 <= score_error(s0, c0, p.sigmoid) + score_error(s1, c1, p.sigmoid);
      if (p.groups > 1 && lo > -INFINITY && hi > -INFINITY && hi < INFINITY) {
        // a group's score sums at most two, each at most the largest score
        const float s = p.sigmoid ? 1.f : (z > 0.f ? 1.f / z : 0.f);
        unsure |= lo - hi <= 2.f * (score_error(s, lo, p.sigmoid) + score_error(s, hi, p.sigmoid)) +
                                 4.f * kUlp * (fabsf(lo) + fabsf(hi));
      }
      if (__any_sync(kFull, unsure)) {
        double z64 = 1.0, lo64, hi64;
        if (!p.sigmoid) {
          z64 = 0.0;
          if (m != -INFINITY) {
#pragma unroll 1
            for (int j = 0; j < V; ++j) {
              const int e = lane + 32 * j;
              if (e < p.E)
                z64 += exp((double)load_logit<kBf16>(p.logits, t * p.E + e) - (double)m);
            }
            z64 = warp_add(z64);
          }
        }
        double c64[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int e = lane + 32 * j;
          const float b = (p.bias != nullptr && e < p.E) ? __ldg(p.bias + e) : 0.f;
          c64[j] = select_score(score_of<double>(l[j], p.sigmoid, m, z64), l[j], b);
        }
        pick = choose<V, double>(c64, p, row64, next, lo64, hi64);
      }
    }
    // a NaN anywhere makes the softmax, and with it every weight of the row, NaN
    bool nan = false;
    if (!p.sigmoid) {
#pragma unroll
      for (int j = 0; j < V; ++j) nan |= l[j] != l[j];
      nan = __any_sync(kFull, nan);
    }
    // weights: lane i < k has slot i
    const bool slot = lane < p.k;
    float lp = -INFINITY;
    if (slot && pick >= 0 && pick < p.E) {
      lp = load_logit<kBf16>(p.logits, t * p.E + pick);
      if (p.bias != nullptr && __ldg(p.bias + pick) == -INFINITY) lp = -INFINITY;
    }
    const bool empty = lp == -INFINITY;
    float w;
    if (p.renorm && !p.sigmoid) {
      // s_i / sum s: the row's sum cancels; the largest chosen logit in its
      // place, so that nothing underflows
      const float mc = warp_max(empty ? -INFINITY : lp);
      w = empty ? 0.f : expf(lp - mc);
    } else {
      w = empty ? 0.f : score_of<float>(lp, p.sigmoid, m, z);
    }
    if (p.renorm) {
      const float sum = warp_add(slot ? w : 0.f);
      w = sum == 0.f ? 0.f : w / sum;
    }
    if (slot) {
      p.experts[t * p.k + lane] = empty ? -1 : pick;
      p.weights[t * p.k + lane] =
          empty ? 0.f : (nan ? __int_as_float(0x7fc00000) : w * p.scale);
    }
  }
}

template <bool kBf16, int V>
__global__ void __launch_bounds__(32 * kWarps)
    k_route_bwd(const void *__restrict__ logits, const int32_t *__restrict__ experts,
                const float *__restrict__ dweights, const float *__restrict__ dscores,
                void *__restrict__ dlogits, int64_t T, int E, int k, bool sigmoid, bool renorm,
                float scale) {
  extern __shared__ float bwd_smem[];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float *extra = bwd_smem + warp * E;  // the chosen experts' ds, 0 elsewhere
  const int64_t stride = (int64_t)gridDim.x * kWarps;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < T; t += stride) {
    const bool dense = !sigmoid || dscores != nullptr;  // every score is needed
    float l[V], ds[V];
    float m = 0.f, z = 1.f;
    if (dense) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = lane + 32 * j;
        l[j] = e < E ? load_logit<kBf16>(logits, t * E + e) : -INFINITY;
        ds[j] = (dscores != nullptr && e < E) ? __ldg(dscores + t * E + e) : 0.f;
      }
      if (!sigmoid) {
        m = l[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
        m = warp_max(m);
        z = 0.f;
        if (m != -INFINITY) {
#pragma unroll
          for (int j = 0; j < V; ++j) z += expf(l[j] - m);
          z = warp_add(z);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane + 32 * j < E) extra[lane + 32 * j] = 0.f;
    // lane i < k: slot i
    int e = -1;
    float s = 0.f, dw = 0.f;
    if (lane < k) {
      e = experts[t * k + lane];
      if (e < 0 || e >= E) e = -1;
      if (e >= 0) {
        s = score_of<float>(load_logit<kBf16>(logits, t * E + e), sigmoid, m, z);
        dw = dweights[t * k + lane];
      }
    }
    float d = scale * dw;
    if (renorm) {
      const float sum = warp_add(s);
      const float mean = sum == 0.f ? 0.f : warp_add(dw * s) / sum;
      d = sum == 0.f ? 0.f : scale * (dw - mean) / sum;
    }
    if (e < 0) d = 0.f;
    // the same expert in two slots: the first of them takes the sum
    bool first = e >= 0;
    float mine = 0.f;
    for (int i = 0; i < k; ++i) {
      const int ei = __shfl_sync(kFull, e, i);
      const float di = __shfl_sync(kFull, d, i);
      if (ei == e) {
        mine += di;
        if (i < lane) first = false;
      }
    }
    __syncwarp();
    if (first) extra[e] = mine;
    __syncwarp();
    float dot = 0.f;
    if (!sigmoid) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int ej = lane + 32 * j;
        if (ej < E) {
          ds[j] += extra[ej];
          l[j] = score_of<float>(l[j], false, m, z);
          dot += l[j] * ds[j];
        }
      }
      dot = warp_add(dot);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int ej = lane + 32 * j;
      if (ej >= E) continue;
      float g;
      if (!sigmoid) {
        g = l[j] * (ds[j] - dot);
      } else {
        const float x = extra[ej] + (dscores != nullptr ? ds[j] : 0.f);
        if (x == 0.f) {
          g = 0.f;
        } else {
          const float lj = dense ? l[j] : load_logit<kBf16>(logits, t * E + ej);
          // 1 - sigma(l) = sigma(-l), without the cancellation
          g = x * score_of<float>(lj, true, 0.f, 1.f) * score_of<float>(-lj, true, 0.f, 1.f);
        }
      }
      if (kBf16)
        static_cast<uint16_t *>(dlogits)[t * E + ej] = f32_to_bf16_bits(g);
      else
        static_cast<float *>(dlogits)[t * E + ej] = g;
    }
    __syncwarp();
  }
}

int route_grid(int64_t T, int num_sms) {
  const int64_t blocks = (T + kWarps - 1) / kWarps;
  const int64_t most = (int64_t)num_sms * 16;
  return (int)(blocks < most ? blocks : most);
}

// The smallest built V with 32 V >= E.
template <class F>
cudaError_t with_values_per_lane(int E, F &&f) {
  if (E <= 32) return f(std::integral_constant<int, 1>{});
  if (E <= 64) return f(std::integral_constant<int, 2>{});
  if (E <= 128) return f(std::integral_constant<int, 4>{});
  if (E <= 256) return f(std::integral_constant<int, 8>{});
  if (E <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

}  // namespace

cudaError_t launch_route(const RouteShape &s, const void *logits, const float *bias,
                         int32_t *experts, float *weights, float *scores, int num_sms,
                         cudaStream_t st) {
  RouteParams p{logits, bias, experts, weights, scores, s.T, s.E, s.k, s.groups,
                s.E / s.groups, s.top_groups, s.group_top, s.sigmoid, s.renorm, s.scale};
  const bool by_logit = bias == nullptr && (s.groups == 1 || s.group_top == 1);
  const size_t smem = s.groups > 1 ? (size_t)kWarps * s.E * sizeof(double) : 0;
  return with_values_per_lane(s.E, [&](auto v) {
    constexpr int V = decltype(v)::value;
    auto *kern = s.bf16 ? (by_logit ? k_route<true, V, true> : k_route<true, V, false>)
                        : (by_logit ? k_route<false, V, true> : k_route<false, V, false>);
    count_launches(1);
    return launch_pdl(kern, dim3(route_grid(s.T, num_sms)), dim3(32 * kWarps), smem, st, p);
  });
}

cudaError_t launch_route_backward(const RouteShape &s, const void *logits,
                                  const int32_t *experts, const float *dweights,
                                  const float *dscores, void *dlogits, int num_sms,
                                  cudaStream_t st) {
  return with_values_per_lane(s.E, [&](auto v) {
    constexpr int V = decltype(v)::value;
    auto *kern = s.bf16 ? k_route_bwd<true, V> : k_route_bwd<false, V>;
    count_launches(1);
    return launch_pdl(kern, dim3(route_grid(s.T, num_sms)), dim3(32 * kWarps),
                      (size_t)kWarps * s.E * sizeof(float), st, logits, experts, dweights,
                      dscores, dlogits, s.T, s.E, s.k, s.sigmoid, s.renorm, s.scale);
  });
}

}  // namespace sfn
