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
// One warp per row, V = E / 32 (rounded up to a built one) values a lane.
// What bounds it is instruction issue, so the picks run on packed keys: the
// score's order key with the expert's index in its low bits, one 32-bit word
// that is unique in the row.  A lane sorts its V words once (a register
// network); a pick is then one warp maximum (redux) over the lanes' heads, and
// the lane that had it moves its list up.  The low bits cost the key some of
// its mantissa: where two neighbours of the order agree in what is left, or
// the last pick agrees with the best word left over, the row goes to the exact
// routine (choose()), which compares whole keys.  bf16 logits fit beside the
// index and are always exact.  Rows of exactly 32 V experts are loaded V
// neighbours a lane (16-byte loads), and groups of a whole number of lanes
// find their two largest scores with shuffles; others go through choose().
//   4096 x 256, 8 groups: 16.8 us; 22.5 us with choose() alone (2557 instructions a row)
//   32768 x 160, bf16:    22.5 us; 38.9 us with choose() alone (772 instructions a row)
//
// The gradient: with n_i = s_i / sum_j s_j,
//   ds_i = scale (dw_i - sum_j dw_j n_j) / sum_j s_j (renormalised), or
//   ds_i = scale dw_i; plus a dense ds (a balance loss on the scores)
//   softmax: dl = s (ds - sum_e s_e ds_e);  sigmoid: dl = s (1 - s) ds
#include <cmath>
#include <initializer_list>
#include <type_traits>

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
  uint32_t low;  // the bits of a packed word that hold the index
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

// The expert that value j of a lane belongs to.
template <int V, bool kBlocked>
__device__ __forceinline__ int expert_of(int j) {
  const int lane = threadIdx.x & 31;
  return kBlocked ? lane * V + j : lane + 32 * j;
}

// The k experts of one row, from the selection scores c of this lane's
// experts (those past E are never looked at).  Lane i returns slot i's
// expert.  `next`: the best expert left over (kNone: none).  gap_lo and
// gap_hi: the worst score of a kept group and the best of a dropped one.
template <int V, bool kBlocked, class R>
__device__ __noinline__ int choose(const R (&c)[V], const RouteParams &p, R *row_smem, int &next,
                                   R &gap_lo, R &gap_hi) {
  using Key = decltype(key_of(R(0)));
  const int lane = threadIdx.x & 31;
  uint32_t gone = 0u;  // bit j: value j is out
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (expert_of<V, kBlocked>(j) >= p.E) gone |= 1u << j;
  gap_lo = (R)INFINITY;
  gap_hi = (R)-INFINITY;
  if (p.groups > 1) {
    // all scores to shared memory; 32 / (groups rounded up to a power of two)
    // lanes per group find its two largest
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (expert_of<V, kBlocked>(j) < p.E) row_smem[expert_of<V, kBlocked>(j)] = c[j];
    __syncwarp();
    int per = 32;
    while (32 / per < p.groups) per >>= 1;
    const int g = lane / per;
    const bool have = g < p.groups;
    const R none = (R)-INFINITY;
    R a = none, b = none;
    Key ak = key_of(none), bk = ak;  // NaN's key is below -inf's: never kept over it
    auto offer = [&](R v) {
      const Key vk = key_of(v);
      if (vk > ak) {
        b = a;
        bk = ak;
        a = v;
        ak = vk;
      } else if (vk > bk) {
        b = v;
        bk = vk;
      }
    };
    if (have)
      for (int i = lane % per; i < p.group_size; i += per) offer(row_smem[g * p.group_size + i]);
    for (int o = per >> 1; o > 0; o >>= 1) {
      const R a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
      offer(a2);
      offer(b2);
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
    // e / group_size without a division: exact, as e + 1/2 is at least
    // 1 / (2 group_size) > 2^-11 away from a whole multiple
    const float inv = 1.f / (float)p.group_size;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int ge = (int)(((float)expert_of<V, kBlocked>(j) + 0.5f) * inv);
      if (!((kept_lanes >> (min(ge, p.groups - 1) * per)) & 1u)) gone |= 1u << j;
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
  Key key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) key[j] = key_of(c[j]);
  int mine = -1;
  Key bk = 0;
  int bi = kNone;
  auto local_best = [&] {
    bk = 0;
    bi = kNone;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (!((gone >> j) & 1u) && (bi == kNone || key[j] > bk)) {
        bk = key[j];
        bi = expert_of<V, kBlocked>(j);
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
      gone |= 1u << (kBlocked ? at % V : at >> 5);
      local_best();
    }
  }
  return mine;
}

// The same choice on packed words: w[j] the order key of value j's score with
// the index in the bits of p.low (complemented: of equal keys the lower index
// is the larger word), 0 for a value that is out.  Lane i returns slot i's
// word; `next` the best word left over.
template <int V>
__device__ __forceinline__ uint32_t choose_packed(uint32_t (&w)[V], int k, uint32_t &next) {
  const int lane = threadIdx.x & 31;
  BitonicSort<0, V, 2>::run(w);
  uint32_t mine = 0u;
  for (int i = 0; i < k; ++i) {
    const uint32_t top = __reduce_max_sync(kFull, w[0]);
    if (lane == i) mine = top;
    if (w[0] == top) {
#pragma unroll
      for (int j = 0; j + 1 < V; ++j) w[j] = w[j + 1];
      w[V - 1] = 0u;
    }
  }
  next = __reduce_max_sync(kFull, w[0]);
  return mine;
}

// Bounds on the error of the float32 scores that the choice is made on
// (u = 2^-24; one unit in the last place is at most 2u relative).  __expf(x) is
// documented to 2 + 1.173 |x| units, __fdividef to 2, an operation rounds u.
//   sigmoid: the exponential's error reaches s through s (1 - s) <= 1/4, and
//   s (1 - s) |l| <= 0.23: below 2u; the sum u s, the quotient 4u s: 8u in all
//   softmax: exp(-x) 2 (2 + 1.173 x) u <= 4u, and the argument's rounding
//   u x exp(-x) < u; the sum's error is at most the weighted mean of its terms'
//   (below 20u for up to 1024 terms) and 37 roundings; the quotient 4u:
//   below 80u s + 8u
// and c = s + b adds u |c|.
constexpr float kUlp = 5.9604645e-8f;
__device__ __forceinline__ float score_error(float s, float c, bool sigmoid) {
  return kUlp * ((sigmoid ? 0.f : 80.f * s) + 8.f + fabsf(c));
}
__device__ __forceinline__ float score_fast(float l, bool sigmoid, float m, float z) {
  if (sigmoid) return __fdividef(1.f, 1.f + __expf(-l));
  return z == 0.f ? 0.f : __fdividef(__expf(l - m), z);
}

// This lane's V logits of row t (-inf past E).
template <bool kBf16, int V, bool kBlocked>
__device__ __forceinline__ void load_row(const void *logits, int64_t t, int E, float (&l)[V]) {
  const int lane = threadIdx.x & 31;
  if constexpr (kBlocked) {
    constexpr int kBytes = V * (kBf16 ? 2 : 4);
    uint32_t raw[kBytes / 4];
    const char *src = static_cast<const char *>(logits) + (t * 32 + lane) * kBytes;
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 v = ld_nc16(src + i * 16);
        raw[4 * i] = v.x;
        raw[4 * i + 1] = v.y;
        raw[4 * i + 2] = v.z;
        raw[4 * i + 3] = v.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src));
      raw[0] = v.x;
      raw[1] = v.y;
    } else {
      raw[0] = __ldg(reinterpret_cast<const uint32_t *>(src));
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
      l[j] = kBf16 ? __uint_as_float((j & 1) ? (raw[j / 2] & 0xffff0000u) : (raw[j / 2] << 16))
                   : __uint_as_float(raw[kBf16 ? 0 : j]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = lane + 32 * j;
      l[j] = e < E ? load_logit<kBf16>(logits, t * E + e) : -INFINITY;
    }
  }
}

// Maximum over the row (NaN ignored) and, given it, the sum of exponentials.
template <int V>
__device__ __forceinline__ float row_max(const float (&l)[V]) {
  float m = l[0];
#pragma unroll
  for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
  const uint32_t key = __reduce_max_sync(kFull, order_key(m));
  return key == 0u ? -INFINITY : key_value(key);
}
template <int V, bool kFast>
__device__ __forceinline__ float row_sum(const float (&l)[V], float m) {
  float z = 0.f;
  if (m != -INFINITY) {
#pragma unroll
    for (int j = 0; j < V; ++j) z += kFast ? __expf(l[j] - m) : expf(l[j] - m);
    z = warp_add(z);
  }
  return z;
}

// kByLogit: no bias, and groups (if any) scored by their largest: the logits
// themselves are ranked.  kGroups: groups > 1.
template <bool kBf16, int V, bool kBlocked, bool kByLogit, bool kGroups>
__global__ void __launch_bounds__(32 * kWarps) k_route(const RouteParams p) {
  extern __shared__ double route_smem[];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double *row64 = route_smem + (size_t)warp * (kGroups ? p.E : 0);
  float *row32 = reinterpret_cast<float *>(row64);
  // groups of a whole number of lanes; then every lane of a group knows it
  const bool lanes_per_group = kGroups && kBlocked && 32 % p.groups == 0;
  const int per = kGroups ? 32 / p.groups : 32;
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
    bool nan = false;
#pragma unroll
    for (int j = 0; j < V; ++j) nan |= l[j] != l[j];
    nan = __any_sync(kFull, nan);
    // softmax statistics, where something needs every score: z_fast for the
    // choice, z for what is written
    float m = 0.f, z = 1.f, z_fast = 1.f;
    const bool exact_z = !p.sigmoid && (p.scores != nullptr || !p.renorm);
    if (!p.sigmoid && (!kByLogit || exact_z)) {
      m = row_max<V>(l);
      if (!kByLogit) z_fast = row_sum<V, true>(l, m);
      if (exact_z) z = row_sum<V, false>(l, m);
    }
    if (p.scores != nullptr) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (expert_of<V, kBlocked>(j) < p.E)
          p.scores[t * p.E + expert_of<V, kBlocked>(j)] = score_of<float>(l[j], p.sigmoid, m, z);
    }
    float c[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
      c[j] = kByLogit ? l[j]
                      : select_score(score_fast(l[j], p.sigmoid, m, z_fast), l[j], bias[j]);

    int pick = -1, next = kNone;
    float lo = INFINITY, hi = -INFINITY;  // as in choose()
    float rest = -INFINITY;               // no score left over is above this
    bool unsure = nan;
    const bool packed = !nan && (!kGroups || lanes_per_group);
    if (packed) {
      bool in = true;  // this lane's group stays
      if (kGroups) {
        float a = -INFINITY, b = -INFINITY;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          b = fmaxf(b, fminf(a, c[j]));
          a = fmaxf(a, c[j]);
        }
        for (int o = per >> 1; o > 0; o >>= 1) {
          const float a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
          b = fmaxf(fmaxf(b, b2), fminf(a, a2));
          a = fmaxf(a, a2);
        }
        const float gs = (p.group_top == 2 && b != -INFINITY) ? a + b : a;
        uint32_t word = (order_key(gs) & ~31u) | (uint32_t)(31 - lane / per);
        uint32_t last = 0u;
        in = false;
        for (int i = 0; i < p.top_groups; ++i) {
          last = __reduce_max_sync(kFull, word);
          if (word == last) {
            in = true;
            lo = gs;
            word = 0u;
          }
        }
        const uint32_t left = __reduce_max_sync(kFull, word);
        if (left != 0u) {
          // the worst kept group and the most a dropped one can have; equal in
          // what the packed word keeps: undecided
          const uint32_t none = order_key(-INFINITY) & ~31u;
          unsure |= (left & ~31u) == (last & ~31u) && (last & ~31u) != none;
          hi = (left & ~31u) == none ? -INFINITY : key_value(left | 31u);
          const uint32_t lk = __reduce_min_sync(kFull, in ? order_key(gs) : 0xffffffffu);
          lo = key_value(lk);
        }
      }
      uint32_t w[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t e = (uint32_t)expert_of<V, kBlocked>(j);
        w[j] = (in && (kBlocked || e < (uint32_t)p.E))
                   ? (order_key(c[j]) & ~p.low) | (p.low - e) : 0u;
      }
      uint32_t left;
      const uint32_t mine = choose_packed<V>(w, p.k, left);
      pick = lane < p.k ? (int)(p.low - (mine & p.low)) : -1;
      uint32_t after = __shfl_down_sync(kFull, mine, 1);
      if (lane == p.k - 1) after = left;
      // do neighbours differ in what the words keep?  Those at -inf are all
      // empty slots, whichever they are.
      if (!(kByLogit && kBf16) && lane < p.k && (mine & ~p.low) == (after & ~p.low) &&
          after != 0u && (mine & ~p.low) != (order_key(-INFINITY) & ~p.low)) {
        // inside the order: equal logits with equal biases are in the right
        // order already; at its end a third value could hide
        bool tie = false;
        if (lane < p.k - 1) {
          const int ea = (int)(p.low - (after & p.low));
          tie = load_logit<kBf16>(p.logits, t * p.E + pick) ==
                load_logit<kBf16>(p.logits, t * p.E + ea);
          if (!kByLogit && p.bias != nullptr)
            tie = tie && __ldg(p.bias + pick) == __ldg(p.bias + ea);
        }
        unsure |= !tie;
      }
      if (left != 0u) {
        next = (int)(p.low - (left & p.low));
        rest = key_value(left | p.low);
      }
    } else if (!nan) {
      pick = choose<V, kBlocked, float>(c, p, row32, next, lo, hi);
    }
    if (!kByLogit && !nan) {
      // Is every decision outside the error of c?  Lane i < k compares slot i
      // with slot i + 1, the last slot with what is left over.
      auto score_at = [&](int e, float &le, float &be, float &se, float &ce) {
        le = -INFINITY;
        be = 0.f;
        se = 0.f;
        ce = -INFINITY;
        if (e >= 0 && e < p.E) {
          le = load_logit<kBf16>(p.logits, t * p.E + e);
          if (p.bias != nullptr) be = __ldg(p.bias + e);
          se = score_fast(le, p.sigmoid, m, z_fast);
          ce = select_score(se, le, be);
        }
      };
      float l0, b0, s0, c0, l1, b1, s1, c1;
      score_at(pick, l0, b0, s0, c0);
      l1 = __shfl_down_sync(kFull, l0, 1);
      b1 = __shfl_down_sync(kFull, b0, 1);
      s1 = __shfl_down_sync(kFull, s0, 1);
      c1 = __shfl_down_sync(kFull, c0, 1);
      bool tie = l0 == l1 && b0 == b1;
      if (lane == p.k - 1) {
        score_at(next, l1, b1, s1, c1);
        // every score left over is within the packed word's resolution of this
        // one: the bound on the largest, with the largest possible s
        tie = !packed && l0 == l1 && b0 == b1;
        if (packed) {
          c1 = rest;
          s1 = p.sigmoid ? 1.f : (z_fast > 0.f ? __fdividef(1.f, z_fast) : 0.f);
        }
      }
      if (lane < p.k && c0 > -INFINITY && c1 > -INFINITY && !tie)
        unsure |= c0 - c1 <= score_error(s0, c0, p.sigmoid) + score_error(s1, c1, p.sigmoid);
      if (kGroups && lo > -INFINITY && hi > -INFINITY && lo < INFINITY) {
        // a group's score sums at most two, each at most the largest score
        const float s = p.sigmoid ? 1.f : (z_fast > 0.f ? __fdividef(1.f, z_fast) : 0.f);
        unsure |= lo - hi <= 2.f * (score_error(s, lo, p.sigmoid) + score_error(s, hi, p.sigmoid)) +
                                 4.f * kUlp * (fabsf(lo) + fabsf(hi));
      }
    }
    if (__any_sync(kFull, unsure)) {
      if constexpr (kByLogit) {
        pick = choose<V, kBlocked, float>(c, p, row32, next, lo, hi);
      } else {
        double z64 = 1.0, lo64, hi64;
        if (!p.sigmoid) {
          z64 = 0.0;
          if (m != -INFINITY) {
#pragma unroll 1
            for (int j = 0; j < V; ++j) {
              const int e = expert_of<V, kBlocked>(j);
              if (e < p.E)
                z64 += exp((double)load_logit<kBf16>(p.logits, t * p.E + e) - (double)m);
            }
            z64 = warp_add(z64);
          }
        }
        double c64[V];
#pragma unroll
        for (int j = 0; j < V; ++j)
          c64[j] = select_score(score_of<double>(l[j], p.sigmoid, m, z64), l[j], bias[j]);
        pick = choose<V, kBlocked, double>(c64, p, row64, next, lo64, hi64);
      }
    }
    // weights: lane i < k has slot i
    const bool slot = lane < p.k;
    float lp = -INFINITY;
    if (slot && pick >= 0 && pick < p.E) {
      lp = load_logit<kBf16>(p.logits, t * p.E + pick);
      if (!kByLogit && p.bias != nullptr && __ldg(p.bias + pick) == -INFINITY) lp = -INFINITY;
    }
    const bool empty = lp == -INFINITY;
    float w;
    if (p.renorm && !p.sigmoid) {
      // s_i / sum s: the row's sum cancels; the largest chosen logit in its
      // place, so that nothing underflows
      const uint32_t key = __reduce_max_sync(kFull, empty ? 0u : order_key(lp));
      w = empty ? 0.f : expf(lp - key_value(key));
    } else {
      w = empty ? 0.f : score_of<float>(lp, p.sigmoid, m, z);
    }
    if (p.renorm) {
      const float sum = warp_add(slot ? w : 0.f);
      w = sum == 0.f ? 0.f : w / sum;
    }
    if (slot) {
      // a NaN anywhere makes the softmax, and with it every weight, NaN
      p.experts[t * p.k + lane] = empty ? -1 : pick;
      p.weights[t * p.k + lane] =
          empty ? 0.f : (nan && !p.sigmoid ? __int_as_float(0x7fc00000) : w * p.scale);
    }
  }
}

struct RouteBwdParams {
  const void *logits;
  const int32_t *experts;
  const float *dweights, *dscores;
  void *dlogits;
  int64_t T;
  int E, k;
  bool sigmoid, renorm;
  float scale;
};

template <bool kBf16>
__device__ __forceinline__ void store_grad(void *p, int64_t i, float g) {
  if (kBf16)
    static_cast<uint16_t *>(p)[i] = f32_to_bf16_bits(g);
  else
    static_cast<float *>(p)[i] = g;
}

// This lane's V gradients of row t.
template <bool kBf16, int V, bool kBlocked>
__device__ __forceinline__ void store_row(void *out, int64_t t, int E, const float (&g)[V]) {
  const int lane = threadIdx.x & 31;
  if constexpr (kBlocked) {
    constexpr int kBytes = V * (kBf16 ? 2 : 4);
    uint32_t raw[kBytes / 4];
#pragma unroll
    for (int i = 0; i < kBytes / 4; ++i)
      raw[i] = kBf16 ? (uint32_t)f32_to_bf16_bits(g[kBf16 ? 2 * i : i]) |
                           ((uint32_t)f32_to_bf16_bits(g[kBf16 ? 2 * i + 1 : i]) << 16)
                     : __float_as_uint(g[kBf16 ? 0 : i]);
    char *dst = static_cast<char *>(out) + (t * 32 + lane) * kBytes;
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4 *>(dst)[i] =
            make_uint4(raw[4 * i], raw[4 * i + 1], raw[4 * i + 2], raw[4 * i + 3]);
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2 *>(dst) = make_uint2(raw[0], raw[1]);
    } else {
      *reinterpret_cast<uint32_t *>(dst) = raw[0];
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane + 32 * j < E) store_grad<kBf16>(out, t * E + lane + 32 * j, g[j]);
  }
}

// One warp per row: the row's dense part (zero without one) in whole rows,
// then, after a warp barrier that orders the two, the chosen experts' full
// gradients over it, lane i slot i's.
// kDense: every score of the row is needed (softmax without renormalisation,
// or a dscores).  Otherwise the gradient outside the chosen experts is 0: for
// the renormalised softmax sum_e s_e ds_e = scale (sum_i dw_i n_i -
// sum_j dw_j n_j sum_i n_i) / D = 0, and s_i / D needs the chosen logits only.
template <bool kBf16, int V, bool kBlocked, bool kDense>
__global__ void __launch_bounds__(32 * kWarps) k_route_bwd(const RouteBwdParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t stride = (int64_t)gridDim.x * kWarps;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < p.T; t += stride) {
    // lane i < k: slot i
    int e = -1;
    float le = -INFINITY, dw = 0.f;
    if (lane < p.k) {
      e = p.experts[t * p.k + lane];
      dw = p.dweights[t * p.k + lane];
      if (e < 0 || e >= p.E) e = -1;
    }
    float l[kDense ? V : 1], ds[kDense ? V : 1];
    if constexpr (kDense) {
      load_row<kBf16, V, kBlocked>(p.logits, t, p.E, l);
      if (p.dscores != nullptr)
        load_row<false, V, kBlocked>(p.dscores, t, p.E, ds);
      else
#pragma unroll
        for (int j = 0; j < V; ++j) ds[j] = 0.f;
    }
    if (e >= 0) le = load_logit<kBf16>(p.logits, t * p.E + e);
    const bool dense = kDense;
    float m = 0.f, z = 1.f;
    if (!p.sigmoid) {
      if constexpr (kDense) {
        m = row_max<V>(l);
        z = row_sum<V, false>(l, m);
      } else {
        // only the ratio to the chosen experts' sum matters
        const uint32_t key = __reduce_max_sync(kFull, e >= 0 ? order_key(le) : 0u);
        m = key == 0u ? le : key_value(key);
        if (m == -INFINITY) z = 0.f;
      }
    }
    const float s = e >= 0 ? score_of<float>(le, p.sigmoid, m, z) : 0.f;
    float d = p.scale * dw;
    if (p.renorm) {
      const float sum = warp_add(s);
      const float mean = sum == 0.f ? 0.f : warp_add(dw * s) / sum;
      d = sum == 0.f ? 0.f : p.scale * (dw - mean) / sum;
    }
    if (e < 0) d = 0.f;
    float dot = 0.f;
    if (kDense && !p.sigmoid) dot = s * d;
    // the same expert in two slots: the first of them takes the sum
    bool first = e >= 0;
    const uint32_t same = __match_any_sync(kFull, e >= 0 ? e : -1 - lane);
    if (__any_sync(kFull, __popc(same) > 1)) {
      float sum = 0.f;
      for (int i = 0; i < p.k; ++i) {
        const float di = __shfl_sync(kFull, d, i);
        if ((same >> i) & 1u) sum += di;
      }
      d = sum;
      first = first && __ffs(same) - 1 == lane;
    }
    float g[V];
    if constexpr (kDense) {
      if (!p.sigmoid) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          l[j] = score_of<float>(l[j], false, m, z);
          // values past E have the score 0; their ds must not be -inf
          if (!kBlocked && expert_of<V, kBlocked>(j) >= p.E) ds[j] = 0.f;
          dot += l[j] * ds[j];
        }
        dot = warp_add(dot);
#pragma unroll
        for (int j = 0; j < V; ++j) g[j] = l[j] * (ds[j] - dot);
      } else {
        // 1 - sigma(l) = sigma(-l), without the cancellation
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float x = expf(-fabsf(l[j])), q = 1.f / (1.f + x);
          g[j] = ds[j] * (x * q) * q;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) g[j] = 0.f;
    }
    store_row<kBf16, V, kBlocked>(p.dlogits, t, p.E, g);
    __syncwarp();
    if (first) {
      const float all = d + ((dense && p.dscores != nullptr) ? __ldg(p.dscores + t * p.E + e) : 0.f);
      float ge;
      if (p.sigmoid) {
        const float x = expf(-fabsf(le)), q = 1.f / (1.f + x);
        ge = all * (x * q) * q;
      } else {
        ge = s * (all - dot);
      }
      store_grad<kBf16>(p.dlogits, t * p.E + e, ge);
    }
  }
}

int route_grid(int64_t T, int num_sms) {
  const int64_t blocks = (T + kWarps - 1) / kWarps;
  const int64_t most = (int64_t)num_sms * 16;
  return (int)(blocks < most ? blocks : most);
}

// f(V, blocked) with the smallest built V with 32 V >= E; blocked: the rows
// are exactly 32 V long and their 16-byte pieces aligned.
template <class F>
cudaError_t with_layout(int E, bool aligned, F &&f) {
  auto with_v = [&](auto v) {
    constexpr int V = decltype(v)::value;
    if constexpr (V > 1)
      if (E == 32 * V && aligned) return f(v, std::true_type{});
    return f(v, std::false_type{});
  };
  if (E <= 32) return with_v(std::integral_constant<int, 1>{});
  if (E <= 64) return with_v(std::integral_constant<int, 2>{});
  if (E <= 128) return with_v(std::integral_constant<int, 4>{});
  if (E <= 256) return with_v(std::integral_constant<int, 8>{});
  if (E <= 512) return with_v(std::integral_constant<int, 16>{});
  return with_v(std::integral_constant<int, 32>{});
}

bool aligned16(std::initializer_list<const void *> ps) {
  for (const void *p : ps)
    if ((uintptr_t)p % 16 != 0) return false;
  return true;
}

// The kernel's grid: blocks of kWarps rows, at most what the SMs hold at once.
template <class P>
cudaError_t launch_rows(void (*kern)(P), int64_t T, size_t smem, int num_sms, cudaStream_t st,
                        const P &p) {
  count_launches(1);
  return launch_pdl(kern, dim3(route_grid(T, num_sms)), dim3(32 * kWarps), smem, st, p);
}

}  // namespace

cudaError_t launch_route(const RouteShape &s, const void *logits, const float *bias,
                         int32_t *experts, float *weights, float *scores, int num_sms,
                         cudaStream_t st) {
  RouteParams p{logits, bias, experts, weights, scores, s.T, s.E, s.k, s.groups,
                s.E / s.groups, s.top_groups, s.group_top, s.sigmoid, s.renorm, s.scale, 1u};
  while (p.low + 1 < (uint32_t)s.E) p.low = 2 * p.low + 1;  // index bits of a packed word
  const bool by_logit = bias == nullptr && (s.groups == 1 || s.group_top == 1);
  const bool groups = s.groups > 1;
  const size_t smem = groups ? (size_t)kWarps * s.E * sizeof(double) : 0;
  return with_layout(s.E, aligned16({logits}), [&](auto v, auto blocked) {
    constexpr int V = decltype(v)::value;
    constexpr bool kB = decltype(blocked)::value;
    auto go = [&](auto bf16, auto logit, auto grouped) {
      return launch_rows(k_route<decltype(bf16)::value, V, kB, decltype(logit)::value,
                                 decltype(grouped)::value>, s.T, smem, num_sms, st, p);
    };
    auto with_groups = [&](auto bf16, auto logit) {
      return groups ? go(bf16, logit, std::true_type{}) : go(bf16, logit, std::false_type{});
    };
    auto with_rank = [&](auto bf16) {
      return by_logit ? with_groups(bf16, std::true_type{}) : with_groups(bf16, std::false_type{});
    };
    return s.bf16 ? with_rank(std::true_type{}) : with_rank(std::false_type{});
  });
}

cudaError_t launch_route_backward(const RouteShape &s, const void *logits,
                                  const int32_t *experts, const float *dweights,
                                  const float *dscores, void *dlogits, int num_sms,
                                  cudaStream_t st) {
  const RouteBwdParams p{logits, experts, dweights, dscores, dlogits, s.T,
                         s.E,    s.k,     s.sigmoid, s.renorm, s.scale};
  const bool dense = dscores != nullptr || (!s.sigmoid && !s.renorm);
  return with_layout(s.E, aligned16({logits, dscores, dlogits}), [&](auto v, auto blocked) {
    constexpr int V = decltype(v)::value;
    constexpr bool kB = decltype(blocked)::value;
    auto go = [&](auto bf16, auto all) {
      return launch_rows(k_route_bwd<decltype(bf16)::value, V, kB, decltype(all)::value>, s.T, 0,
                         num_sms, st, p);
    };
    auto with_all = [&](auto bf16) {
      return dense ? go(bf16, std::true_type{}) : go(bf16, std::false_type{});
    };
    return s.bf16 ? with_all(std::true_type{}) : with_all(std::false_type{});
  });
}

}  // namespace sfn
