// route.cuh -- routing of tokens to experts: scores, balance biases, groups,
// top-k and its weights.  The kernels; route_f32.cu, route_bf16.cu and
// route_lanes.cu build them, route_backward.cu the gradient's, route.cu chooses.
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
// the ranking of l and is done on l itself (groups by their two largest: on c).
// With one, c is computed in float32 and every decision the row took (between
// neighbours in the order, at the k-th place, between groups) is checked against
// a bound on the error of c; what is inside the bound is decided again in float64.
//
// One warp per row, V = E / 32 (rounded up to a built one) values a lane.
// With whole keys instruction issue bounded it; the picks run on packed keys: the
// score's order key with the value's place in its lane in the low bits, one
// 32-bit word.  A lane sorts its V words once (a register network); a pick is
// then one warp maximum (redux) over the lanes' heads, and the lane that had it
// moves its list up.  The low bits cost the key some of its mantissa: the slots
// are put in order by their whole scores afterwards, and only a row whose k-th
// place the words cannot tell from the rest goes to the exact routine
// (settle_row()), which compares whole keys.  bf16 logits fit beside the whole
// index and are always exact.  Rows of exactly 32 V experts are loaded V
// neighbours a lane (16-byte loads), and groups of a whole number of lanes
// find their two largest scores with shuffles; others go through settle_row().
// What the rare paths cost is their latency, at the end of a launch: each
// level (words, whole scores, float64 of the slots and the next two, float64 of
// the row) is there so that few rows see the next.
//   4096 x 256, 8 groups: 10.7 us (of it 3 us of rows decided in float64); 22.5
//   us with whole keys alone, 20.9 us with float64 rows in place of float64 slots
//   32768 x 160, bf16, k 6: 18.4 us, 11.7 us with eight lanes a row
//   (route_lanes.cu); 38.9 us with whole keys
#pragma once

#include <cmath>
#include <initializer_list>
#include <type_traits>

#include "async_util.cuh"
#include "experts.cuh"

namespace sfn {

struct RouteParams {
  const void *logits;
  const float *bias;
  int32_t *experts;
  float *weights;
  float *scores;
  int64_t T;
  int E, k, groups, group_size, top_groups, group_top;
  bool sigmoid, renorm, bf16;
  float scale;
  uint32_t low;  // the bits of a packed word that hold the index
};

// The launchers of one type, and the two ways of taking the rows.
template <bool kBf16>
cudaError_t launch_route_warps(const RouteParams &p, bool by_logit, int num_sms, cudaStream_t st);
template <bool kBf16>
cudaError_t launch_route_lanes(const RouteParams &p, bool by_logit, int num_sms, cudaStream_t st);

namespace {


constexpr int kWarps = 4;  // rows in flight per block
constexpr int kNone = 0x7fffffff;


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

// A chosen expert's share in the renormalised weights, up to a factor that all of
// the row's shares have: exp(-m) s with m the row's largest chosen logit `top`
// (softmax; its sum over the row cancels) or the smaller of it and 0 (sigmoid), so
// that the shares of scores below float32's range are not lost.  The largest share
// is at least 1/2.
__device__ __forceinline__ float share_of(float l, bool sigmoid, float top) {
  if (!sigmoid) return expf(l - top);
  const float m = fminf(top, 0.f);
  return 1.f / (expf(m) + expf(m - l));
}
// Are the chosen scores 0, as float64 gives them?  (m: the row's largest logit;
// softmax only.)  Then the weights are, as masks of a type's lowest value mean it.
__device__ __forceinline__ bool shares_vanish(bool sigmoid, float top, float m) {
  return sigmoid ? top < -709.7827f : top == -INFINITY || top - m < -745.1332f;
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
// experts (those past E are never looked at): groups by c, the experts of those
// that stay by c too or, by_l, by their logits l.  Lane i returns slot i's
// expert.  `next`: the best expert left over (kNone: none).  gap_lo and
// gap_hi: the worst score of a kept group and the best of a dropped one.
template <int V, bool kBlocked, class R>
__device__ __noinline__ int choose(const R (&c)[V], const float (&l)[V], bool by_l,
                                   const RouteParams &p, R *row_smem, int &next, R &gap_lo,
                                   R &gap_hi) {
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
  for (int j = 0; j < V; ++j) key[j] = key_of(by_l ? (R)l[j] : c[j]);
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

template <int V>
__device__ __forceinline__ void sort_descending(uint32_t (&w)[V]) {
  // Batcher's odd-even merge sort, for any V; all indices are constants
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p))
            cex_desc(w[i + j], w[i + j + q]);
}
// The same choice on packed words, unique in a lane, 0 for a value that is
// out.  Lane i returns slot i's word and, in `winner`, the lane that had it
// (of equal words the lowest); `next` is the best word left over.
// kUnique: no two lanes have the same word.  w: sorted, and what is left of it
// afterwards; slots [k0, k) are filled.
template <int V, bool kUnique>
__device__ __forceinline__ void pick_packed(uint32_t (&w)[V], int k0, int k, uint32_t &mine,
                                            int &winner) {
  const int lane = threadIdx.x & 31;
  for (int i = k0; i < k; ++i) {
    const uint32_t top = __reduce_max_sync(kFull, w[0]);
    bool won = w[0] == top;
    if constexpr (!kUnique) {
      const int at = __ffs(__ballot_sync(kFull, won)) - 1;
      won = lane == at;
      if (lane == i) winner = at;
    }
    if (lane == i) mine = top;
    if (won) {
#pragma unroll
      for (int j = 0; j + 1 < V; ++j) w[j] = w[j + 1];
      w[V - 1] = 0u;
    }
  }
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
// Decisions are tested as !(difference > bound), so that what is no number counts
// as undecided: the difference of two infinities (of biases, of a sum of two that
// passed the range), and the bound that a packed word of +inf gives, whose place
// bits make it a NaN.
constexpr float kUlp = 5.9604645e-8f;
__device__ __forceinline__ float score_error(float s, float c, bool sigmoid) {
  return kUlp * ((sigmoid ? 0.f : 80.f * s) + 8.f + fabsf(c));
}
__device__ __forceinline__ float score_fast(float l, bool sigmoid, float m, float z) {
  if (sigmoid) return __fdividef(1.f, 1.f + __expf(-l));
  return z == 0.f ? 0.f : __fdividef(__expf(l - m), z);
}

// This lane's V logits of row t (-inf past E).
// A lane's part of a blocked row is a vector load.
template <int V>
constexpr bool vector_part() {
  return (V & (V - 1)) == 0;
}
template <bool kBf16, int V, bool kBlocked, int kLanes = 32>
__device__ __forceinline__ void load_row(const void *logits, int64_t t, int E, float (&l)[V]) {
  const int lane = threadIdx.x % kLanes;
  if constexpr (kBlocked && !vector_part<V>()) {
#pragma unroll
    for (int j = 0; j < V; ++j) l[j] = load_logit<kBf16>(logits, t * E + lane * V + j);
  } else if constexpr (kBlocked) {
    constexpr int kBytes = V * (kBf16 ? 2 : 4);
    uint32_t raw[kBytes / 4];
    const char *src = static_cast<const char *>(logits) + (t * kLanes + lane) * kBytes;
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
      const int e = lane + kLanes * j;
      l[j] = e < E ? load_logit<kBf16>(logits, t * E + e) : -INFINITY;
    }
  }
}

// Maximum over the row (nan: it has a NaN, and so is the maximum) and, given it,
// the sum of exponentials.
template <int V>
__device__ __forceinline__ float row_max(const float (&l)[V], bool nan) {
  float m = l[0];
#pragma unroll
  for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
  const uint32_t key = __reduce_max_sync(kFull, order_key(m));
  return nan ? __int_as_float(0x7fc00000) : key_value(key);
}
template <int V>
__device__ __forceinline__ bool row_has_nan(const float (&l)[V]) {
  bool nan = false;
#pragma unroll
  for (int j = 0; j < V; ++j) nan |= l[j] != l[j];
  return __any_sync(kFull, nan);
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

// Blocks of kWarps rows an SM holds at once (the launch bound and the grid): as
// many as the registers allow without spills on the usual path; the kernels that
// rank by logit need fewer of them.  us, k 8.  By score, 7 blocks (V <= 4) or 5 (V <=
// 8) against 8 or 7: 128 experts, 512 / 4096 / 8192 rows 3.9 / 7.1 / 10.1 against 4.3 /
// 7.5 / 10.6; 256 4.4 / 9.0 / 13.9 against 5.0 / 9.3 / 13.9; 256 in 8 groups, 512 / 4096 /
// 32768 rows 5.0 / 10.7 / 52.1 against 5.9 / 11.7 / 58.8.  By logit, 7 against 5: 192
// in 8 groups 3.9 / 6.9 / 34.0 against 3.9 / 7.2 / 39.5.
template <int V, bool kByLogit>
constexpr int route_blocks() {
  if (kByLogit) return V <= 4 ? 8 : (V <= 8 ? 7 : (V <= 16 ? 4 : 2));
  return V <= 4 ? 7 : (V <= 8 ? 5 : (V <= 16 ? 4 : 2));
}

// Mask of a value's place among a lane's V, in the low bits of a packed word.
template <int V>
constexpr uint32_t places() {
  return V <= 1 ? 0u : V <= 2 ? 1u : V <= 4 ? 3u : V <= 8 ? 7u : V <= 16 ? 15u : 31u;
}

// As route_blocks(), of the kernels with eight lanes a row.  By score five of V <=
// 16 against seven and eight: 16384 / 32768 rows of 64 experts 11.8 / 15.3 us against
// 12.7 / 17.9, of 128 13.6 / 21.3 against 16.0 / 25.6; four of more values against
// three: of 256 20.3 / 34.2 against 22.4 / 36.1.  By logit eight and seven against six
// and five: 8192 / 32768 rows of 64 4.6 / 9.7 us against 4.6 / 9.6, of 128 5.1 / 12.0
// against 5.5 / 12.6, of 160 6.0 / 13.7 against 6.1 / 15.1, of 256 7.5 / 17.8 against
// 8.1 / 20.3.  The dense gradient: 64 4.4 / 8.8 against 4.5 / 10.0 (six), 128 6.5 /
// 14.1 against 7.0 / 15.6 (five), 256 with four 11.5 / 35.8 against 14.8 / 37.0 (three).
enum class Lanes { kByLogit, kByScore, kGradient };
template <int V, Lanes kKind>
constexpr int lanes_blocks() {
  if (kKind == Lanes::kByLogit) return V <= 8 ? 8 : 7;
  if (kKind == Lanes::kByScore) return V <= 16 ? 5 : 4;
  return V <= 8 ? 8 : (V <= 16 ? 7 : 4);
}

// Among a row's eight lanes.
constexpr int kRowLanes = 8;
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
  for (int o = 1; o < kRowLanes; o <<= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float lanes_add(float v) {
#pragma unroll
  for (int o = 1; o < kRowLanes; o <<= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Order key of a number (not NaN): as order_key(), in three instructions.
__device__ __forceinline__ uint32_t number_key(float f) {
  const int b = __float_as_int(f + 0.f);  // -0 -> +0
  return (uint32_t)(b ^ ((b >> 31) | (int)0x80000000));
}

// The choice of one row with whole keys, for rows that the packed words leave
// undecided and for groups that are no whole number of lanes: in float32 with
// every decision checked, and in float64 where one is inside the error bound.
// Lane i returns slot i's expert.
// Built once for both types and layouts and for powers of two: it is rare.
template <int V, bool kByLogit>
__device__ __noinline__ int settle_row(const RouteParams &p, int64_t t, double *row64) {
  const int lane = threadIdx.x & 31;
  float *row32 = reinterpret_cast<float *>(row64);
  float l[V];
  if (p.bf16)
    load_row<true, V, false>(p.logits, t, p.E, l);
  else
    load_row<false, V, false>(p.logits, t, p.E, l);
  auto logit = [&](int e) {
    return p.bf16 ? load_logit<true>(p.logits, t * p.E + e)
                  : load_logit<false>(p.logits, t * p.E + e);
  };
  int next;
  float lo, hi;
  if constexpr (kByLogit) {
    return choose<V, false, float>(l, l, true, p, row32, next, lo, hi);
  } else {
    const bool by_l = p.bias == nullptr;
    float bias[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = expert_of<V, false>(j);
      bias[j] = (p.bias != nullptr && e < p.E) ? __ldg(p.bias + e) : 0.f;
    }
    const bool nan = row_has_nan<V>(l);
    float m = 0.f, z = 1.f;
    if (!p.sigmoid) {
      m = row_max<V>(l, nan);
      z = row_sum<V, true>(l, m);
    }
    if (!nan) {
      float c[V];
#pragma unroll
      for (int j = 0; j < V; ++j)
        c[j] = select_score(score_fast(l[j], p.sigmoid, m, z), l[j], bias[j]);
      const int pick = choose<V, false, float>(c, l, by_l, p, row32, next, lo, hi);
      // Is every decision outside the error of c?  Lane i < k compares slot i
      // with slot i + 1, the last slot with the best left over.
      auto score_at = [&](int e, float &le, float &be, float &se, float &ce) {
        le = -INFINITY;
        be = 0.f;
        se = 0.f;
        ce = -INFINITY;
        if (e >= 0 && e < p.E) {
          le = logit(e);
          if (p.bias != nullptr) be = __ldg(p.bias + e);
          se = score_fast(le, p.sigmoid, m, z);
          ce = select_score(se, le, be);
        }
      };
      float l0, b0, s0, c0, l1, b1, s1, c1;
      score_at(pick, l0, b0, s0, c0);
      l1 = __shfl_down_sync(kFull, l0, 1);
      b1 = __shfl_down_sync(kFull, b0, 1);
      s1 = __shfl_down_sync(kFull, s0, 1);
      c1 = __shfl_down_sync(kFull, c0, 1);
      if (lane == p.k - 1) score_at(next, l1, b1, s1, c1);
      // equal logits with equal biases are in the right order already
      const bool tie = l0 == l1 && b0 == b1;
      bool unsure = !by_l && lane < p.k && c0 > -INFINITY && c1 > -INFINITY && !tie &&
                    !(c0 - c1 > score_error(s0, c0, p.sigmoid) + score_error(s1, c1, p.sigmoid));
      // at the end of the order a third value could hide behind a tie
      if (!by_l && lane == p.k - 1 && tie && c1 > -INFINITY) unsure = true;
      if (lo > -INFINITY && hi > -INFINITY) {
        // a group's score sums at most two, each at most the largest score
        const float s = p.sigmoid ? 1.f : (z > 0.f ? __fdividef(1.f, z) : 0.f);
        unsure |= !(lo - hi > 2.f * (score_error(s, lo, p.sigmoid) +
                                     score_error(s, hi, p.sigmoid)) +
                                  4.f * kUlp * (fabsf(lo) + fabsf(hi)));
      }
      if (!__any_sync(kFull, unsure)) return pick;
    }
    double z64 = 1.0, lo64, hi64;
    if (!p.sigmoid) {
      z64 = 0.0;
      if (m != -INFINITY) {
#pragma unroll 1
        for (int j = 0; j < V; ++j) {
          const int e = expert_of<V, false>(j);
          if (e < p.E) z64 += exp((double)logit(e) - (double)m);
        }
        z64 = warp_add(z64);
      }
    }
    double c64[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
      c64[j] = select_score(score_of<double>(l[j], p.sigmoid, m, z64), l[j], bias[j]);
    return choose<V, false, double>(c64, l, by_l, p, row64, next, lo64, hi64);
  }
}

// The row's sum of exponentials in float64; rare.
template <bool kBf16>
__device__ __noinline__ double row_sum64(const void *logits, int64_t t, int E, float m) {
  double z = 0.0;
  if (m != -INFINITY)
    for (int e = threadIdx.x & 31; e < E; e += 32)
      z += exp((double)load_logit<kBf16>(logits, t * E + e) - (double)m);
  return warp_add(z);
}
// Does this lane's group stay?  In float64 (by logit: on the logits, exactly),
// for groups of `per` lanes with V neighbouring experts each; rare.
template <int V, bool kByLogit>
__device__ __noinline__ bool settle_groups(const RouteParams &p, int64_t t, const float (&c)[V],
                                           float m, int per) {
  const int lane = threadIdx.x & 31;
  const double z = p.sigmoid || kByLogit ? 1.0
                   : p.bf16              ? row_sum64<true>(p.logits, t, p.E, m)
                                         : row_sum64<false>(p.logits, t, p.E, m);
  const double none = -INFINITY;
  double a = none, b = none;
  auto offer = [&](int j) {
    const int e = lane * V + j;
    const float l = p.bf16 ? load_logit<true>(p.logits, t * p.E + e)
                           : load_logit<false>(p.logits, t * p.E + e);
    const float be = p.bias != nullptr ? __ldg(p.bias + e) : 0.f;
    const double c =
        kByLogit ? (double)l : select_score(score_of<double>(l, p.sigmoid, m, z), l, be);
    b = fmax(b, fmin(a, c));
    a = fmax(a, c);
  };
  // the lane's two largest by their float32 scores, unless a third comes close
  float c1 = -INFINITY, c2 = -INFINITY, c3 = -INFINITY;
  int j1 = 0, j2 = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (c[j] > c1) {
      c3 = c2;
      c2 = c1;
      j2 = j1;
      c1 = c[j];
      j1 = j;
    } else if (c[j] > c2) {
      c3 = c2;
      c2 = c[j];
      j2 = j;
    } else {
      c3 = fmaxf(c3, c[j]);
    }
  }
  const float most = p.sigmoid ? 1.f : (z > 0. ? (float)(1. / z) : 0.f);
  const bool third = V > 2 && c3 > -INFINITY &&
                     c2 - c3 <= score_error(most, c2, p.sigmoid) + score_error(most, c3, p.sigmoid);
  if (__any_sync(kFull, third)) {
    for (int j = 0; j < V; ++j) offer(j);
  } else {
    offer(j1);
    if (V > 1) offer(j2 != j1 ? j2 : (j1 + 1) % V);
  }
  for (int o = per >> 1; o > 0; o >>= 1) {
    const double a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
    b = fmax(fmax(b, b2), fmin(a, a2));
    a = fmax(a, a2);
  }
  const double gs = (p.group_top == 2 && b != none) ? a + b : a;
  int rank = 0;
  for (int h = 0; h < p.groups; ++h) {
    const double hs = __shfl_sync(kFull, gs, h * per);
    rank += (hs > gs) | ((hs == gs) & (h < lane / per));
  }
  return rank < p.top_groups;
}

// Does (score c1, expert e1) come before (c0, e0)?  Those at -inf are empty
// slots in any order.
template <class R>
__device__ __forceinline__ bool before(R c1, int e1, R c0, int e0) {
  return c0 < c1 || (c0 == c1 && e0 > e1 && c0 > (R)-INFINITY);
}
// Lanes [0, n) of each run of lanes that starts at `first` in order, by
// exchanges of neighbours (`sub`: this lane's number in its run); rare.
template <class R>
__device__ __noinline__ void exchange_sort(int n, int sub, int first, R &c, int &e, float &l,
                                           float &b) {
  for (int i = 0; i < n; ++i) {
    const int other = (i & 1) ? ((sub - 1) ^ 1) + 1 : sub ^ 1;
    const bool both = other >= 0 && other < n && sub < n;
    const int from = first + (both ? other : sub);
    const R c2 = __shfl_sync(kFull, c, from);
    const int e2 = __shfl_sync(kFull, e, from);
    const float l2 = __shfl_sync(kFull, l, from), b2 = __shfl_sync(kFull, b, from);
    if (both && (sub < other ? before(c2, e2, c, e) : before(c, e, c2, e2))) {
      c = c2;
      e = e2;
      l = l2;
      b = b2;
    }
  }
}

// The k experts of one row from this lane's V logits; lane i < k returns slot
// i's, with its logit and bias.  m, z: the softmax's maximum and sum (kByLogit:
// not used).  row64: E doubles of shared memory for this warp (kGroups).
// kByLogit: no bias, and groups (if any) scored by their largest: the logits
// themselves are ranked.  Else, without a bias (groups scored by their two
// largest), the groups are ranked by scores and their experts by logits.  kGroups:
// groups > 1.
template <bool kBf16, int V, bool kBlocked, bool kByLogit, bool kGroups>
__device__ __forceinline__ int select_row(const RouteParams &p, int64_t t, const float (&l)[V],
                                          const float (&bias)[kByLogit ? 1 : V], bool nan, float m,
                                          float z_fast, double *row64, float &lp, float &bp) {
  const int lane = threadIdx.x & 31;
  // groups of a whole number of lanes; then every lane of a group knows it
  const bool packed = !kGroups || (kBlocked && 32 % p.groups == 0);
  const int per = kGroups ? 32 / p.groups : 32;
  const uint32_t none = order_key(-INFINITY);
  // packed words: the order key with this value's place in its lane below it
  // (complemented: of equal keys the lower index is the larger word); for bf16
  // logits the whole index, which fits below their 16 bits
  constexpr bool kWhole = kByLogit && kBf16;
  constexpr uint32_t kPlaces = places<V>();
  const uint32_t low = kWhole ? p.low : kPlaces;
  const bool slot = lane < p.k;  // lane i < k has slot i
  int pick = -1;
  lp = -INFINITY;  // its logit and bias
  bp = 0.f;
  auto look_up = [&] {
    lp = -INFINITY;
    bp = 0.f;
    if (slot && pick >= 0 && pick < p.E) {
      lp = load_logit<kBf16>(p.logits, t * p.E + pick);
      if (!kByLogit && p.bias != nullptr) bp = __ldg(p.bias + pick);
    }
  };
  float c[V];
  bool number = true;  // the words have no room for a NaN (of l, of a bias, of exp(inf - inf))
#pragma unroll
  for (int j = 0; j < V; ++j) {
    c[j] = kByLogit ? l[j]
                    : select_score(score_fast(l[j], p.sigmoid, m, z_fast), l[j], bias[j]);
    if (!kByLogit) number &= c[j] == c[j];
  }
  bool unsure = nan || !packed || (!kByLogit && !__all_sync(kFull, number));
  if (!unsure) {
    // the largest score there can be, for the error bounds
    const float most = p.sigmoid || kByLogit ? 1.f : (z_fast > 0.f ? __fdividef(1.f, z_fast) : 0.f);
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
      uint32_t word = (number_key(gs) & ~31u) | (uint32_t)(31 - lane / per);
      uint32_t last = 0u;
      in = false;
      for (int i = 0; i < p.top_groups; ++i) {
        last = __reduce_max_sync(kFull, word);
        if (word == last) {
          in = true;
          word = 0u;
        }
      }
      const uint32_t left = __reduce_max_sync(kFull, word);
      if (left != 0u && (last & ~31u) != (none & ~31u) && (left & ~31u) != (none & ~31u)) {
        // may the worst kept group and the best dropped one have changed
        // places?  First by the words (32 units of the last place apart),
        // then by the whole scores.  A group's score sums at most two.
        auto close = [&](float lo, float hi) {
          return kByLogit ? !(lo > hi)
                          : !(lo - hi > 2.f * (score_error(most, lo, p.sigmoid) +
                                               score_error(most, hi, p.sigmoid)) +
                                            4.f * kUlp * (fabsf(lo) + fabsf(hi)));
        };
        if (close(key_value(last & ~31u), key_value(left | 31u))) {
          const uint32_t key = number_key(gs);
          const float lo = key_value(__reduce_min_sync(kFull, in ? key : 0xffffffffu));
          const float hi = key_value(__reduce_max_sync(kFull, in ? 0u : key));
          if (close(lo, hi)) in = settle_groups<V, kByLogit>(p, t, c, m, per);
        }
      }
    }
    // what ranks the experts of the groups that stay
    const bool by_l = kGroups && !kByLogit && p.bias == nullptr;
    if (by_l) {
#pragma unroll
      for (int j = 0; j < V; ++j) c[j] = l[j];
    }
    uint32_t w[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t e = (uint32_t)expert_of<V, kBlocked>(j);
      const uint32_t place = kWhole ? p.low - e : kPlaces - (uint32_t)j;
      w[j] = (in && (kBlocked || e < (uint32_t)p.E)) ? (number_key(c[j]) & ~low) | place : 0u;
    }
    uint32_t mine = 0u;
    int winner = 0;
    sort_descending<V>(w);
    pick_packed<V, kWhole>(w, 0, p.k, mine, winner);
    if constexpr (kWhole) {
      if (slot) {
        pick = (int)(p.low - (mine & p.low));
        const uint32_t kept = mine & ~low;
        // a bf16's key is all in the upper half (negative numbers: complemented)
        lp = __uint_as_float((kept & 0x80000000u) ? kept & 0x7fff0000u : ~kept & 0xffff0000u);
      }
    } else {
      auto expert_at = [&] {
        const int place = (int)(kPlaces - (mine & kPlaces));
        return kBlocked ? winner * V + place : winner + 32 * place;
      };
      if (slot) pick = expert_at();
      look_up();
      float cp = -INFINITY;  // the slot's selection score in full
      if (slot)
        cp = kByLogit || by_l ? lp
                              : select_score(score_fast(lp, p.sigmoid, m, z_fast), lp, bp);
      // neighbours whose words agree may be in the wrong order: exchange
      // them, by whole scores and then by index
      float c1 = __shfl_down_sync(kFull, cp, 1);
      const int e1 = __shfl_down_sync(kFull, pick, 1);
      if (__any_sync(kFull, lane < p.k - 1 && before(c1, e1, cp, pick))) {
        exchange_sort(p.k, lane, 0, cp, pick, lp, bp);
        c1 = __shfl_down_sync(kFull, cp, 1);
      }
      // the most that what is left over can have, against the last slot
      uint32_t left = __reduce_max_sync(kFull, w[0]);
      bool rest = left != 0u && (left & ~low) != (none & ~low);
      if constexpr (kByLogit) {
        unsure |= lane == p.k - 1 && rest && !(cp > key_value(left | low));
      } else {
        auto bound = [&](float c) { return by_l ? 0.f : score_error(most, c, p.sigmoid); };
        const float l1 = __shfl_down_sync(kFull, lp, 1), b1 = __shfl_down_sync(kFull, bp, 1);
        bool close = false;
        if (slot && cp > -INFINITY) {
          if (lane == p.k - 1) {
            const float hi = key_value(left | low);
            close = rest && !(cp - hi > bound(cp) + bound(hi));
          } else {  // equal logits with equal biases are in the right order
            close = c1 > -INFINITY && !(lp == l1 && bp == b1) &&
                    !(cp - c1 > bound(cp) + bound(c1));
          }
        }
        if (!__any_sync(kFull, unsure) && __any_sync(kFull, close)) {
          // inside the error of float32: the slots and the next two, in
          // float64, and the order again; undecided only if what is left
          // over is that close too
          const int kx = min(p.k + 2, 32);
          pick_packed<V, false>(w, p.k, kx, mine, winner);
          left = __reduce_max_sync(kFull, w[0]);
          rest = left != 0u && (left & ~low) != (none & ~low);
          const bool more = lane >= p.k && lane < kx && mine != 0u;
          if (more) {
            pick = expert_at();
            lp = load_logit<kBf16>(p.logits, t * p.E + pick);
            if (p.bias != nullptr) bp = __ldg(p.bias + pick);
          }
          const double z64 =
              p.sigmoid || by_l ? 1.0 : row_sum64<kBf16>(p.logits, t, p.E, m);
          double c64 = -INFINITY;
          if (slot || more)
            c64 = by_l ? (double)lp
                       : select_score(score_of<double>(lp, p.sigmoid, m, z64), lp, bp);
          const double c64_1 = __shfl_down_sync(kFull, c64, 1);
          const int e64_1 = __shfl_down_sync(kFull, pick, 1);
          if (__any_sync(kFull, lane < kx - 1 && before(c64_1, e64_1, c64, pick)))
            exchange_sort(kx, lane, 0, c64, pick, lp, bp);
          const double last = __shfl_sync(kFull, c64, p.k - 1);
          const float hi = key_value(left | low);
          unsure = rest && !((float)last - hi > bound(hi) + (by_l ? 0.f : 2.f * kUlp * fabsf(hi)));
        }
      }
    }
  }
  if (__any_sync(kFull, unsure)) {
    constexpr int kPow2 = (int)kPlaces + 1;
    pick = settle_row<kPow2, kByLogit>(p, t, row64);
    look_up();
  }
  return pick;
}


// f(V, blocked) with the smallest built V with 32 V >= E; blocked (V
// neighbours a lane): the rows are exactly 32 V long, and a lane's part is an
// aligned vector load or groups need their experts side by side.
template <class F>
cudaError_t with_layout(int E, bool aligned, bool groups, F &&f) {
  auto with_v = [&](auto v) {
    constexpr int V = decltype(v)::value;
    if constexpr (V > 1)
      if (E == 32 * V && (vector_part<V>() ? aligned : groups)) return f(v, std::true_type{});
    return f(v, std::false_type{});
  };
  if (E <= 32) return with_v(std::integral_constant<int, 1>{});
  if (E <= 64) return with_v(std::integral_constant<int, 2>{});
  if (E <= 128) return with_v(std::integral_constant<int, 4>{});
  if (E <= 160) return with_v(std::integral_constant<int, 5>{});
  if (E <= 192) return with_v(std::integral_constant<int, 6>{});
  if (E <= 256) return with_v(std::integral_constant<int, 8>{});
  if (E <= 384) return with_v(std::integral_constant<int, 12>{});
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
cudaError_t launch_rows(void (*kern)(P), int64_t T, int blocks_per_sm, size_t smem, int num_sms,
                        cudaStream_t st, const P &p) {
  const int64_t blocks = (T + kWarps - 1) / kWarps, most = (int64_t)num_sms * blocks_per_sm;
  count_launches(1);
  return launch_pdl(kern, dim3((unsigned)(blocks < most ? blocks : most)), dim3(32 * kWarps), smem,
                    st, p);
}

}  // namespace
}  // namespace sfn
