// route_backward.cu -- the gradient of routing (route.cuh).
//
// Through the scores: with ds a dense gradient of them (a balance loss), plus
// scale dw_i on the chosen experts where the weights are not renormalised,
//   softmax: dl = s (ds - sum_e s_e ds_e);  sigmoid: dl = s (1 - s) ds
// Renormalised weights: with the shares n_i = s_i / sum_j s_j (share_of()) the
// chosen logits' gradients are, on top of that,
//   v_i = scale n_i (dw_i - sum_j n_j dw_j), with sigmoid scores times 1 - s_i
// (with softmax the sum over the row of s ds is 0 for this part).  So formed, it
// does not depend on how small the chosen scores are in the row: through ds_i =
// v_i / s_i it would pass float32's range where they are 90 below the largest.
#include "route.cuh"

namespace sfn {
namespace {

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

__device__ __forceinline__ uint32_t pack_bf16x2(float lower, float upper) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(upper), "f"(lower));
  return r;
}

// This lane's V gradients of row t.
template <bool kBf16, int V, bool kBlocked, int kLanes = 32>
__device__ __forceinline__ void store_row(void *out, int64_t t, int E, const float (&g)[V]) {
  const int lane = threadIdx.x % kLanes;
  if constexpr (kBlocked) {
    constexpr int kBytes = V * (kBf16 ? 2 : 4);
    uint32_t raw[kBytes / 4];
#pragma unroll
    for (int i = 0; i < kBytes / 4; ++i)
      raw[i] = kBf16 ? pack_bf16x2(g[kBf16 ? 2 * i : i], g[kBf16 ? 2 * i + 1 : i])
                     : __float_as_uint(g[kBf16 ? 0 : i]);
    char *dst = static_cast<char *>(out) + (t * kLanes + lane) * kBytes;
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
      if (lane + kLanes * j < E) store_grad<kBf16>(out, t * E + lane + kLanes * j, g[j]);
  }
}

// s (1 - s) of a sigmoid score: 1 - sigma(l) = sigma(-l), without the cancellation.
__device__ __forceinline__ float slope(float l) {
  const float x = expf(-fabsf(l)), q = 1.f / (1.f + x);
  return (x * q) * q;
}

// Blocks of kWarps rows an SM holds at once.
template <int V>
constexpr int backward_blocks() {
  return V <= 4 ? 10 : (V <= 8 ? 6 : (V <= 16 ? 4 : 2));
}

// What of a row's logits the gradient needs.
// kDense: every score (softmax without renormalisation, or a dscores): the
// slots' parts are added to the lanes' values in slot order, and the row is
// written once.  Otherwise the gradient outside the chosen experts is 0 and
// theirs needs their shares only; the row is written as zeros and, after a warp
// barrier that orders the two, the chosen experts' gradients over it, lane i slot
// i's.
// kRow (softmax): the largest, and whether one is NaN or +inf: then the row's
// scores, weights and gradients are NaN.
// kChosen (sigmoid): the chosen ones.
enum class Needs { kChosen, kRow, kDense };

// One warp per row.
template <bool kBf16, int V, bool kBlocked, Needs kNeeds>
__global__ void __launch_bounds__(32 * kWarps, backward_blocks<V>())
    k_route_bwd(const RouteBwdParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t stride = (int64_t)gridDim.x * kWarps;
  constexpr bool kDense = kNeeds == Needs::kDense, kLogits = kNeeds != Needs::kChosen;
  // the next row's inputs are on their way while this one is done
  constexpr int kRow = kLogits ? V : 1;
  int next_e = -1;
  float next_dw = 0.f, next_l[kRow], next_ds[kRow];
  auto fetch = [&](int64_t t) {
    if (lane < p.k) {
      next_e = p.experts[t * p.k + lane];
      next_dw = p.dweights[t * p.k + lane];
    }
    if constexpr (kLogits) load_row<kBf16, V, kBlocked>(p.logits, t, p.E, next_l);
    if constexpr (kDense)
      if (p.dscores != nullptr) load_row<false, V, kBlocked>(p.dscores, t, p.E, next_ds);
  };
  int64_t t = (int64_t)blockIdx.x * kWarps + warp;
  if (t < p.T) fetch(t);
  for (; t < p.T; t += stride) {
    // lane i < k: slot i
    const int e = next_e >= 0 && next_e < p.E ? next_e : -1;
    const float dw = e >= 0 ? next_dw : 0.f;  // an empty slot's says nothing
    float le = -INFINITY, l[kRow], ds[kRow];
    if (e >= 0) le = load_logit<kBf16>(p.logits, t * p.E + e);
    if constexpr (kLogits) {
#pragma unroll
      for (int j = 0; j < V; ++j) l[j] = next_l[j];
    }
    if constexpr (kDense) {
#pragma unroll
      for (int j = 0; j < V; ++j) ds[j] = p.dscores != nullptr ? next_ds[j] : 0.f;
    }
    if (t + stride < p.T) fetch(t + stride);
    float m = 0.f;
    bool bad = false;
    if constexpr (kLogits && !kDense) {
      m = row_max<V>(l, false);
#pragma unroll
      for (int j = 0; j < V; ++j) bad |= !(l[j] < INFINITY);
      bad = __any_sync(kFull, bad);
    }
    if constexpr (kDense) {
      if (!p.sigmoid) {
        // l becomes the row's scores
        m = row_max<V>(l, row_has_nan<V>(l));
        float z = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          l[j] = m == -INFINITY ? 0.f : expf(l[j] - m);
          z += l[j];
        }
        z = warp_add(z);
        const float inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
        for (int j = 0; j < V; ++j) l[j] *= inv;
      }
    }
    float d = p.scale * dw;  // the slot's: of its score, or (renormalised) of its logit
    if (p.renorm) {
      const uint32_t key = e >= 0 ? order_key(le) : 0u;
      const uint32_t top_key = __reduce_max_sync(kFull, key);
      const float top = key_value(top_key);
      const bool none = shares_vanish(p.sigmoid, top, kLogits ? m : top);
      const float part = e < 0 || none ? 0.f : share_of(le, p.sigmoid, top);
      // dw_i - sum_j dw_j n_j on the differences from one slot's dw: the sum of
      // the n is 1, and what all slots have in common (for k = 1 everything)
      // then cancels exactly.  The slot of the largest score (its n is at least
      // 1 / k), so that a large dw of a slot with next to no weight stays out of
      // the others' gradients.
      const int ref = __ffs(__ballot_sync(kFull, e >= 0 && key == top_key)) - 1;
      const float by = dw - __shfl_sync(kFull, dw, ref < 0 ? 0 : ref);
      const float sum = warp_add(part), dot = warp_add(by * part);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      d = p.scale * (part * inv) * (by - dot * inv);
      if (p.sigmoid) d *= 1.f / (1.f + expf(le));
    } else if (!kDense) {
      d *= slope(le);
    }
    if (e < 0) d = 0.f;
    float g[V];
    if constexpr (kDense) {
      auto to_slots = [&](float (&v)[V]) {  // v += the slots' d
        for (int i = 0; i < p.k; ++i) {
          const int ei = __shfl_sync(kFull, e, i);
          const float di = __shfl_sync(kFull, d, i);
          // the owner lane and the value's place in it (-1: an empty slot, nobody)
          const int at =
              ei < 0 ? -1 : (kBlocked ? ei - lane * V : ((ei & 31) == lane ? ei >> 5 : -1));
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (at == j) v[j] += di;
        }
      };
      if (!p.renorm) to_slots(ds);
      if (!p.sigmoid) {
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          // values past E have the score 0; their ds must not be -inf
          if (!kBlocked && expert_of<V, kBlocked>(j) >= p.E) ds[j] = 0.f;
          dot += l[j] * ds[j];
        }
        dot = warp_add(dot);
#pragma unroll
        for (int j = 0; j < V; ++j) g[j] = l[j] * (ds[j] - dot);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) g[j] = ds[j] * slope(l[j]);
      }
      if (p.renorm) to_slots(g);
      store_row<kBf16, V, kBlocked>(p.dlogits, t, p.E, g);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) g[j] = bad ? __int_as_float(0x7fc00000) : 0.f;
      store_row<kBf16, V, kBlocked>(p.dlogits, t, p.E, g);
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
      __syncwarp();
      if (first && !bad) store_grad<kBf16>(p.dlogits, t * p.E + e, d);
    }
  }
}

// The dense form with eight lanes per row, four rows a warp, k <= 8, for many
// rows (what does not depend on E is shared by four rows).  The rows are written
// without their slots, then, after a warp barrier, each slot's whole gradient
// over them by a lane of its own.
template <bool kBf16, int V, bool kBlocked>
__global__ void __launch_bounds__(32 * kWarps, (lanes_blocks<V, Lanes::kGradient>()))
    k_route_bwd_lanes(const RouteBwdParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % kRowLanes, first = lane - sub;
  const int64_t stride = (int64_t)gridDim.x * kWarps * 4;
  for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * 4; t0 < p.T; t0 += stride) {
    const bool live = t0 + first / kRowLanes < p.T;
    const int64_t t = live ? t0 + first / kRowLanes : p.T - 1;
    float l[V], ds[V];
    load_row<kBf16, V, kBlocked, kRowLanes>(p.logits, t, p.E, l);
    if (p.dscores != nullptr) load_row<false, V, kBlocked, kRowLanes>(p.dscores, t, p.E, ds);
    int e = -1;
    float dw = 0.f, le = -INFINITY, de = 0.f;
    if (sub < p.k) {
      e = p.experts[t * p.k + sub];
      dw = p.dweights[t * p.k + sub];
      if (e < 0 || e >= p.E) {
        e = -1;
        dw = 0.f;
      }
    }
    if (e >= 0) {
      le = load_logit<kBf16>(p.logits, t * p.E + e);
      if (p.dscores != nullptr) de = __ldg(p.dscores + t * p.E + e);
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
      // values past E have the score 0; their ds must not be -inf
      if (p.dscores == nullptr || (!kBlocked && sub + kRowLanes * j >= p.E)) ds[j] = 0.f;
    float s = 0.f, m = 0.f;  // the slot's score; the row's largest logit
    if (!p.sigmoid) {
      m = l[0];
#pragma unroll
      for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
      const uint32_t key = lanes_max(order_key(m));
      m = key_value(key);
      float z = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        // l becomes the scores; a NaN stays one and makes all of them NaN
        l[j] = m == -INFINITY && l[j] == m ? 0.f : expf(l[j] - m);
        z += l[j];
      }
      z = lanes_add(z);
      const float inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
      for (int j = 0; j < V; ++j) l[j] *= inv;
      if (e >= 0 && m != -INFINITY) s = expf(le - m) * inv;
    }
    float d = p.scale * dw;
    if (p.renorm) {
      // as in k_route_bwd; collectives by all lanes: the rows of a warp differ
      const uint32_t key = e >= 0 ? order_key(le) : 0u;
      const uint32_t top_key = lanes_max(key);
      const float top = key_value(top_key);
      const bool none = shares_vanish(p.sigmoid, top, m);
      const float part = e < 0 || none ? 0.f : share_of(le, p.sigmoid, top);
      const uint32_t at_top = __ballot_sync(kFull, e >= 0 && key == top_key) & (0xffu << first);
      const float by = dw - __shfl_sync(kFull, dw, at_top == 0u ? first : __ffs(at_top) - 1);
      const float sum = lanes_add(part), dot = lanes_add(by * part);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      d = p.scale * (part * inv) * (by - dot * inv);
      if (p.sigmoid) d *= 1.f / (1.f + expf(le));
    }
    if (e < 0) d = 0.f;
    const float mine = p.renorm ? 0.f : s * d;  // of the row's sum of s ds
    // the same expert in two slots: the first of them takes the sum
    bool store = e >= 0;
    const uint32_t same = __match_any_sync(kFull, e >= 0 ? first / kRowLanes * p.E + e : -1 - lane);
    if (__any_sync(kFull, __popc(same) > 1)) {
      float sum = 0.f;
      for (int i = 0; i < p.k; ++i) {
        const float di = __shfl_sync(kFull, d, first + i);
        if ((same >> (first + i)) & 1u) sum += di;
      }
      d = sum;
      store = store && __ffs(same) - 1 == lane;
    }
    float g[V], ge;
    if (!p.sigmoid) {
      float dot = mine;
#pragma unroll
      for (int j = 0; j < V; ++j) dot += l[j] * ds[j];
      dot = lanes_add(dot);
#pragma unroll
      for (int j = 0; j < V; ++j) g[j] = l[j] * (ds[j] - dot);
      ge = p.renorm ? s * (de - dot) + d : s * (de + d - dot);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) g[j] = ds[j] * slope(l[j]);
      ge = p.renorm ? de * slope(le) + d : (de + d) * slope(le);
    }
    if (live) store_row<kBf16, V, kBlocked, kRowLanes>(p.dlogits, t, p.E, g);
    __syncwarp();
    if (store && live) store_grad<kBf16>(p.dlogits, t * p.E + e, ge);
  }
}

}  // namespace

cudaError_t launch_route_backward(const RouteShape &s, const void *logits,
                                  const int32_t *experts, const float *dweights,
                                  const float *dscores, void *dlogits, int num_sms,
                                  cudaStream_t st) {
  const RouteBwdParams p{logits, experts, dweights, dscores, dlogits, s.T,
                         s.E,    s.k,     s.sigmoid, s.renorm, s.scale};
  const bool dense = dscores != nullptr || (!s.sigmoid && !s.renorm);
  const bool vectors = aligned16({logits, dscores, dlogits});
  // Many rows: eight lanes each.  us with dscores, k 8, against a warp a row at 2048 /
  // 8192 / 32768 rows: bf16 64 experts 3.5 / 4.0 / 6.7 against 3.0 / 5.1 / 13.6, 128 3.6 /
  // 5.0 / 10.1 against 3.0 / 6.1 / 17.4, 256 5.0 / 8.3 / 23.9 against 4.0 / 9.1 / 28.7;
  // float32 64 3.4 / 4.6 / 8.6 against 3.1 / 6.2 / 16.9, 192 5.5 / 8.0 / 25.0 against 4.0 /
  // 9.5 / 28.5; but of 256 (a lane's part a whole 128-byte line, in vectors) 6.1 / 11.7 /
  // 36.0 against 4.1 / 10.2 / 29.7.
  const bool lines = vectors && !s.bf16 && s.E == 32 * kRowLanes;  // (not built below)
  if (dense && s.T >= 8192 && s.k <= kRowLanes && s.E <= 256 && !lines) {
    auto go = [&](auto v) {
      constexpr int V = decltype(v)::value;
      auto launch = [&](auto *kern) {
        return launch_rows(kern, (s.T + 3) / 4, lanes_blocks<V, Lanes::kGradient>(), 0, num_sms,
                           st, p);
      };
      const bool blocked = vectors && s.E == kRowLanes * V;
      if (s.bf16)
        return blocked ? launch(k_route_bwd_lanes<true, V, true>)
                       : launch(k_route_bwd_lanes<true, V, false>);
      if constexpr (V < 32)
        if (blocked) return launch(k_route_bwd_lanes<false, V, true>);
      return launch(k_route_bwd_lanes<false, V, false>);
    };
    if (s.E <= 64) return go(std::integral_constant<int, 8>{});
    if (s.E <= 128) return go(std::integral_constant<int, 16>{});
    return go(std::integral_constant<int, 32>{});
  }
  return with_layout(s.E, vectors, false, [&](auto v, auto blocked) {
    constexpr int V = decltype(v)::value;
    constexpr bool kB = decltype(blocked)::value;
    auto go = [&](auto bf16, auto needs) {
      if constexpr (kB && !vector_part<V>())  // (not reached, and not built)
        return cudaErrorInvalidValue;
      else
        return launch_rows(k_route_bwd<decltype(bf16)::value, V, kB, decltype(needs)::value>, s.T,
                           backward_blocks<V>(), 0, num_sms, st, p);
    };
    auto with_all = [&](auto bf16) {
      if (dense) return go(bf16, std::integral_constant<Needs, Needs::kDense>{});
      return s.sigmoid ? go(bf16, std::integral_constant<Needs, Needs::kChosen>{})
                       : go(bf16, std::integral_constant<Needs, Needs::kRow>{});
    };
    return s.bf16 ? with_all(std::true_type{}) : with_all(std::false_type{});
  });
}

}  // namespace sfn
