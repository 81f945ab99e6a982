// route.cu -- routing of tokens to experts (route.cuh): which kernel takes a call.
#include "route.cuh"

namespace sfn {
namespace {

// Eight lanes a row instead of a warp, k 8, us at 512 / 2048 / 8192 / 32768 rows.
// By logit: bf16 64 experts 3.1 / 3.3 / 4.2 / 8.1 against 3.0 / 3.5 / 6.4 / 15.4, 160
// 3.5 / 3.5 / 5.0 / 11.8 against 3.1 / 4.0 / 7.1 / 20.3, 256 4.0 / 4.1 / 6.4 / 15.7
// against 2.9 / 3.9 / 7.2 / 21.9; float32 192 4.2 / 5.1 / 6.7 / 17.6 against 3.4 / 4.5 /
// 8.5 / 27.0 (the worst at 2048); in 8 groups 256 5.1 / 5.5 / 9.0 / 20.5 against 3.9 /
// 5.5 / 12.1 / 38.3.  With a bias, where rows may be left to the whole warp, the two
// meet later: at 2048 / 8192 / 16384 / 32768 rows 64 experts 6.7 / 8.0 / 12.1 / 15.6
// against 5.0 / 8.9 / 14.7 / 25.0, 128 8.2 / 11.2 / 13.7 / 21.5 against 5.4 / 10.1 / 16.0 /
// 29.7, 192 10.4 / 13.7 / 19.4 / 33.6 against 6.0 / 12.1 / 20.2 / 38.9, 256 10.0 / 13.5 /
// 20.3 / 34.1 against 6.5 / 14.1 / 22.8 / 41.4.
bool by_lanes(const RouteParams &p, bool by_logit) {
  if (p.k > 8 || p.scores != nullptr || p.E > 256) return false;
  if (p.groups > 1)  // a lane's values are neighbours, as many as are built
    return by_logit && p.T >= 2048 && 8 % p.groups == 0 && aligned16({p.logits}) &&
           (p.E == 64 || p.E == 128 || p.E == 160 || p.E == 256);
  return p.T >= (by_logit ? 2048 : 16384);
}

}  // namespace

cudaError_t launch_route(const RouteShape &s, const void *logits, const float *bias,
                         int32_t *experts, float *weights, float *scores, int num_sms,
                         cudaStream_t st) {
  RouteParams p{logits, bias, experts, weights, scores, s.T, s.E, s.k, s.groups,
                s.E / s.groups, s.top_groups, s.group_top, s.sigmoid, s.renorm, s.bf16, s.scale, 1u};
  while (p.low + 1 < (uint32_t)s.E) p.low = 2 * p.low + 1;  // index bits of a packed word
  const bool by_logit = bias == nullptr && (s.groups == 1 || s.group_top == 1);
  if (by_lanes(p, by_logit))
    return s.bf16 ? launch_route_lanes<true>(p, by_logit, num_sms, st)
                  : launch_route_lanes<false>(p, by_logit, num_sms, st);
  return s.bf16 ? launch_route_warps<true>(p, by_logit, num_sms, st)
                : launch_route_warps<false>(p, by_logit, num_sms, st);
}

}  // namespace sfn
