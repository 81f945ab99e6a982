// route.cu -- routing of tokens to experts (route.cuh): which kernel takes a call.
#include "route.cuh"

namespace sfn {
namespace {

// Eight lanes a row instead of a warp: 32768 x 160 bf16 11.5 us against 18.4,
// 8192 x 64 3.6 against 6.1, 2048 x 160 3.0 against 3.2; float32 32768 x 160 13.3
// against 24.1.  With a bias, where rows may be left to the whole warp, for many
// rows only: 32768 x 64 20.8 us against 30.0, but 4096 x 256 in groups 15.6
// against 11.0.
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
