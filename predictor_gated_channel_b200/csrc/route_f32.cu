// route_f32.cu -- routing (route.cuh), a warp per row, float32 logits.
#include "route_warps.cuh"

namespace sfn {
template cudaError_t launch_route_warps<false>(const RouteParams &, bool, int, cudaStream_t);
}
