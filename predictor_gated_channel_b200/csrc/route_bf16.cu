// route_bf16.cu -- routing (route.cuh), a warp per row, bf16 logits.
#include "route_warps.cuh"

namespace sfn {
template cudaError_t launch_route_warps<true>(const RouteParams &, bool, int, cudaStream_t);
}
