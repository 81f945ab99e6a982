// experts.cu -- the experts' SwiGLU products around the grouped 8-bit integer
// GEMMs of tc_i8.cu: which row belongs to which expert, and the weighted sum
// over a token's slots.
//
//   y_t = sum_i w[t][i] o[t][i],   o = Wd_e h,   h = bf16(silu(Wg_e x) (Wu_e x))
//
// for e = experts[t][i]; empty slots (expert -1) add nothing.
#include "async_util.cuh"
#include "experts.cuh"
#include "quant_i8.cuh"

namespace sfn {
namespace {

constexpr int kPlanThreads = 1024;  // >= kMaxExperts: one thread per expert scans
constexpr int kCombineThreads = 256;

// Counting sort of the slots by expert, one block.  Where a slot lands among
// its expert's rows depends on the order of the shared-memory atomics, but no
// result does: rows are computed independently of one another, and the
// combine reads each slot's row through pos.
__global__ void __launch_bounds__(kPlanThreads)
    k_expert_plan(const int32_t *experts, int32_t *offsets, int32_t *pos, int64_t slots, int E,
                  unsigned *err) {
  __shared__ int cursor[kMaxExperts];
  __shared__ int warp_sum[32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < E) cursor[tid] = 0;
  __syncthreads();
  bool bad = false;
  for (int64_t i = tid; i < slots; i += kPlanThreads) {
    const int e = experts[i];
    if (e >= 0 && e < E)
      atomicAdd(&cursor[e], 1);
    else
      bad |= e >= E;
  }
  if (bad) report_error(err, kDevErrBounds);
  __syncthreads();
  const int count = tid < E ? cursor[tid] : 0;
  int incl = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += warp_sum[w];
  if (tid < E) {
    cursor[tid] = before + incl - count;
    offsets[tid + 1] = before + incl;
  }
  if (tid == 0) offsets[0] = 0;
  __syncthreads();
  for (int64_t i = tid; i < slots; i += kPlanThreads) {
    const int e = experts[i];
    pos[i] = (e >= 0 && e < E) ? atomicAdd(&cursor[e], 1) : -1;
  }
}

// One block per token: float32 sum over the slots in slot order.
__global__ void __launch_bounds__(kCombineThreads)
    k_expert_combine(const float *__restrict__ o, const int32_t *__restrict__ pos,
                     const float *__restrict__ weights, uint16_t *__restrict__ y, int k, int d) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = blockIdx.x;
  for (int c = threadIdx.x * 4; c < d; c += kCombineThreads * 4) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < k; ++i) {
      const int r = pos[t * k + i];
      if (r < 0) continue;
      const float w = weights[t * k + i];
      const float4 v = *reinterpret_cast<const float4 *>(o + (int64_t)r * d + c);
      s.x += w * v.x;
      s.y += w * v.y;
      s.z += w * v.z;
      s.w += w * v.w;
    }
    uint2 out;
    out.x = (uint32_t)f32_to_bf16_bits(s.x) | ((uint32_t)f32_to_bf16_bits(s.y) << 16);
    out.y = (uint32_t)f32_to_bf16_bits(s.z) | ((uint32_t)f32_to_bf16_bits(s.w) << 16);
    *reinterpret_cast<uint2 *>(y + t * d + c) = out;
  }
}

}  // namespace

ExpertPlan plan_experts(const ExpertShape &s) {
  ExpertPlan p{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  const size_t R = (size_t)s.slots();
  p.off_offsets = take((size_t)(s.E + 1) * 4);
  p.off_pos = take(R * 4);
  p.off_xq = take(R * s.d);
  p.off_sx = take(R * 4);
  p.off_h = take(R * s.f * 2);
  p.off_hq = take(R * s.f);
  p.off_sh = take(R * 4);
  p.off_o = take(R * s.d * 4);
  p.total = off;
  return p;
}

cudaError_t launch_expert_plan(const ExpertShape &s, const int32_t *experts, int32_t *offsets,
                               int32_t *pos, unsigned *err, cudaStream_t st) {
  count_launches(1);
  return launch_pdl(k_expert_plan, dim3(1), dim3(kPlanThreads), 0, st, experts, offsets, pos,
                    s.slots(), s.E, err);
}

cudaError_t launch_expert_combine(const ExpertShape &s, const float *o, const int32_t *pos,
                                  const float *weights, uint16_t *y, cudaStream_t st) {
  count_launches(1);
  return launch_pdl(k_expert_combine, dim3((unsigned)s.T), dim3(kCombineThreads), 0, st, o, pos,
                    weights, y, s.k, s.d);
}

}  // namespace sfn
