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
constexpr int kPlanBatch = 8;
constexpr int kCombineThreads = 128;

// Counting sort of the slots by expert, one block.  Where a slot lands among
// its expert's rows depends on the order of the shared-memory atomics, but no
// result does: rows are computed independently of one another, and the
// combine reads each slot's row through pos.
__global__ void __launch_bounds__(kPlanThreads)
    k_expert_plan(const int32_t *__restrict__ experts, int32_t *__restrict__ offsets,
                  int32_t *__restrict__ pos, int64_t slots, int E, unsigned *err) {
  __shared__ int cursor[kMaxExperts];
  __shared__ int warp_sum[32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < E) cursor[tid] = 0;
  __syncthreads();
  bool bad = false;
  // kPlanBatch loads at a time: one block's only way to hide their latency
  auto each = [&](auto &&f) {
    for (int64_t i0 = tid; i0 < slots; i0 += kPlanThreads * kPlanBatch) {
      int e[kPlanBatch];
#pragma unroll
      for (int j = 0; j < kPlanBatch; ++j) {
        const int64_t i = i0 + (int64_t)j * kPlanThreads;
        e[j] = i < slots ? __ldg(experts + i) : -1;
      }
#pragma unroll
      for (int j = 0; j < kPlanBatch; ++j) {
        const int64_t i = i0 + (int64_t)j * kPlanThreads;
        if (i < slots) f(i, e[j]);
      }
    }
  };
  each([&](int64_t, int e) {
    if (e >= 0 && e < E)
      atomicAdd(&cursor[e], 1);
    else
      bad |= e >= E;
  });
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
  each([&](int64_t i, int e) { pos[i] = (e >= 0 && e < E) ? atomicAdd(&cursor[e], 1) : -1; });
}

// y_t = sum over the slots, in slot order and float32; a thread has 8 channels.
// Bound by the reads of o; the loads of four slots are issued together.
__global__ void __launch_bounds__(kCombineThreads)
    k_expert_combine(const float *__restrict__ o, const int32_t *__restrict__ pos,
                     const float *__restrict__ weights, uint16_t *__restrict__ y, int k, int d) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = blockIdx.x;
  const int c = (blockIdx.y * kCombineThreads + threadIdx.x) * 8;
  if (c >= d) return;
  float s[8] = {};
#pragma unroll 4
  for (int i = 0; i < k; ++i) {
    const int64_t at = t * k + i;
    const int r = pos[at];
    if (r < 0) continue;
    const float *src = o + (int64_t)r * d + c;
    const uint4 a = ld_stream16(src), b = ld_stream16(src + 4);
    const float w = weights[at];
    const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = __fmaf_rn(w, __uint_as_float(v[j]), s[j]);
  }
  uint32_t out[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    out[j] = (uint32_t)f32_to_bf16_bits(s[2 * j]) |
             ((uint32_t)f32_to_bf16_bits(s[2 * j + 1]) << 16);
  *reinterpret_cast<uint4 *>(y + t * d + c) = make_uint4(out[0], out[1], out[2], out[3]);
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
  const unsigned parts = (unsigned)((s.d + 8 * kCombineThreads - 1) / (8 * kCombineThreads));
  count_launches(1);
  return launch_pdl(k_expert_combine, dim3((unsigned)s.T, parts), dim3(kCombineThreads), 0, st, o,
                    pos, weights, y, s.k, s.d);
}

}  // namespace sfn
