// experts.cuh -- host launcher declarations of the expert operators: routing
// to experts (route.cu), the product in 8-bit integers (quant_i8.cu,
// tc_i8.cu) and the experts' SwiGLU products (experts.cu).
#pragma once

#include "sfn_internal.cuh"

namespace sfn {

// ------------------------------------------------------------------ routing
constexpr int kMaxExperts = 1024;    // V = 32 values per lane of a row's warp
constexpr int kMaxExpertsPerTok = 32;  // lane i of the row's warp holds slot i
constexpr int kMaxGroups = 32;       // at least one lane per group

struct RouteShape {
  int64_t T;
  int E, k;
  bool bf16;     // logits (and dlogits) in bf16, else float32
  bool sigmoid;  // scores: sigmoid, else softmax
  int groups, top_groups, group_top;
  bool renorm;
  float scale;
};
cudaError_t launch_route(const RouteShape &s, const void *logits, const float *bias,
                         int32_t *experts, float *weights, float *scores, int num_sms,
                         cudaStream_t st);
cudaError_t launch_route_backward(const RouteShape &s, const void *logits,
                                  const int32_t *experts, const float *dweights,
                                  const float *dscores, void *dlogits, int num_sms,
                                  cudaStream_t st);

// ------------------------------------------------------- 8-bit integer product
// Row-wise symmetric quantisation: scale = max |x| / 127, q = rint(127 x / max |x|).
cudaError_t launch_quantize_rows(const void *x, bool bf16, int8_t *q, float *scale, int64_t T,
                                 int K, int num_sms, cudaStream_t st);

// y[t][n] = sx[t] sw[n] sum_k xq[t][k] wq[n][k].  weights_early: the kernel
// launched before this one on the stream neither writes wq nor lets this one
// start before all work ahead of it is complete.
struct I8Shape {
  int64_t T;
  int N, K;
  bool out_bf16;
};
cudaError_t launch_i8_gemm(const I8Shape &s, const DeviceInfo &dev, const int8_t *xq,
                           const float *sx, const int8_t *wq, const float *sw, void *y,
                           bool weights_early, cudaStream_t st);

// An integer sum times its row's and its channel's scale.  The row's first, but
// where that passes float32's range (a row that holds a type's lowest value as a
// mask has a scale of 2^121) the channel's.
#ifdef __CUDACC__
__device__ __forceinline__ float scaled_sum(float acc, float row, float channel) {
  const float t = __fmul_rn(acc, row);
  return fabsf(t) == INFINITY ? __fmul_rn(__fmul_rn(acc, channel), row) : __fmul_rn(t, channel);
}
#endif

// For a few tokens: the quantisation and the product in one kernel that
// streams the weight rows.
constexpr int kGemvTokens = 4;
bool linear_gemv_ok(const I8Shape &s, int num_sms);
cudaError_t launch_linear_gemv(const I8Shape &s, bool x_bf16, const DeviceInfo &dev,
                               const void *x, const int8_t *wq, const float *sw, void *y,
                               cudaStream_t st);

// ------------------------------------------------------------- expert products
struct ExpertShape {
  int64_t T;
  int E, k, d, f;
  int64_t slots() const { return T * k; }
};
// Rows grouped by expert: expert e's rows are [offsets[e], offsets[e + 1]).
// h[row][f] = bf16(silu(g) u), g and u the int8 products with Wg, Wu.
cudaError_t launch_i8_experts_gateup(const ExpertShape &s, const DeviceInfo &dev,
                                     const int32_t *offsets, const int8_t *xq, const float *sx,
                                     const int8_t *Wg, const float *sg, const int8_t *Wu,
                                     const float *su, uint16_t *h, cudaStream_t st);
// o[row][d] float32, the int8 product with Wd.
cudaError_t launch_i8_experts_down(const ExpertShape &s, const DeviceInfo &dev,
                                   const int32_t *offsets, const int8_t *hq, const float *sh,
                                   const int8_t *Wd, const float *sd, float *o, cudaStream_t st);

// What follows the integer sums is the same in the tiles and in the streams
// below, operation by operation, so that a token's bits do not depend on how many
// tokens share the call:
//   g = scaled_sum(acc, sx, sg), u likewise; h = bf16(swiglu_f32(g, u))
//   o = scaled_sum(acc, sh, sd); y = bf16(the sum of fmaf(w, o, .) in slot order)
// silu(g) u, rounded once, to bf16, by the caller: the element type the FFN's
// activations have in this library, and what is requantised.  The fast exponential
// is off by at most (2 + 1.2 |g|) 2^-23, the quotient by 2^-22: together below 2^-16
// from g = -87 on, where bf16 rounds by 2^-8; below -87 the quotient is 0.  With expf
// and a rounded quotient short products wait for the epilogue: 2497 tokens x 7 of 21
// experts of 400 x 240 83 us against 59, 1199 x 8 of 64 of 576 x 416 102 against 74,
// 1024 x 8 of 16 of 4096 x 1792 229 against 221.  Named roundings: fused in one kernel
// and not in the other, bits would differ.
#ifdef __CUDACC__
__device__ __forceinline__ float swiglu_f32(float g, float u) {
  return __fmul_rn(__fdividef(g, __fadd_rn(1.f, __expf(-g))), u);
}
#endif

// For a few slots (T k <= kGemvSlots, what a warp's lanes hold): gate/up and down
// as streams of the slots' weight rows, each slot on its own.  h is [T k][f] in slot
// order.
constexpr int kGemvSlots = 32;
bool experts_gemv_ok(const ExpertShape &s, int num_sms);
cudaError_t launch_experts_gemv_gateup(const ExpertShape &s, const DeviceInfo &dev, const void *x,
                                       const int32_t *experts, const int8_t *Wg, const float *sg,
                                       const int8_t *Wu, const float *su, uint16_t *h,
                                       cudaStream_t st);
cudaError_t launch_experts_gemv_down(const ExpertShape &s, const DeviceInfo &dev,
                                     const uint16_t *h, const int32_t *experts,
                                     const float *weights, const int8_t *Wd, const float *sd,
                                     uint16_t *y, cudaStream_t st);

// Scratch of the experts' products.
struct ExpertPlan {
  size_t off_offsets, off_pos, off_xq, off_sx, off_h, off_hq, off_sh, off_o, total;
};
ExpertPlan plan_experts(const ExpertShape &s);

// offsets[E + 1] and, for slot t * k + i, its row pos (-1: empty slot).
cudaError_t launch_expert_plan(const ExpertShape &s, const int32_t *experts, int32_t *offsets,
                               int32_t *pos, unsigned *err, cudaStream_t st);
// Quantise x once per token and copy it to the rows of the token's slots.
cudaError_t launch_quantize_gather(const ExpertShape &s, const void *x, const int32_t *pos,
                                   int8_t *xq, float *sx, int num_sms, cudaStream_t st);
// Quantise the first offsets[E] rows of h.
cudaError_t launch_quantize_expert_rows(const ExpertShape &s, const uint16_t *h,
                                        const int32_t *offsets, int8_t *hq, float *sh,
                                        int num_sms, cudaStream_t st);
// y[t] = sum_i weights[t][i] o[pos[t][i]].
cudaError_t launch_expert_combine(const ExpertShape &s, const float *o, const int32_t *pos,
                                  const float *weights, uint16_t *y, cudaStream_t st);

}  // namespace sfn
