// quant_i8.cu -- row-wise symmetric quantisation to 8-bit integers.
//
//   amax = max |x|,  scale = amax / 127,  q = rint(127 x / amax)
//
// q is that integer exactly, for both types: a value half way between two (x =
// amax / 2 is one) is seen as exactly half way and goes to the even one, and one
// next to half way to its own side, by the exact remainder.  A row of zeros has
// scale 0 and q 0.  A row with an infinity or a NaN has scale NaN and q 0, so that
// everything computed from it is NaN.
//
// kRowWarps warps per row hold it in registers, kHeld 16-byte chunks a thread,
// between the maximum and the quantisation (one read of x); longer rows are read
// again (from L2).  Short rows have kernels of their own: the unrolled chunks that
// they do not have would cost as much as theirs.
#include "async_util.cuh"
#include "experts.cuh"
#include "quant_i8.cuh"

namespace sfn {
namespace {

constexpr int kQuantWarps = 8;  // per block

// Source rows -> destination rows of one launch.
struct QuantParams {
  const void *x;
  int8_t *q;
  float *scale;
  int64_t rows;
  int K;
  const int32_t *limit;  // if set: only the first *limit rows
  const int32_t *pos;    // if set: row t is written to the rows pos[t * copies + i] >= 0
  int copies;
};

template <class Elt, int kRowWarps, int kHeld>
__global__ void __launch_bounds__(32 * kQuantWarps, kHeld <= 2 ? 8 : 4) k_quantize_rows(const QuantParams p) {
  constexpr int kThreads = 32 * kRowWarps;       // per row
  constexpr int kRows = kQuantWarps / kRowWarps;  // per block
  __shared__ uint32_t part[kQuantWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int sub = threadIdx.x / kThreads, th = threadIdx.x % kThreads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = p.K / Elt::kVec;
  const int64_t rows = p.limit != nullptr ? min((int64_t)*p.limit, p.rows) : p.rows;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < rows; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t r = r0 + sub;
    const bool have = r < rows;
    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const char *>(p.x) +
                                                       (have ? r : r0) * p.K * Elt::kBytes);
    uint4 held[kHeld];
    uint32_t amax = 0u;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int c = th + i * kThreads;
      held[i] = c < chunks ? src[c] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) amax = max(amax, abs_bits_max<Elt>(held[i]));
    for (int c = th + kHeld * kThreads; c < chunks; c += kThreads)
      amax = max(amax, abs_bits_max<Elt>(src[c]));
    amax = __reduce_max_sync(kFull, amax);
    if (kRowWarps > 1) {
      if (lane == 0) part[warp] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) amax = max(amax, part[sub * kRowWarps + w]);
      __syncthreads();
    }
    const QuantScale qs(amax);
    if (!have) continue;
    using Out = typename QuantOut<Elt>::type;
    const int copies = p.pos != nullptr ? p.copies : 1;
    Out out[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) out[i] = quantize_chunk<Elt>(held[i], qs);
    for (int k = 0; k < copies; ++k) {
      const int64_t d = p.pos != nullptr ? p.pos[r * copies + k] : r;
      if (d < 0) continue;
      Out *dst = reinterpret_cast<Out *>(p.q + d * p.K);
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (th + i * kThreads < chunks) dst[th + i * kThreads] = out[i];
#pragma unroll 1
      for (int c = th + kHeld * kThreads; c < chunks; c += kThreads)
        dst[c] = quantize_chunk<Elt>(src[c], qs);
      if (th == 0) p.scale[d] = qs.scale;
    }
  }
}

template <class Elt>
cudaError_t launch(const QuantParams &p, int num_sms, cudaStream_t st) {
  const int chunks = p.K / Elt::kVec;
  auto go = [&](auto *kern, int row_warps) {
    const int64_t rows_per = kQuantWarps / row_warps;
    const int64_t blocks = (p.rows + rows_per - 1) / rows_per;
    const int64_t most = (int64_t)num_sms * 8;
    count_launches(1);
    return launch_pdl(kern, dim3((unsigned)(blocks < most ? blocks : most)),
                      dim3(32 * kQuantWarps), 0, st, p);
  };
  // the fewest warps and chunks that hold a row in registers
  if (chunks <= 32) return go(k_quantize_rows<Elt, 1, 1>, 1);
  if (chunks <= 64) return go(k_quantize_rows<Elt, 1, 2>, 1);
  if (chunks <= 128) return go(k_quantize_rows<Elt, 1, 4>, 1);
  if (chunks <= 256) return go(k_quantize_rows<Elt, 1, 8>, 1);
  if (chunks <= 512) return go(k_quantize_rows<Elt, 2, 8>, 2);
  if (chunks <= 1024) return go(k_quantize_rows<Elt, 4, 8>, 4);
  return go(k_quantize_rows<Elt, 8, 8>, 8);
}

}  // namespace

cudaError_t launch_quantize_rows(const void *x, bool bf16, int8_t *q, float *scale, int64_t T,
                                 int K, int num_sms, cudaStream_t st) {
  const QuantParams p{x, q, scale, T, K, nullptr, nullptr, 1};
  return bf16 ? launch<EltBF16>(p, num_sms, st) : launch<EltF32>(p, num_sms, st);
}

cudaError_t launch_quantize_gather(const ExpertShape &s, const void *x, const int32_t *pos,
                                   int8_t *xq, float *sx, int num_sms, cudaStream_t st) {
  const QuantParams p{x, xq, sx, s.T, s.d, nullptr, pos, s.k};
  return launch<EltBF16>(p, num_sms, st);
}

cudaError_t launch_quantize_expert_rows(const ExpertShape &s, const uint16_t *h,
                                        const int32_t *offsets, int8_t *hq, float *sh,
                                        int num_sms, cudaStream_t st) {
  const QuantParams p{h, hq, sh, s.slots(), s.f, offsets + s.E, nullptr, 1};
  return launch<EltBF16>(p, num_sms, st);
}

}  // namespace sfn
