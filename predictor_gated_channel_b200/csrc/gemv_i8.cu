// gemv_i8.cu -- the 8-bit integer products for a few tokens: one pass over the
// weight rows at the rate of memory, on the CUDA cores (dp4a).
//
//   k_linear_gemv    y[t][n] = sx[t] sw[n] sum_k xq[t][k] wq[n][k], x quantised
//                    in the kernel
//   k_experts_gateup h[s][c] = bf16(silu(g) u) for the slots s = (t, i)
//   k_experts_down   y[t][n] = sum_i w[t][i] sh[s] sd[e][n] sum_c hq[s][c] Wd[e][n][c],
//                    h quantised in the kernel
//
// With so few tokens a product is a stream of weight rows and nothing else, so
// the work is split for the stream: the rows of the launch are dealt to the
// CTAs (one per SM) in equal contiguous runs, and a CTA's run, cut into pieces
// of at most 2 KB of one row, to its warps in equal contiguous runs again,
// across row boundaries.  Each warp keeps a ring of its own in shared memory
// that bulk copies fill kStages pieces ahead: 128 KB in flight per SM, as 32
// warps x 2 x 2 KB.  Measured on the 8-of-64 experts of 4096 x 1792, one token:
// 39.8 us; 16 warps x 4 x 2 KB 41.9 us, 16 x 2 x 4 KB 41.8 us; the pieces held
// in registers instead, eight loads ahead, 90 us (a warp has too few load
// scoreboards to wait for one of many).
// Where a warp's part of a row ends it adds its lanes up (one integer warp
// reduction) and adds the sum to the row's accumulator in shared memory;
// integer sums are exact in any order, so the result does not depend on the
// split.  The tokens' quantised rows stay in shared memory.
#include "async_util.cuh"
#include "experts.cuh"
#include "quant_i8.cuh"

namespace sfn {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kPiece = 2048;  // most bytes of a row per bulk copy
constexpr int kStages = 2;    // pieces in flight per warp
constexpr int kHeldX = 2;     // 16-byte chunks of x a thread holds
constexpr size_t kRingBytes = (size_t)kWarps * kStages * kPiece;
constexpr size_t kSmemMost = 232448 - 1024;  // of 227 KB: room for the static arrays

// Rows [0, rows) of x (length K, contiguous) quantised into xq [rows][K] with
// their scales.  All threads of the block.
template <class Elt>
__device__ __forceinline__ void quantize_to_smem(const void *x, int rows, int K, int8_t *xq,
                                                 float *scale, uint32_t *amax) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunks = K / Elt::kVec;
  // 2^n warps per row, so that few rows still use every warp
  int per = kWarps;
  while (per > 1 && kWarps / per < rows) per >>= 1;
  const int sub = warp / per, within = (warp % per) * 32 + lane;
  for (int r = tid; r < rows; r += kThreads) amax[r] = 0u;
  __syncthreads();
  // a thread's first chunks of its first row stay in registers between the
  // maximum and the quantisation; what does not fit is read again
  auto source = [&](int r) {
    return reinterpret_cast<const uint4 *>(static_cast<const char *>(x) +
                                           (size_t)r * K * Elt::kBytes);
  };
  uint4 held[kHeldX];
  for (int r = sub; r < rows; r += kWarps / per) {
    const uint4 *src = source(r);
    uint32_t m = 0u;
    if (r == sub) {
#pragma unroll
      for (int i = 0; i < kHeldX; ++i) {
        const int c = within + i * per * 32;
        held[i] = c < chunks ? src[c] : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < kHeldX; ++i) m = max(m, abs_bits_max<Elt>(held[i]));
    }
    for (int c = within + (r == sub ? kHeldX : 0) * per * 32; c < chunks; c += per * 32)
      m = max(m, abs_bits_max<Elt>(src[c]));
    m = __reduce_max_sync(kFull, m);
    if (lane == 0) atomicMax(&amax[r], m);
  }
  __syncthreads();
  for (int r = sub; r < rows; r += kWarps / per) {
    const uint4 *src = source(r);
    using Out = typename QuantOut<Elt>::type;
    Out *dst = reinterpret_cast<Out *>(xq + (size_t)r * K);
    const QuantScale qs(amax[r]);
    if (r == sub) {
#pragma unroll
      for (int i = 0; i < kHeldX; ++i) {
        const int c = within + i * per * 32;
        if (c < chunks) dst[c] = quantize_chunk<Elt>(held[i], qs);
      }
    }
    for (int c = within + (r == sub ? kHeldX : 0) * per * 32; c < chunks; c += per * 32)
      dst[c] = quantize_chunk<Elt>(src[c], qs);
    if (within == 0) scale[r] = qs.scale;
  }
}

// One CTA's weight rows [0, rows) (length K): acc[v * kTok + t] += dot of row
// v with token row t of its x.  Rows: a cursor over the CTA's rows, with
// start(v), next(), row() and x(); one copy walks ahead for the loads.
// ready(): called once, after the first copies are issued and before the
// first use of x.  ring: kRingBytes; bars: kWarps * kStages barriers,
// initialised.
template <int kTok, class Rows, class Ready>
__device__ __forceinline__ void stream_rows(int rows, int K, int *acc, unsigned char *ring,
                                            uint64_t *bars, unsigned *err, Rows ahead,
                                            Ready &&ready) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ring += (size_t)warp * kStages * kPiece;
  bars += warp * kStages;
  const int per_row = (K + kPiece - 1) / kPiece;
  const int last_bytes = K - (per_row - 1) * kPiece;  // of a row's last piece
  const int64_t total = (int64_t)rows * per_row;
  const int64_t begin = total * warp / kWarps;
  const int n = (int)(total * (warp + 1) / kWarps - begin);
  int v = (int)(begin / per_row), k = (int)(begin - (int64_t)v * per_row);
  int lk = k;
  Rows at = ahead;
  const int8_t *lp = nullptr, *xp = nullptr;
  if (n > 0) {
    ahead.start(v);
    at.start(v);
    lp = ahead.row() + lk * kPiece;
    xp = at.x() + k * kPiece;
  }
  int issued = 0;
  const uint64_t once = make_evict_first_policy();
  auto issue = [&](int s) {  // the next piece into stage s (one lane copies)
    const bool end_of_row = lk == per_row - 1;
    if (lane == 0) {
      const uint32_t bytes = end_of_row ? last_bytes : kPiece;
      mbar_arrive_expect_tx(&bars[s], bytes);
      bulk_g2s_hint(ring + s * kPiece, lp, bytes, &bars[s], once);
    }
    ++issued;
    ++lk;
    lp += kPiece;
    if (end_of_row && issued < n) {
      lk = 0;
      ahead.next();
      lp = ahead.row();
    }
  };
  for (int s = 0; s < kStages && issued < n; ++s) issue(s);
  ready();
  // four sums a token: a chain of dependent dp4a per 16 bytes of a lane
  int sum[kTok][4];
#pragma unroll
  for (int t = 0; t < kTok; ++t) sum[t][0] = sum[t][1] = sum[t][2] = sum[t][3] = 0;
  auto dot = [&](const unsigned char *w, const int8_t *x) {
    const uint4 wv = *reinterpret_cast<const uint4 *>(w);
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      const uint4 xv = *reinterpret_cast<const uint4 *>(x + (size_t)t * K);
      sum[t][0] = __dp4a((int)wv.x, (int)xv.x, sum[t][0]);
      sum[t][1] = __dp4a((int)wv.y, (int)xv.y, sum[t][1]);
      sum[t][2] = __dp4a((int)wv.z, (int)xv.z, sum[t][2]);
      sum[t][3] = __dp4a((int)wv.w, (int)xv.w, sum[t][3]);
    }
  };
  int s = 0;
  uint32_t phase = 0;
  for (int i = 0; i < n; ++i) {
    if (!mbar_wait(&bars[s], phase, err)) {
      // give the copies in flight one more bounded wait each, then give up
      for (int j = i; j < issued; ++j) {
        mbar_wait(&bars[s], phase, err);
        if (++s == kStages) {
          s = 0;
          phase ^= 1u;
        }
      }
      return;
    }
    const bool end_of_row = k == per_row - 1;
    const unsigned char *w = ring + s * kPiece + lane * 16;
    const int8_t *xr = xp + lane * 16;
    if (!end_of_row || last_bytes == kPiece) {
#pragma unroll
      for (int o = 0; o < kPiece; o += 512) dot(w + o, xr + o);
    } else {
      for (int o = 0; o < last_bytes; o += 512)
        if (o + lane * 16 < last_bytes) dot(w + o, xr + o);
    }
    __syncwarp();  // every lane has read the stage
    if (issued < n) issue(s);
    if (++s == kStages) {
      s = 0;
      phase ^= 1u;
    }
    ++k;
    xp += kPiece;
    if (end_of_row || i + 1 == n) {
#pragma unroll
      for (int t = 0; t < kTok; ++t) {
        const int r = __reduce_add_sync(kFull, sum[t][0] + sum[t][1] + sum[t][2] + sum[t][3]);
        if (lane == 0) atomicAdd(&acc[v * kTok + t], r);
        sum[t][0] = sum[t][1] = sum[t][2] = sum[t][3] = 0;
      }
      if (i + 1 < n) {
        k = 0;
        ++v;
        at.next();
        xp = at.x();
      }
    }
  }
}

// Initialise the rings' barriers; the block synchronises before their use.
__device__ __forceinline__ void init_bars(uint64_t *bars) {
  if (threadIdx.x < kWarps * kStages) mbar_init(&bars[threadIdx.x], 1);
  fence_barrier_init();
}

// A CTA's share of n units: [first, last).
__device__ __forceinline__ void my_share(int n, int &first, int &last) {
  first = (int)((int64_t)n * blockIdx.x / gridDim.x);
  last = (int)((int64_t)n * (blockIdx.x + 1) / gridDim.x);
}

// Cursors over a CTA's rows (stream_rows).
struct LinearRows {  // rows n0, n0 + 1, ... of one matrix
  const int8_t *w;
  const int8_t *xq;
  int K;
  __device__ __forceinline__ void start(int v) { w += (int64_t)v * K; }
  __device__ __forceinline__ void next() { w += K; }
  __device__ __forceinline__ const int8_t *row() const { return w; }
  __device__ __forceinline__ const int8_t *x() const { return xq; }
};
struct GateUpRows {  // units (slot s, channel c) from u0 on, Wg's row, then Wu's
  const int8_t *Wg, *Wu, *xq;
  const int *ids;
  int u0, f, d, k;
  int s, c, up;
  const int8_t *g, *u;  // this unit's rows
  // an empty slot reads expert 0 and its h is written as 0: a decode step
  // seldom has one
  __device__ __forceinline__ void seek() {
    const int64_t o = ((int64_t)max(ids[s], 0) * f + c) * d;
    g = Wg + o;
    u = Wu + o;
  }
  __device__ __forceinline__ void start(int v) {
    const int unit = u0 + (v >> 1);
    up = v & 1;
    s = unit / f;
    c = unit - s * f;
    seek();
  }
  __device__ __forceinline__ void next() {
    up ^= 1;
    if (up) return;
    g += d;
    u += d;
    if (++c == f) {
      c = 0;
      ++s;
      seek();
    }
  }
  __device__ __forceinline__ const int8_t *row() const { return up ? u : g; }
  __device__ __forceinline__ const int8_t *x() const { return xq + (size_t)(s / k) * d; }
};
struct DownRows {  // units (token t, output channel n) from u0 on, k slots' rows each
  const int8_t *Wd, *hq;
  const int *ids;
  int u0, f, d, k;
  int t, n, j;
  __device__ __forceinline__ void start(int v) {
    const int u = u0 + v / k;
    j = v % k;
    t = u / d;
    n = u - t * d;
  }
  __device__ __forceinline__ void next() {
    if (++j == k) {
      j = 0;
      if (++n == d) {
        n = 0;
        ++t;
      }
    }
  }
  __device__ __forceinline__ const int8_t *row() const {
    return Wd + ((int64_t)max(ids[t * k + j], 0) * d + n) * f;
  }
  __device__ __forceinline__ const int8_t *x() const {
    return hq + (size_t)(t * k + j) * f;
  }
};

template <class Elt, int kTok, bool kOutBf16>
__global__ void __launch_bounds__(kThreads)
    k_linear_gemv(const void *__restrict__ x, const int8_t *__restrict__ wq,
                  const float *__restrict__ sw, void *__restrict__ y, int T, int N, int K,
                  int acc_bytes, unsigned *err) {
  extern __shared__ __align__(16) unsigned char smem[];
  int *acc = reinterpret_cast<int *>(smem + kRingBytes);
  int8_t *xq = reinterpret_cast<int8_t *>(smem + kRingBytes + acc_bytes);
  __shared__ uint64_t bars[kWarps * kStages];
  init_bars(bars);
  __shared__ float sx[kTok];
  __shared__ uint32_t amax[kTok];
  pdl_wait();
  pdl_launch_dependents();
  int n0, n1;
  my_share(N, n0, n1);
  const int rows = n1 - n0;
  for (int i = threadIdx.x; i < rows * kTok; i += kThreads) acc[i] = 0;
  __syncthreads();
  stream_rows<kTok>(
      rows, K, acc, smem, bars, err, LinearRows{wq + (int64_t)n0 * K, xq, K}, [&] {
        quantize_to_smem<Elt>(x, T, K, xq, sx, amax);
        __syncthreads();
      });
  __syncthreads();
  for (int i = threadIdx.x; i < rows * T; i += kThreads) {
    const int t = i / rows, v = i - t * rows;
    const float r = (float)acc[v * kTok + t] * sx[t] * sw[n0 + v];
    const int64_t o = (int64_t)t * N + n0 + v;
    if (kOutBf16)
      static_cast<uint16_t *>(y)[o] = f32_to_bf16_bits(r);
    else
      static_cast<float *>(y)[o] = r;
  }
}

// Units: (slot, channel) pairs of rows, Wg's then Wu's.
__global__ void __launch_bounds__(kThreads)
    k_experts_gateup(const void *__restrict__ x, const int32_t *__restrict__ experts,
                     const int8_t *__restrict__ Wg, const float *__restrict__ sg,
                     const int8_t *__restrict__ Wu, const float *__restrict__ su,
                     uint16_t *__restrict__ h, int T, int E, int k, int d, int f, int acc_bytes,
                     unsigned *err) {
  extern __shared__ __align__(16) unsigned char smem[];
  int *acc = reinterpret_cast<int *>(smem + kRingBytes);
  int8_t *xq = reinterpret_cast<int8_t *>(smem + kRingBytes + acc_bytes);
  __shared__ uint64_t bars[kWarps * kStages];
  init_bars(bars);
  __shared__ float sx[kGemvSlots];
  __shared__ uint32_t amax[kGemvSlots];
  __shared__ int ids[kGemvSlots];
  pdl_wait();
  pdl_launch_dependents();
  const int slots = T * k;
  for (int i = threadIdx.x; i < slots; i += kThreads) {
    const int e = experts[i];
    if (e >= E) report_error(err, kDevErrBounds);
    ids[i] = (e >= 0 && e < E) ? e : -1;
  }
  int u0, u1;
  my_share(slots * f, u0, u1);
  const int units = u1 - u0;
  for (int i = threadIdx.x; i < 2 * units; i += kThreads) acc[i] = 0;
  __syncthreads();
  stream_rows<1>(2 * units, d, acc, smem, bars, err, GateUpRows{Wg, Wu, xq, ids, u0, f, d, k},
      [&] {
        quantize_to_smem<EltBF16>(x, T, d, xq, sx, amax);
        __syncthreads();
      });
  __syncthreads();
  for (int i = threadIdx.x; i < units; i += kThreads) {
    const int u = u0 + i, s = u / f;
    const int64_t row = (int64_t)max(ids[s], 0) * f + (u - s * f);
    const float a = sx[s / k];
    const float g = (float)acc[2 * i] * a * sg[row], up = (float)acc[2 * i + 1] * a * su[row];
    h[u] = ids[s] < 0 ? (uint16_t)0 : f32_to_bf16_bits(g * sigmoid_f32(g) * up);
  }
}

// Units: (token, output channel), each k rows of Wd, one per slot.
__global__ void __launch_bounds__(kThreads)
    k_experts_down(const uint16_t *__restrict__ h, const int32_t *__restrict__ experts,
                   const float *__restrict__ weights, const int8_t *__restrict__ Wd,
                   const float *__restrict__ sd, uint16_t *__restrict__ y, int T, int E, int k,
                   int d, int f, int acc_bytes, unsigned *err) {
  extern __shared__ __align__(16) unsigned char smem[];
  int *acc = reinterpret_cast<int *>(smem + kRingBytes);
  int8_t *hq = reinterpret_cast<int8_t *>(smem + kRingBytes + acc_bytes);
  __shared__ uint64_t bars[kWarps * kStages];
  init_bars(bars);
  __shared__ float sh[kGemvSlots];
  __shared__ uint32_t amax[kGemvSlots];
  __shared__ int ids[kGemvSlots];
  const int slots = T * k;
  int u0, u1;
  my_share(T * d, u0, u1);
  const int units = u1 - u0;
  for (int i = threadIdx.x; i < units * k; i += kThreads) acc[i] = 0;
  // experts and weights were there before this call's first kernel, which
  // waited for all earlier work before it let this one start: only h needs
  // the wait, so the first weight rows are on their way before it
  for (int i = threadIdx.x; i < slots; i += kThreads) {
    const int e = experts[i];
    ids[i] = (e >= 0 && e < E) ? e : -1;
  }
  __syncthreads();
  stream_rows<1>(units * k, f, acc, smem, bars, err, DownRows{Wd, hq, ids, u0, f, d, k},
      [&] {
        pdl_wait();
        pdl_launch_dependents();
        quantize_to_smem<EltBF16>(h, slots, f, hq, sh, amax);
        __syncthreads();
      });
  __syncthreads();
  for (int i = threadIdx.x; i < units; i += kThreads) {
    const int u = u0 + i, t = u / d, n = u - t * d;
    float s = 0.f;
    for (int j = 0; j < k; ++j) {
      const int e = ids[t * k + j];
      if (e >= 0)
        s += weights[t * k + j] *
             ((float)acc[i * k + j] * sh[t * k + j] * sd[(int64_t)e * d + n]);
    }
    y[u] = f32_to_bf16_bits(s);
  }
}

int ctas_for(int64_t units, int num_sms) { return (int)(units < num_sms ? units : num_sms); }
// bytes of one CTA's accumulators: `per` integers for each of its units
size_t acc_bytes_for(int64_t units, int per, int num_sms) {
  const int64_t ctas = ctas_for(units, num_sms);
  return align_up((size_t)((units + ctas - 1) / ctas) * per * sizeof(int), 16);
}
template <class F, class... Args>
cudaError_t go(F *kern, size_t smem, int ctas, cudaStream_t st, Args... args) {
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kern), smem);
  if (e != cudaSuccess) return e;
  count_launches(1);
  return launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, st, args...);
}

}  // namespace

bool linear_gemv_ok(const I8Shape &s, int num_sms) {
  if (s.T > kGemvTokens) return false;
  const int tok = s.T > 2 ? 4 : (int)s.T;
  return kRingBytes + acc_bytes_for(s.N, tok, num_sms) + (size_t)tok * s.K <= kSmemMost;
}

cudaError_t launch_linear_gemv(const I8Shape &s, bool x_bf16, const DeviceInfo &dev,
                               const void *x, const int8_t *wq, const float *sw, void *y,
                               cudaStream_t st) {
  auto run = [&](auto elt, auto tok, auto out) {
    using Elt = decltype(elt);
    constexpr int kTok = decltype(tok)::value;
    constexpr bool kOut = decltype(out)::value;
    const size_t acc = acc_bytes_for(s.N, kTok, dev.num_sms);
    return go(k_linear_gemv<Elt, kTok, kOut>, kRingBytes + acc + (size_t)kTok * s.K,
              ctas_for(s.N, dev.num_sms), st, x, wq, sw, y, (int)s.T, s.N, s.K, (int)acc, dev.err);
  };
  auto with_out = [&](auto elt, auto tok) {
    return s.out_bf16 ? run(elt, tok, std::true_type{}) : run(elt, tok, std::false_type{});
  };
  auto with_tok = [&](auto elt) {
    if (s.T == 1) return with_out(elt, std::integral_constant<int, 1>{});
    if (s.T == 2) return with_out(elt, std::integral_constant<int, 2>{});
    return with_out(elt, std::integral_constant<int, 4>{});
  };
  return x_bf16 ? with_tok(EltBF16{}) : with_tok(EltF32{});
}

bool experts_gemv_ok(const ExpertShape &s, int num_sms) {
  if (s.slots() > kGemvSlots || s.slots() * s.f * 2 > 0x7fffffffLL ||
      s.slots() * s.d > 0x7fffffffLL)
    return false;
  const size_t up = kRingBytes + acc_bytes_for(s.slots() * s.f, 2, num_sms) + (size_t)s.T * s.d;
  const size_t down = kRingBytes + acc_bytes_for(s.T * s.d, s.k, num_sms) + (size_t)s.slots() * s.f;
  return up <= kSmemMost && down <= kSmemMost;
}

cudaError_t launch_experts_gemv_gateup(const ExpertShape &s, const DeviceInfo &dev, const void *x,
                                       const int32_t *experts, const int8_t *Wg, const float *sg,
                                       const int8_t *Wu, const float *su, uint16_t *h,
                                       cudaStream_t st) {
  const int64_t units = s.slots() * s.f;
  const size_t acc = acc_bytes_for(units, 2, dev.num_sms);
  return go(k_experts_gateup, kRingBytes + acc + (size_t)s.T * s.d, ctas_for(units, dev.num_sms), st,
            x, experts, Wg, sg, Wu, su, h, (int)s.T, s.E, s.k, s.d, s.f, (int)acc, dev.err);
}

cudaError_t launch_experts_gemv_down(const ExpertShape &s, const DeviceInfo &dev,
                                     const uint16_t *h, const int32_t *experts,
                                     const float *weights, const int8_t *Wd, const float *sd,
                                     uint16_t *y, cudaStream_t st) {
  const int64_t units = s.T * s.d;
  const size_t acc = acc_bytes_for(units, s.k, dev.num_sms);
  return go(k_experts_down, kRingBytes + acc + (size_t)s.slots() * s.f, ctas_for(units, dev.num_sms),
            st, h, experts, weights, Wd, sd, y, (int)s.T, s.E, s.k, s.d, s.f, (int)acc, dev.err);
}

}  // namespace sfn
