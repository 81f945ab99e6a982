// gemv_i8.cu -- the 8-bit integer products for a few tokens: one pass over the
// weight rows at the rate of memory, on the CUDA cores (dp4a).
//
//   k_linear_gemv    y[t][n] = sx[t] sw[n] sum_k xq[t][k] wq[n][k], x quantised
//                    in the kernel
//   k_experts_gateup h[s][c] = bf16(silu(g) u) for the slots s = (t, i)
//   k_experts_down   y[t][n] = sum_i w[t][i] (sum_c hq[s][c] Wd[e][n][c]) sh[s] sd[e][n],
//                    h quantised in the kernel
//
// With so few tokens a product is a stream of weight rows and nothing else, so
// the work is split for the stream: the rows of the launch are dealt to the
// CTAs (one per SM) in equal contiguous runs, and a CTA's run, cut into pieces
// of at most 2 KB of one row, to its warps in equal contiguous runs again,
// across row boundaries.  Each warp keeps a ring of its own in shared memory
// that bulk copies fill kStages pieces ahead: 128 KB in flight per SM, as 32
// warps x 2 x 2 KB.  Measured on the 8-of-64 experts of 4096 x 1792, one token:
// 37.4 us (when it took 36.9: a third stage 42.5 us, pieces of 1 KB 46 us, the
// pieces dealt round robin 39.4 us; the pieces held in registers instead, eight
// loads ahead, 90 us: a warp has too few load scoreboards to wait for one of
// many).  The stream runs at the rate of memory (58.7 MB in 8.6 us); what is left is
// 4.6 us a kernel: its launch, the rows' quantisation, the last sums.
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
constexpr size_t kSmemMost = 232448 - 1280;  // of 227 KB: room for the static arrays

// Rows [0, rows) of x (length K, contiguous) quantised into xq [rows][K] with
// their scales, by all threads of the block: load() starts the reads of a
// thread's first chunks, store() does the rest.
template <class Elt>
struct RowQuantizer {
  const void *x;
  int rows, K, per, sub, within, chunks;
  uint4 held[kHeldX];
  __device__ __forceinline__ const uint4 *source(int r) const {
    return reinterpret_cast<const uint4 *>(static_cast<const char *>(x) +
                                           (size_t)r * K * Elt::kBytes);
  }
  __device__ __forceinline__ void load(const void *x_, int rows_, int K_) {
    x = x_;
    rows = rows_;
    K = K_;
    chunks = K / Elt::kVec;
    // 2^n warps per row, so that few rows still use every warp
    per = kWarps;
    while (per > 1 && kWarps / per < rows) per >>= 1;
    sub = (threadIdx.x >> 5) / per;
    within = ((threadIdx.x >> 5) % per) * 32 + (threadIdx.x & 31);
#pragma unroll
    for (int i = 0; i < kHeldX; ++i) {
      const int c = within + i * per * 32;
      held[i] = sub < rows && c < chunks ? source(sub)[c] : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  // amax: zeroed, and a barrier since
  __device__ __forceinline__ void store(int8_t *xq, float *scale, uint32_t *amax) {
    // a thread's first chunks of its first row stay in registers between the
    // maximum and the quantisation; what does not fit is read again
    for (int r = sub; r < rows; r += kWarps / per) {
      uint32_t m = 0u;
      if (r == sub) {
#pragma unroll
        for (int i = 0; i < kHeldX; ++i) m = max(m, abs_bits_max<Elt>(held[i]));
      }
      for (int c = within + (r == sub ? kHeldX : 0) * per * 32; c < chunks; c += per * 32)
        m = max(m, abs_bits_max<Elt>(source(r)[c]));
      m = __reduce_max_sync(kFull, m);
      if ((threadIdx.x & 31) == 0) atomicMax(&amax[r], m);
    }
    __syncthreads();
    using Out = typename QuantOut<Elt>::type;
    for (int r = sub; r < rows; r += kWarps / per) {
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
        dst[c] = quantize_chunk<Elt>(source(r)[c], qs);
      if (within == 0) scale[r] = qs.scale;
    }
  }
};

// One CTA's weight rows [0, rows) (length K): acc[v * kTok + t] += dot of row
// v with token row t of its x.  Rows: a cursor over the CTA's rows, with
// start(v), next(), row() and x(); one copy walks ahead for the loads.
// ready(): called once, after the first copies are issued and before the
// first use of x.  ring: kWarps * kStages * kPiece bytes; bars: kWarps * kStages
// barriers, initialised.
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

// The kernels' dynamic shared memory: the ring, the accumulators, a scale for
// each accumulator (read at the start: at the end a cold read would cost its
// latency once more), the quantised rows.
struct Layout {
  size_t acc, scale, rows, total;
  Layout(int64_t accs, int64_t scales, int64_t row_bytes) {
    acc = (size_t)kWarps * kStages * kPiece;
    scale = acc + align_up((size_t)accs * sizeof(int), 16);
    rows = scale + align_up((size_t)scales * sizeof(float), 16);
    total = rows + (size_t)row_bytes;
  }
};

template <class Elt, int kTok, bool kOutBf16>
__global__ void __launch_bounds__(kThreads)
    k_linear_gemv(const void *__restrict__ x, const int8_t *__restrict__ wq,
                  const float *__restrict__ sw, void *__restrict__ y, int T, int N, int K,
                  const Layout lay, unsigned *err) {
  extern __shared__ __align__(16) unsigned char smem[];
  int *acc = reinterpret_cast<int *>(smem + lay.acc);
  float *scale = reinterpret_cast<float *>(smem + lay.scale);
  int8_t *xq = reinterpret_cast<int8_t *>(smem + lay.rows);
  __shared__ uint64_t bars[kWarps * kStages];
  __shared__ float sx[kTok];
  __shared__ uint32_t amax[kTok];
  init_bars(bars);
  if (threadIdx.x < kTok) amax[threadIdx.x] = 0u;
  int n0, n1;
  my_share(N, n0, n1);
  const int rows = n1 - n0;
  for (int i = threadIdx.x; i < rows * kTok; i += kThreads) acc[i] = 0;
  pdl_wait();
  pdl_launch_dependents();
  RowQuantizer<Elt> quant;
  quant.load(x, T, K);
  const float first_scale = threadIdx.x < rows ? sw[n0 + threadIdx.x] : 0.f;
  __syncthreads();
  stream_rows<kTok>(
      rows, K, acc, smem, bars, err, LinearRows{wq + (int64_t)n0 * K, xq, K}, [&] {
        quant.store(xq, sx, amax);
        for (int i = threadIdx.x; i < rows; i += kThreads)
          scale[i] = i < kThreads ? first_scale : sw[n0 + i];
        __syncthreads();
      });
  __syncthreads();
  for (int i = threadIdx.x; i < rows * T; i += kThreads) {
    const int t = i / rows, v = i - t * rows;
    const float r = scaled_sum((float)acc[v * kTok + t], sx[t], scale[v]);
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
                     uint16_t *__restrict__ h, int T, int E, int k, int d, int f,
                     const Layout lay, unsigned *err) {
  extern __shared__ __align__(16) unsigned char smem[];
  int *acc = reinterpret_cast<int *>(smem + lay.acc);
  float2 *scale = reinterpret_cast<float2 *>(smem + lay.scale);
  int8_t *xq = reinterpret_cast<int8_t *>(smem + lay.rows);
  __shared__ uint64_t bars[kWarps * kStages];
  __shared__ float sx[kGemvSlots];
  __shared__ uint32_t amax[kGemvSlots];
  __shared__ int ids[kGemvSlots];
  init_bars(bars);
  const int slots = T * k;
  int u0, u1;
  my_share(slots * f, u0, u1);
  const int units = u1 - u0;
  for (int i = threadIdx.x; i < 2 * units; i += kThreads) acc[i] = 0;
  if (threadIdx.x < kGemvSlots) amax[threadIdx.x] = 0u;
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x < slots) {
    const int e = experts[threadIdx.x];
    if (e >= E) report_error(err, kDevErrBounds);
    ids[threadIdx.x] = (e >= 0 && e < E) ? e : -1;
  }
  RowQuantizer<EltBF16> quant;
  quant.load(x, T, d);
  __syncthreads();
  stream_rows<1>(
      2 * units, d, acc, smem, bars, err, GateUpRows{Wg, Wu, xq, ids, u0, f, d, k}, [&] {
        for (int i = threadIdx.x; i < units; i += kThreads) {
          const int u = u0 + i, s = u / f;
          const int64_t row = (int64_t)max(ids[s], 0) * f + (u - s * f);
          scale[i] = make_float2(sg[row], su[row]);
        }
        quant.store(xq, sx, amax);
        __syncthreads();
      });
  __syncthreads();
  for (int i = threadIdx.x; i < units; i += kThreads) {
    const int u = u0 + i, s = u / f;
    const float a = sx[s / k];
    const float2 w = scale[i];
    const float g = scaled_sum((float)acc[2 * i], a, w.x);
    const float up = scaled_sum((float)acc[2 * i + 1], a, w.y);
    h[u] = ids[s] < 0 ? (uint16_t)0 : f32_to_bf16_bits(swiglu_f32(g, up));
  }
}

// Units: (token, output channel), each k rows of Wd, one per slot.
__global__ void __launch_bounds__(kThreads)
    k_experts_down(const uint16_t *__restrict__ h, const int32_t *__restrict__ experts,
                   const float *__restrict__ weights, const int8_t *__restrict__ Wd,
                   const float *__restrict__ sd, uint16_t *__restrict__ y, int T, int E, int k,
                   int d, int f, const Layout lay, unsigned *err) {
  extern __shared__ __align__(16) unsigned char smem[];
  int *acc = reinterpret_cast<int *>(smem + lay.acc);
  float *scale = reinterpret_cast<float *>(smem + lay.scale);
  int8_t *hq = reinterpret_cast<int8_t *>(smem + lay.rows);
  __shared__ uint64_t bars[kWarps * kStages];
  __shared__ float sh[kGemvSlots];
  __shared__ uint32_t amax[kGemvSlots];
  __shared__ int ids[kGemvSlots];
  __shared__ float slot_weight[kGemvSlots];
  init_bars(bars);
  const int slots = T * k;
  int u0, u1;
  my_share(T * d, u0, u1);
  const int units = u1 - u0;
  // experts and weights were there before this call's first kernel, which
  // waited for all earlier work before it let this one start: only h needs
  // the wait, so the first weight rows are on their way before it
  if (threadIdx.x < slots) {
    const int e = experts[threadIdx.x];
    ids[threadIdx.x] = (e >= 0 && e < E) ? e : -1;
  }
  if (threadIdx.x < kGemvSlots) amax[threadIdx.x] = 0u;
  __syncthreads();
  stream_rows<1>(
      units * k, f, acc, smem, bars, err, DownRows{Wd, hq, ids, u0, f, d, k}, [&] {
        if (threadIdx.x < slots) slot_weight[threadIdx.x] = weights[threadIdx.x];
        for (int i = threadIdx.x; i < units * k; i += kThreads) {
          const int u = u0 + i / k, s = u / d * k + i % k;
          acc[i] = 0;
          scale[i] = ids[s] >= 0 ? sd[(int64_t)ids[s] * d + u % d] : 0.f;
        }
        pdl_wait();
        pdl_launch_dependents();
        RowQuantizer<EltBF16> quant;
        quant.load(h, slots, f);
        quant.store(hq, sh, amax);
        __syncthreads();
      });
  __syncthreads();
  for (int i = threadIdx.x; i < units; i += kThreads) {
    const int u = u0 + i, t = u / d;
    float s = 0.f;
    for (int j = 0; j < k; ++j)
      if (ids[t * k + j] >= 0)
        s = __fmaf_rn(slot_weight[t * k + j],
                      scaled_sum((float)acc[i * k + j], sh[t * k + j], scale[i * k + j]), s);
    y[u] = f32_to_bf16_bits(s);
  }
}

int ctas_for(int64_t units, int num_sms) { return (int)(units < num_sms ? units : num_sms); }
// most units of one CTA
int64_t share_of(int64_t units, int num_sms) {
  const int64_t ctas = ctas_for(units, num_sms);
  return (units + ctas - 1) / ctas;
}
Layout linear_layout(const I8Shape &s, int tok, int num_sms) {
  const int64_t rows = share_of(s.N, num_sms);
  return Layout(rows * tok, rows, (int64_t)tok * s.K);
}
Layout gateup_layout(const ExpertShape &s, int num_sms) {
  const int64_t units = share_of(s.slots() * s.f, num_sms);
  return Layout(2 * units, 2 * units, s.T * s.d);
}
Layout down_layout(const ExpertShape &s, int num_sms) {
  const int64_t units = share_of(s.T * s.d, num_sms);
  return Layout(units * s.k, units * s.k, s.slots() * s.f);
}
int tokens_for(int64_t T) { return T > 2 ? 4 : (int)T; }

template <class F, class... Args>
cudaError_t go(F *kern, const Layout &lay, int ctas, cudaStream_t st, Args... args) {
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kern), lay.total);
  if (e != cudaSuccess) return e;
  count_launches(1);
  return launch_pdl(kern, dim3(ctas), dim3(kThreads), lay.total, st, args...);
}
}  // namespace

// Three and four tokens keep pace with the stream for small matrices only: of
// 4096 x 4096 9.7 us against 9.7 on the tensor cores, of 4096 x 14336 19.5
// against 17.9 (two tokens: 15.4 against 17.9).
bool linear_gemv_ok(const I8Shape &s, int num_sms) {
  if (s.T > kGemvTokens || (s.T > 2 && (int64_t)s.N * s.K > ((int64_t)1 << 24))) return false;
  return linear_layout(s, tokens_for(s.T), num_sms).total <= kSmemMost;
}

cudaError_t launch_linear_gemv(const I8Shape &s, bool x_bf16, const DeviceInfo &dev,
                               const void *x, const int8_t *wq, const float *sw, void *y,
                               cudaStream_t st) {
  auto run = [&](auto elt, auto tok, auto out) {
    using Elt = decltype(elt);
    constexpr int kTok = decltype(tok)::value;
    constexpr bool kOut = decltype(out)::value;
    const Layout lay = linear_layout(s, kTok, dev.num_sms);
    return go(k_linear_gemv<Elt, kTok, kOut>, lay, ctas_for(s.N, dev.num_sms), st, x, wq, sw, y,
              (int)s.T, s.N, s.K, lay, dev.err);
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

// A slot streams its expert's weights by itself, also where another slot has the
// same expert: tiles read them once, but take three or four launches more.  us with
// streams against tiles: 16 experts of 4096 x 1792, 1 / 4 / 16 slots 15.5 / 26.5 /
// 68.7 against 44.2 / 50.6 / 78.9; 8 of 2048 x 4096 15.7 / 24.7 / 57.8 against 41.8 /
// 44.9 / 63.8; 64 of 1024 x 512, 8 / 32 slots 14.4 / 26.7 against 43.4 / 46.3.  The
// weights that slots have in common cost more than that from about 200 MB on: 2
// experts of 4096 x 1792, 8 / 12 / 32 slots 29.8 / 40.3 / 86.6 against 43.0 / 43.4 /
// 42.0 (132, 220, 660 MB); 8 experts, 16 / 24 slots 52.0 / 95.5 against 58.1 / 60.5
// (176, 352 MB); 1 of 2048 x 4096, 8 / 12 slots 31.8 / 44.6 against 38.9 / 38.7 (176,
// 277 MB).
constexpr int64_t kGemvAgain = 200'000'000;
bool experts_gemv_ok(const ExpertShape &s, int num_sms) {
  if (s.slots() > kGemvSlots || s.slots() * s.f * 2 > 0x7fffffffLL ||
      s.slots() * s.d > 0x7fffffffLL)
    return false;
  const int64_t again = s.slots() - (s.slots() < s.E ? s.slots() : s.E);
  if (again * 3 * s.d * s.f > kGemvAgain) return false;
  return gateup_layout(s, num_sms).total <= kSmemMost &&
         down_layout(s, num_sms).total <= kSmemMost;
}

cudaError_t launch_experts_gemv_gateup(const ExpertShape &s, const DeviceInfo &dev, const void *x,
                                       const int32_t *experts, const int8_t *Wg, const float *sg,
                                       const int8_t *Wu, const float *su, uint16_t *h,
                                       cudaStream_t st) {
  const Layout lay = gateup_layout(s, dev.num_sms);
  return go(k_experts_gateup, lay, ctas_for(s.slots() * s.f, dev.num_sms), st, x,
            experts, Wg, sg, Wu, su, h, (int)s.T, s.E, s.k, s.d, s.f, lay, dev.err);
}

cudaError_t launch_experts_gemv_down(const ExpertShape &s, const DeviceInfo &dev,
                                     const uint16_t *h, const int32_t *experts,
                                     const float *weights, const int8_t *Wd, const float *sd,
                                     uint16_t *y, cudaStream_t st) {
  const Layout lay = down_layout(s, dev.num_sms);
  return go(k_experts_down, lay, ctas_for(s.T * s.d, dev.num_sms), st, h, experts,
            weights, Wd, sd, y, (int)s.T, s.E, s.k, s.d, s.f, lay, dev.err);
}

}  // namespace sfn
