// tc_i8.cu -- products in 8-bit integers on the 5th-generation tensor cores
// (tcgen05.mma kind::i8: s8 x s8 -> s32), with a scale for each token and each
// output channel applied in the epilogue:
//
//   acc[t][n] = sum_k xq[t][k] wq[n][k]          exact in 32 bits
//   kScale   y[t][n] = sx[t] sw[n] acc[t][n]
//   kSwiGlu  g, u as above with two weight matrices, h = bf16(silu(g) u)
//
// The rows may be grouped (rows of expert e against expert e's weights): the
// same kernel serves one weight matrix and a whole set of experts, which
// differ in how a unit number becomes a tile.
//
// The weights are the MMA's A operand (128 output channels a tile) and the
// tokens its B operand, whose width N is any multiple of 16: a tile of a few
// rows costs the weight bytes it must stream and little else, and the ragged
// end of an expert's rows wastes at most 15 columns.
//
// One persistent, warp-specialised kernel (one CTA per SM):
//   warp 0      TMA producer: 128-byte K slices (128-byte swizzle) of the
//               weight tile(s) and of the rows into a ring of stages
//   warp 1      allocates 512 TMEM columns; one thread issues the MMAs
//               (M 128, K 32) into one of two accumulators
//   warps 2..9  epilogue, two per TMEM lane quadrant (32 channels): lane =
//               channel, register = row; a store writes 32 neighbouring
//               channels of one row
// Every mbarrier wait is bounded (async_util.cuh).
#include "experts.cuh"
#include "tc_util.cuh"

#include <cudaTypedefs.h>

namespace sfn {
namespace {

constexpr int kTileN = 128;                    // output channels per tile (UMMA M)
constexpr int kSliceK = 128;                   // K bytes per stage
constexpr uint32_t kTileBytes = kTileN * kSliceK;
constexpr int kAccCols = 256;                  // TMEM columns per accumulator
constexpr int kRaster = 16;                    // row tiles of a rasterisation group
constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr size_t kMaxDynSmem = 232448;
constexpr int kMaxStages = 12;

struct I8Params {
  int64_t rows;            // one weight matrix: its rows
  const int32_t *offsets;  // grouped: row ranges of the groups; null: one group, [0, rows)
  int groups;
  int n;                   // output channels (weight rows) per group
  int tiles_n;             // ceil(n / 128)
  int k_slices;
  int bn;                  // most rows per tile
  int box;                 // rows per TMA box (divides bn)
  int stages;
  uint32_t stage_bytes;
  const float *sx, *sw, *sw2;
  void *out;               // [rows][n]
  unsigned *err;
};

// D (+)= A B^T, s8 x s8 -> s32.
__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor (format in tc_util.cuh): D s32 (2), A and B s8 (1),
// both K-major.
__device__ __forceinline__ uint32_t idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// One output tile: channels [ch0, ch0 + 128) of group g, rows [row0, row1).
struct Tile {
  int g, ch0, width;  // width: rows rounded up to the MMA's multiple of 16
  int row0, row1;
};

// Unit numbers -> tiles, in increasing order.  Within a group the row tiles
// are of even size, and neighbouring units share a weight tile; kRaster row
// tiles at a time, so that a long group's rows stay in L2.
struct TileWalk {
  int g = -1;
  int begin = 0, end = 0, tiles = 0, first = 0, count = 0;
  __device__ __forceinline__ bool at(int unit, const I8Params &p, const int *offs, Tile &t) {
    while (unit >= end) {
      if (++g >= p.groups) return false;
      first = p.offsets ? offs[g] : 0;
      count = p.offsets ? offs[g + 1] - first : (int)p.rows;
      tiles = (count + p.bn - 1) / p.bn;
      begin = end;
      end += tiles * p.tiles_n;
    }
    const int idx = unit - begin;
    const int group = idx / (kRaster * p.tiles_n);
    const int r0 = group * kRaster, gm = min(kRaster, tiles - r0);
    const int in = idx - r0 * p.tiles_n;
    const int mb = r0 + in % gm, nb = in / gm;
    const int per = ((count + tiles - 1) / tiles + 15) & ~15;
    t.g = g;
    t.ch0 = nb * kTileN;
    t.row0 = first + min(count, mb * per);
    t.row1 = first + min(count, (mb + 1) * per);
    // rounding up may leave the last tile no rows: an empty tile of 16 columns
    t.width = max(16, (t.row1 - t.row0 + 15) & ~15);
    return true;
  }
};

template <bool kSwiGlu, bool kOutBf16>
__global__ void __launch_bounds__(kThreads, 1)
    k_i8_gemm(const __grid_constant__ CUtensorMap tX, const __grid_constant__ CUtensorMap tW,
              const __grid_constant__ CUtensorMap tW2, const I8Params p) {
  constexpr int kNumW = kSwiGlu ? 2 : 1;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + (size_t)p.stages * p.stage_bytes);
  uint64_t *full = bars, *empty = bars + kMaxStages;
  uint64_t *tfull = bars + 2 * kMaxStages, *tempty = tfull + 2, *done = tempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  int *offs = reinterpret_cast<int *>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kEpiWarps * 32);
    }
    mbar_init(done, 1);
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, 2 * kAccCols);
  pdl_wait();
  pdl_launch_dependents();
  if (p.offsets)
    for (int i = threadIdx.x; i <= p.groups; i += kThreads) offs[i] = p.offsets[i];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&tX);
      prefetch_tmap(&tW);
      if (kSwiGlu) prefetch_tmap(&tW2);
      TileWalk walk;
      Tile t;
      uint32_t it = 0;
      bool ok = true;
      for (int unit = blockIdx.x; ok && walk.at(unit, p, offs, t); unit += gridDim.x) {
        const int boxes = (t.width + p.box - 1) / p.box;
        const uint32_t tx = kNumW * kTileBytes + (uint32_t)(boxes * p.box * kSliceK);
        const int wrow = t.g * p.n + t.ch0;
        for (int kb = 0; kb < p.k_slices; ++kb, ++it) {
          const int s = (int)(it % p.stages);
          const uint32_t use = it / p.stages;
          if (use > 0 && !mbar_wait(&empty[s], (use - 1) & 1u, p.err)) {
            ok = false;
            break;
          }
          unsigned char *st = smem + (size_t)s * p.stage_bytes;
          mbar_arrive_expect_tx(&full[s], tx);
          tma_load_2d(st, &tW, kb * kSliceK, wrow, &full[s]);
          if (kSwiGlu) tma_load_2d(st + kTileBytes, &tW2, kb * kSliceK, wrow, &full[s]);
          unsigned char *b = st + kNumW * kTileBytes;
          for (int q = 0; q < boxes; ++q)
            tma_load_2d(b + (size_t)q * p.box * kSliceK, &tX, kb * kSliceK, t.row0 + q * p.box,
                        &full[s]);
        }
      }
      // the last load of every stage has landed before this CTA ends
      for (int s = 0; s < p.stages && (uint32_t)s < it; ++s) {
        const uint32_t last = s + ((it - 1 - s) / p.stages) * p.stages;
        mbar_wait(&full[s], (last / p.stages) & 1u, p.err);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      TileWalk walk;
      Tile t;
      uint32_t it = 0, lt = 0;
      bool ok = true;
      for (int unit = blockIdx.x; ok && walk.at(unit, p, offs, t); unit += gridDim.x, ++lt) {
        const uint32_t acc = lt & 1u, use = lt >> 1;
        if (use > 0 && !mbar_wait(&tempty[acc], (use - 1) & 1u, p.err)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + acc * kAccCols;
        const uint32_t idesc = idesc_i8(kTileN, t.width);
        for (int kb = 0; kb < p.k_slices; ++kb, ++it) {
          const int s = (int)(it % p.stages);
          if (!mbar_wait(&full[s], (it / p.stages) & 1u, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const unsigned char *st = smem + (size_t)s * p.stage_bytes;
          const uint64_t w = desc_kmajor_sw128(st);
          const uint64_t w2 = desc_kmajor_sw128(st + kTileBytes);
          const uint64_t x = desc_kmajor_sw128(st + kNumW * kTileBytes);
#pragma unroll
          for (int kk = 0; kk < kSliceK / 32; ++kk) {
            const uint32_t more = (kb > 0 || kk > 0) ? 1u : 0u;
            umma_i8(d, w + kk * 2, x + kk * 2, idesc, more);
            if (kSwiGlu) umma_i8(d + kAccCols / 2, w2 + kk * 2, x + kk * 2, idesc, more);
          }
          umma_commit(&empty[s]);
        }
        if (ok) umma_commit(&tfull[acc]);
      }
      umma_commit(done);
      mbar_wait(done, 0, p.err);
    }
  } else {
    const int q = warp & 3;              // TMEM lane quadrant: channels 32 q ..
    const int half = (warp - 2) >> 2;    // which of the quadrant's two warps
    TileWalk walk;
    Tile t;
    uint32_t lt = 0;
    for (int unit = blockIdx.x; walk.at(unit, p, offs, t); unit += gridDim.x, ++lt) {
      const uint32_t acc = lt & 1u, use = lt >> 1;
      const int ch = t.ch0 + q * 32 + lane;
      const bool valid = ch < p.n;
      const int64_t wch = (int64_t)t.g * p.n + ch;
      const float sw = valid ? __ldg(p.sw + wch) : 0.f;
      const float sw2 = (kSwiGlu && valid) ? __ldg(p.sw2 + wch) : 0.f;
      if (!mbar_wait(&tfull[acc], use & 1u, p.err)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * kAccCols;
      for (int c0 = 32 * half; c0 < t.row1 - t.row0; c0 += 64) {
        const int row = t.row0 + c0;
        const int nr = min(32, t.row1 - row);
        const float sx = lane < nr ? p.sx[row + lane] : 0.f;
        uint32_t v[32];
        tmem_ld_32x32b_x32(taddr + c0, v);
        if constexpr (kSwiGlu) {
          uint32_t u[32];
          tmem_ld_32x32b_x32(taddr + kAccCols / 2 + c0, u);
          tmem_ld_wait();
          uint16_t *dst = static_cast<uint16_t *>(p.out) + (int64_t)row * p.n + ch;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float a = __shfl_sync(kFull, sx, i);
            const float g = (float)(int)v[i] * a * sw, uu = (float)(int)u[i] * a * sw2;
            // silu(g) u, rounded once to bf16: the element type the FFN's
            // activations have in this library, and what is requantised
            if (valid && i < nr) dst[(int64_t)i * p.n] = f32_to_bf16_bits(g * sigmoid_f32(g) * uu);
          }
        } else {
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float y = (float)(int)v[i] * __shfl_sync(kFull, sx, i) * sw;
            if (valid && i < nr) {
              const int64_t o = (int64_t)(row + i) * p.n + ch;
              if (kOutBf16)
                static_cast<uint16_t *>(p.out)[o] = f32_to_bf16_bits(y);
              else
                static_cast<float *>(p.out)[o] = y;
            }
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&tempty[acc]);
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 2 * kAccCols);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void *f = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// Row-major 8-bit matrix [rows][k], box {128, box_rows}, 128-byte swizzle,
// zero fill outside.
bool map_i8(CUtensorMap *m, const void *base, uint64_t k, uint64_t rows, uint32_t box_rows) {
  if (encode_fn() == nullptr) return false;
  cuuint64_t dims[2] = {k, rows};
  cuuint64_t strides[1] = {k};
  cuuint32_t box[2] = {kSliceK, box_rows};
  cuuint32_t es[2] = {1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims,
                     strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kSwiGlu, bool kOutBf16>
cudaError_t launch(const CUtensorMap &tX, const CUtensorMap &tW, const CUtensorMap &tW2,
                   I8Params p, int64_t units, int num_sms, cudaStream_t st) {
  p.stage_bytes = (kSwiGlu ? 2 : 1) * kTileBytes + (uint32_t)p.bn * kSliceK;
  // alignment slack, barriers, the groups' offsets
  const size_t fixed = 1024 + (2 * kMaxStages + 5) * 8 + 16 +
                       (p.offsets ? (size_t)(p.groups + 1) * sizeof(int) : 0);
  p.stages = (int)((kMaxDynSmem - fixed) / p.stage_bytes);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  if (p.stages < 2) return cudaErrorInvalidValue;
  const size_t smem = fixed + (size_t)p.stages * p.stage_bytes;
  auto kern = k_i8_gemm<kSwiGlu, kOutBf16>;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kern), smem);
  if (e != cudaSuccess) return e;
  const int grid = (int)(units < num_sms ? units : num_sms);
  count_launches(1);
  return launch_pdl(kern, dim3(grid), dim3(kThreads), smem, st, tX, tW, tW2, p);
}

// Rows per tile: even tiles of at most `most`, a multiple of 16.
int tile_rows(int64_t rows, int most) {
  const int64_t tiles = (rows + most - 1) / most;
  return (int)(((rows + tiles - 1) / tiles + 15) / 16 * 16);
}

// Rows per TMA box: the whole tile up to 64 rows, else 64, so that a ragged
// tile loads no more than 63 rows past its end.
int box_rows(int &bn) {
  if (bn <= 64) return bn;
  bn = (bn + 63) / 64 * 64;
  return 64;
}

}  // namespace

cudaError_t launch_i8_gemm(const I8Shape &s, const DeviceInfo &dev, const int8_t *xq,
                           const float *sx, const int8_t *wq, const float *sw, void *y,
                           cudaStream_t st) {
  I8Params p{};
  p.rows = s.T;
  p.groups = 1;
  p.n = s.N;
  p.tiles_n = (s.N + kTileN - 1) / kTileN;
  p.k_slices = (s.K + kSliceK - 1) / kSliceK;
  p.bn = tile_rows(s.T, 256);
  p.box = box_rows(p.bn);
  p.sx = sx;
  p.sw = sw;
  p.out = y;
  p.err = dev.err;
  CUtensorMap mX, mW;
  if (!map_i8(&mX, xq, (uint64_t)s.K, (uint64_t)s.T, (uint32_t)p.box) ||
      !map_i8(&mW, wq, (uint64_t)s.K, (uint64_t)s.N, kTileN))
    return cudaErrorInvalidValue;
  const int64_t units = (s.T + p.bn - 1) / p.bn * p.tiles_n;
  return s.out_bf16 ? launch<false, true>(mX, mW, mW, p, units, dev.num_sms, st)
                    : launch<false, false>(mX, mW, mW, p, units, dev.num_sms, st);
}

namespace {
// Tiles of the grouped products.  How many rows an expert has is known on the
// device only; the tile is as wide as twice the average asks for, so that a
// decode batch does not pay for a prefill's stages.
I8Params grouped(const ExpertShape &s, const DeviceInfo &dev, const int32_t *offsets, int n,
                 int k, int most) {
  I8Params p{};
  p.rows = s.slots();
  p.offsets = offsets;
  p.groups = s.E;
  p.n = n;
  p.tiles_n = (n + kTileN - 1) / kTileN;
  p.k_slices = (k + kSliceK - 1) / kSliceK;
  const int64_t twice = 2 * s.slots() / s.E + 16;
  p.bn = tile_rows(twice < most ? twice : most, most);
  p.box = box_rows(p.bn);
  p.err = dev.err;
  return p;
}
}  // namespace

cudaError_t launch_i8_experts_gateup(const ExpertShape &s, const DeviceInfo &dev,
                                     const int32_t *offsets, const int8_t *xq, const float *sx,
                                     const int8_t *Wg, const float *sg, const int8_t *Wu,
                                     const float *su, uint16_t *h, cudaStream_t st) {
  I8Params p = grouped(s, dev, offsets, s.f, s.d, 128);
  p.sx = sx;
  p.sw = sg;
  p.sw2 = su;
  p.out = h;
  CUtensorMap mX, mG, mU;
  if (!map_i8(&mX, xq, (uint64_t)s.d, (uint64_t)s.slots(), (uint32_t)p.box) ||
      !map_i8(&mG, Wg, (uint64_t)s.d, (uint64_t)s.E * s.f, kTileN) ||
      !map_i8(&mU, Wu, (uint64_t)s.d, (uint64_t)s.E * s.f, kTileN))
    return cudaErrorInvalidValue;
  return launch<true, true>(mX, mG, mU, p, (int64_t)s.E * p.tiles_n + s.slots(), dev.num_sms, st);
}

cudaError_t launch_i8_experts_down(const ExpertShape &s, const DeviceInfo &dev,
                                   const int32_t *offsets, const int8_t *hq, const float *sh,
                                   const int8_t *Wd, const float *sd, float *o,
                                   cudaStream_t st) {
  I8Params p = grouped(s, dev, offsets, s.d, s.f, 256);
  p.sx = sh;
  p.sw = sd;
  p.out = o;
  CUtensorMap mX, mW;
  if (!map_i8(&mX, hq, (uint64_t)s.f, (uint64_t)s.slots(), (uint32_t)p.box) ||
      !map_i8(&mW, Wd, (uint64_t)s.f, (uint64_t)s.E * s.d, kTileN))
    return cudaErrorInvalidValue;
  return launch<false, false>(mX, mW, mW, p, (int64_t)s.E * p.tiles_n + s.slots(), dev.num_sms,
                              st);
}

}  // namespace sfn
