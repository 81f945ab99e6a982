// tc_i8.cu -- products in 8-bit integers on the 5th-generation tensor cores
// (tcgen05.mma kind::i8: s8 x s8 -> s32), with a scale for each token and each
// output channel applied in the epilogue:
//
//   acc[t][n] = sum_k xq[t][k] wq[n][k]          exact in 32 bits
//   scale    y[t][n] = sx[t] sw[n] acc[t][n]
//   SwiGLU   g, u as above with two weight matrices, h = bf16(silu(g) u)
//
// The rows may be grouped (rows of expert e against expert e's weights): the
// same kernel serves one weight matrix and a whole set of experts, which
// differ in how a unit number becomes a tile.
//
// The weights are the MMA's A operand (128 output channels a CTA) and the
// tokens its B operand, whose width N is any multiple of 16: a tile of a few
// rows costs the weight bytes it must stream and little else, and the ragged
// end of an expert's rows wastes at most 15 columns.
//
// One warp-specialised kernel (one CTA per SM):
//   warp 0      TMA producer: 128-byte K slices (128-byte swizzle) of the
//               weight tile(s) and of the rows into a ring of stages
//   warp 1      allocates 512 TMEM columns; one thread issues the MMAs
//   warps 2...  epilogue, two or four per TMEM lane quadrant (32 channels):
//               lane = channel, register = row; a store writes 32 neighbouring
//               channels of one row
// in three forms:
//   kOne    a CTA per tile, persistent over tiles
//   kPair   a cluster of two CTAs per tile of 256 channels (cta_group::2):
//           each loads its own 128 channels and half of the rows.  What bounds
//           large products is the bytes an SM takes from L2: a 128 x 256 tile
//           on its own takes 48 KB a slice, half a pair's 256 x 256 tile 32 KB.
//   kSplit  for few tiles (few tokens): the CTAs of a cluster take a share of
//           the K slices of one tile each and add the partial sums up through
//           each other's shared memory, so that the weight stream has every
//           SM's copies in flight.
// The weights do not depend on the kernel before this one (which quantises the
// rows), so the ring's first stages of weights are loaded before the wait for
// it.  Every mbarrier wait is bounded (async_util.cuh).
#include "experts.cuh"
#include "tc_util.cuh"

#include <cudaTypedefs.h>

#include <type_traits>

namespace sfn {
namespace {

enum class Span { kOne, kPair, kSplit };
// What the scaled product is stored as.
enum class Out { kF32, kBF16 };

constexpr int kTileN = 128;                    // output channels per CTA (UMMA M, half of a pair's)
constexpr int kSliceK = 128;                   // K bytes per stage
constexpr uint32_t kTileBytes = kTileN * kSliceK;
constexpr int kTmemCols = 512;
constexpr int kRaster = 16;                    // row tiles of a rasterisation group
constexpr size_t kMaxDynSmem = 232448;
constexpr int kMaxStages = 12;
constexpr int kMaxSplit = 8;                   // CTAs of a split tile (portable cluster size)

struct I8Params {
  int64_t rows;            // one weight matrix: its rows
  const int32_t *offsets;  // grouped: row ranges of the groups; null: one group, [0, rows)
  int groups;
  int n;                   // output channels (weight rows) per group
  int tiles_n;             // tiles of 128 (a pair: 256) channels
  int k_slices;
  int bn;                  // most rows per tile
  int box;                 // rows per TMA box
  int stages;
  uint32_t stage_bytes;
  int bufs;                // accumulators (of kTmemCols / bufs columns)
  bool early;              // the weights and offsets are there before the previous kernel's end
  const float *sx, *sw, *sw2;
  void *out;               // [rows][n]
  unsigned *err;
};

// ------------------------------------------------------------- PTX wrappers
// D (+)= A B^T, s8 x s8 -> s32.
template <bool kPair>
__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// As umma_commit; of a pair, the barrier at the same place in both CTAs.
template <bool kPair>
__device__ __forceinline__ void commit_to(uint64_t *bar) {
  if constexpr (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    umma_commit(bar);
}

// As umma_commit, after a pair's MMAs too.
template <bool kPair>
__device__ __forceinline__ void commit_own(uint64_t *bar) {
  if constexpr (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_u32(bar))
        : "memory");
  else
    umma_commit(bar);
}

template <bool kPair>
__device__ __forceinline__ void tmem_take(uint32_t *slot) {
  if constexpr (kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(slot, kTmemCols);
  }
}
template <bool kPair>
__device__ __forceinline__ void tmem_give(uint32_t base) {
  if constexpr (kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base),
                 "r"(kTmemCols)
                 : "memory");
  else
    tmem_dealloc(base, kTmemCols);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared `p` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t at_rank(const void *p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
// Relaxed: what the arrival tells is that TMEM was read (tc_fence_before
// orders that); a release would wait for the thread's global stores too.
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}
__device__ __forceinline__ int4 ld_cluster16(uint32_t cluster_addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(cluster_addr));
  return v;
}

// tma_load_2d whose bytes complete on the barrier at `bar` (a shared::cluster
// address), in this CTA or the other of its pair.
template <bool kPair>
__device__ __forceinline__ void load_tile(void *dst, const CUtensorMap *map, int c0, int c1,
                                          uint32_t bar) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx"
        "::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// Instruction descriptor (format in tc_util.cuh): D s32 (2), A and B s8 (1),
// both K-major.
__device__ __forceinline__ uint32_t idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// One output tile: channels from ch0 on of group g, rows [row0, row1).
struct Tile {
  int g, ch0, width;  // width: rows rounded up to the MMA's multiple
  int row0, row1;
};

// Unit numbers -> tiles, in increasing order.  Within a group the row tiles
// are of even size, and neighbouring units share a weight tile; kRaster row
// tiles at a time, so that a long group's rows stay in L2.
template <int kChannels, int kStep>
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
    const int per = ((count + tiles - 1) / tiles + kStep - 1) / kStep * kStep;
    t.g = g;
    t.ch0 = nb * kChannels;
    t.row0 = first + min(count, mb * per);
    t.row1 = first + min(count, (mb + 1) * per);
    // rounding up may leave the last tile no rows: an empty tile of one step
    t.width = max(kStep, (t.row1 - t.row0 + kStep - 1) / kStep * kStep);
    return true;
  }
};

__device__ __forceinline__ uint16_t bf16_bits(float f) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(f));
  return r;
}

// Epilogue warps: 16 where a wide SwiGLU tile takes all of TMEM, so that the
// MMAs wait for half as long (64 experts of 4096 x 1792 with 128 rows each: 346
// us against 357 with 8), else 8 (8 rows an expert: 235 us against 241 with 16).
template <bool kSwiGlu, Span kSpan>
constexpr int epi_warps() {
  return kSwiGlu && kSpan == Span::kPair ? 16 : 8;
}
template <bool kSwiGlu, Span kSpan>
constexpr int block_threads() {
  return (2 + epi_warps<kSwiGlu, kSpan>()) * 32;
}

template <Out kOut>
__device__ __forceinline__ auto out_value(float y) {
  if constexpr (kOut == Out::kBF16)
    return bf16_bits(y);
  else
    return y;
}

// The epilogue's stores of a lane's channel for 32 rows (n of them; sx: of the
// lane's row), with scaled_sum(); rare.
struct Chunk {
  uint32_t v[32];
};
template <bool kSwiGlu, Out kOut, class Elt>
__device__ __noinline__ void store_scaled(Chunk v, Chunk u, float sx, float sw, float sw2,
                                          Elt *dst, int stride, int n) {
#pragma unroll 1
  for (int i = 0; i < 32; ++i, dst += stride) {
    const float a = __shfl_sync(kFull, sx, i), x = scaled_sum((float)(int)v.v[i], a, sw);
    Elt y;
    if constexpr (kSwiGlu)
      y = bf16_bits(swiglu_f32(x, scaled_sum((float)(int)u.v[i], a, sw2)));
    else
      y = out_value<kOut>(x);
    if (i < n) *dst = y;
  }
}

template <bool kSwiGlu, Out kOut, Span kSpan>
__global__ void __launch_bounds__((block_threads<kSwiGlu, kSpan>()), 1)
    k_i8_gemm(const __grid_constant__ CUtensorMap tX, const __grid_constant__ CUtensorMap tW,
              const __grid_constant__ CUtensorMap tW2, const I8Params p) {
  constexpr bool kPair = kSpan == Span::kPair, kSplit = kSpan == Span::kSplit;
  static_assert(!(kSplit && kSwiGlu), "the split form has the scaled product only");
  constexpr int kNumW = kSwiGlu ? 2 : 1;
  constexpr int kEpiWarps = epi_warps<kSwiGlu, kSpan>(), kThreads = (2 + kEpiWarps) * 32;
  constexpr int kEpiParts = kEpiWarps / 4;          // warps per TMEM lane quadrant
  constexpr int kEpiChunks = 256 / 32 / kEpiParts;  // most 32-row chunks of a warp
  using Walk = TileWalk<kPair ? 2 * kTileN : kTileN, kPair ? 32 : 16>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + (size_t)p.stages * p.stage_bytes);
  uint64_t *full = bars, *empty = bars + kMaxStages;
  uint64_t *tfull = bars + 2 * kMaxStages, *tempty = tfull + 2, *done = tempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  int *offs = reinterpret_cast<int *>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kSpan == Span::kOne ? 0u : cluster_rank();
  const uint32_t ctas = kSpan == Span::kOne ? 1u : cluster_size();
  const bool leader = !kPair || rank == 0u;  // issues the MMAs
  const int first_unit = (int)(blockIdx.x / ctas), unit_step = (int)(gridDim.x / ctas);
  // this CTA's K slices
  const int kb0 = kSplit ? (int)(p.k_slices * rank / ctas) : 0;
  const int kb1 = kSplit ? (int)(p.k_slices * (rank + 1) / ctas) : p.k_slices;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kEpiWarps * (kPair ? 2 : 1));
    }
    mbar_init(done, 1);
    fence_barrier_init();
  }
  if (warp == 1) tmem_take<kPair>(tmem_slot);
  if (!p.early) {
    pdl_wait();
    pdl_launch_dependents();
  }
  if (p.offsets)
    for (int i = threadIdx.x; i <= p.groups; i += kThreads) offs[i] = p.offsets[i];
  tc_fence_before();
  if (kSpan == Span::kOne)
    __syncthreads();
  else
    cluster_sync();  // the other CTAs' barriers are initialised too
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t acc_cols = kTmemCols / p.bufs;

  if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&tX);
      prefetch_tmap(&tW);
      if (kSwiGlu) prefetch_tmap(&tW2);
      // One thread feeds the ring, so its own time per slice counts: stage,
      // phase and coordinates are carried along, with no division by a
      // variable in the loop (with them a slice took 0.23 us of this thread,
      // more than its copies).
      Walk walk;
      Tile t;
      uint32_t s = 0, phase = 1;  // phase: parity that frees the stage (first pass: free)
      uint32_t used = 0;          // stages loaded at least once
      bool ok = true, first = true;
      auto bar_of = [&](uint32_t i) { return kPair ? at_rank(&full[i], 0) : smem_u32(&full[i]); };
      const uint32_t bar0 = bar_of(0);
      for (int unit = first_unit; ok && walk.at(unit, p, offs, t); unit += unit_step) {
        const int rows = kPair ? t.width / 2 : t.width;
        const int row0 = t.row0 + (kPair ? (int)rank * rows : 0);
        const int wrow = t.g * p.n + t.ch0 + (kPair ? (int)rank * kTileN : 0);
        const int boxes = (rows + p.box - 1) / p.box;
        const uint32_t tx = (kPair ? 2u : 1u) *
                            (kNumW * kTileBytes + (uint32_t)(boxes * p.box * kSliceK));
        auto load_weights = [&](uint32_t i, int k) {
          unsigned char *st = smem + (size_t)i * p.stage_bytes;
          if (leader) mbar_arrive_expect_tx(&full[i], tx);
          load_tile<kPair>(st, &tW, k, wrow, bar0 + i * 8u);
          if (kSwiGlu) load_tile<kPair>(st + kTileBytes, &tW2, k, wrow, bar0 + i * 8u);
        };
        int ahead = kb0;  // slices below this have their weights under way
        if (first && p.early) {
          ahead = min(kb1, kb0 + p.stages);
          for (int kb = kb0; kb < ahead; ++kb) load_weights(kb - kb0, kb * kSliceK);
          pdl_wait();
        }
        first = false;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (kb >= ahead) {
            if (!mbar_wait(&empty[s], phase, p.err)) {
              ok = false;
              break;
            }
            load_weights(s, kb * kSliceK);
          }
          unsigned char *b = smem + (size_t)s * p.stage_bytes + kNumW * kTileBytes;
          for (int q = 0; q < rows; q += p.box)
            load_tile<kPair>(b + (size_t)q * kSliceK, &tX, kb * kSliceK, row0 + q, bar0 + s * 8u);
          if (++s == (uint32_t)p.stages) {
            s = 0;
            phase ^= 1u;
          }
          used = max(used, s == 0 ? (uint32_t)p.stages : s);
        }
      }
      // before this CTA ends, the last load of every stage has landed; of a
      // pair, both CTAs' loads complete on the leader's barriers, and the
      // other CTA waits for the last signals of the leader's MMAs to its own.
      // Stages before s were last used in the pass that s is in (its `full`
      // parity is the opposite of `phase`), the others in the one before.
      for (uint32_t i = 0; i < used; ++i)
        mbar_wait(leader ? &full[i] : &empty[i], i < s ? phase ^ 1u : phase, p.err);
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      Walk walk;
      Tile t;
      uint32_t s = 0, phase = 0;       // of the ring
      uint32_t acc = 0, acc_phase = 1;  // of the accumulators (free at first)
      bool ok = true;
      for (int unit = first_unit; ok && walk.at(unit, p, offs, t); unit += unit_step) {
        if (!mbar_wait(&tempty[acc], acc_phase, p.err)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + acc * acc_cols;
        const uint32_t idesc = idesc_i8(kPair ? 2 * kTileN : kTileN, t.width);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&full[s], phase, p.err)) {
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
            const uint32_t more = (kb > kb0 || kk > 0) ? 1u : 0u;
            umma_i8<kPair>(d, w + kk * 2, x + kk * 2, idesc, more);
            if (kSwiGlu) umma_i8<kPair>(d + acc_cols / 2, w2 + kk * 2, x + kk * 2, idesc, more);
          }
          commit_to<kPair>(&empty[s]);
          if (++s == (uint32_t)p.stages) {
            s = 0;
            phase ^= 1u;
          }
        }
        if (ok) commit_to<kPair>(&tfull[acc]);
        if (++acc == (uint32_t)p.bufs) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      commit_own<kPair>(done);
      mbar_wait(done, 0, p.err);
    }
  } else {
    // every CTA waits here, so that this kernel never ends before the one
    // that it follows
    if (p.early) {
      pdl_wait();
      pdl_launch_dependents();
    }
    const int q = warp & 3;              // TMEM lane quadrant: channels 32 q ..
    const int part = (warp - 2) >> 2;    // which of the quadrant's warps
    Walk walk;
    Tile t;
    uint32_t lt = 0;
    for (int unit = first_unit; walk.at(unit, p, offs, t); unit += unit_step, ++lt) {
      const uint32_t acc = lt % p.bufs, use = lt / p.bufs;
      const int ch = t.ch0 + (kPair ? (int)rank * kTileN : 0) + q * 32 + lane;
      const bool valid = ch < p.n;
      const int64_t wch = (int64_t)t.g * p.n + ch;
      const float sw = valid ? __ldg(p.sw + wch) : 0.f;
      const float sw2 = (kSwiGlu && valid) ? __ldg(p.sw2 + wch) : 0.f;
      // the rows' scales, before the wait for the tile
      const int rows = t.row1 - t.row0;
      float sx[kEpiChunks];
      if constexpr (!kSplit) {
#pragma unroll
        for (int j = 0; j < kEpiChunks; ++j) {
          const int r = 32 * (part + j * kEpiParts) + lane;
          sx[j] = r < rows ? p.sx[t.row0 + r] : 0.f;
        }
      }
      if (!mbar_wait(&tfull[acc], use & 1u, p.err)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * acc_cols;
      // the accumulator is free once it is in registers
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (kPair)
            arrive_at(at_rank(&tempty[acc], 0));
          else
            mbar_arrive(&tempty[acc]);
        }
      };
      if (32 * part >= rows) release();
#pragma unroll
      for (int j = 0; j < kEpiChunks; ++j) {
        const int c0 = 32 * (part + j * kEpiParts);
        if (c0 >= rows) break;
        const int row = t.row0 + c0;
        const int nr = min(32, rows - c0);
        uint32_t v[32];
        tmem_ld_32x32b_x32(taddr + c0, v);
        uint32_t u[kSwiGlu ? 32 : 1];
        if constexpr (kSwiGlu) tmem_ld_32x32b_x32(taddr + acc_cols / 2 + c0, u);
        tmem_ld_wait();
        if (c0 + 32 * kEpiParts >= rows) release();
        if constexpr (kSplit) {
          // partial sums [row][channel] over the ring, whose loads and MMAs
          // are all complete
          int *sums = reinterpret_cast<int *>(smem) + (size_t)c0 * kTileN + q * 32 + lane;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < nr) sums[i * kTileN] = (int)v[i];
          continue;
        }
        using Elt = std::conditional_t<kOut == Out::kF32, float, uint16_t>;
        Elt *dst = static_cast<Elt *>(p.out) + (int64_t)row * p.n + ch;
        // a row of the chunk whose scale may take an integer sum (at most 2^31) past
        // the range: not here (with the test in these loops, or beside them a third,
        // a short product takes 7 % more)
        if (__any_sync(kFull, fabsf(sx[j]) > 0x1p96f)) {
          Chunk first, second;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            first.v[i] = v[i];
            second.v[i] = kSwiGlu ? u[kSwiGlu ? i : 0] : 0u;
          }
          store_scaled<kSwiGlu, kOut>(first, second, sx[j], sw, sw2, dst, p.n, valid ? nr : 0);
          continue;
        }
        auto value = [&](int i) -> Elt {
          const float x = (float)(int)v[i];
          if constexpr (kSwiGlu) {
            const float a = __shfl_sync(kFull, sx[j], i);
            const float g = x * a * sw, up = (float)(int)u[i] * a * sw2;
            return bf16_bits(swiglu_f32(g, up));
          } else {
            return out_value<kOut>(x * __shfl_sync(kFull, sx[j], i) * sw);
          }
        };
        if (nr == 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i, dst += p.n) {
            const Elt y = value(i);
            if (valid) *dst = y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i, dst += p.n) {
            const Elt y = value(i);
            if (valid && i < nr) *dst = y;
          }
        }
      }
    }
  }

  if constexpr (kSplit) {
    // one tile per cluster: this CTA sums its share of the tile's rows
    cluster_sync();
    pdl_wait();
    Walk walk;
    Tile t;
    if (walk.at(first_unit, p, offs, t)) {
      const int rows = t.row1 - t.row0;
      const int r0 = (int)(rows * rank / ctas), r1 = (int)(rows * (rank + 1) / ctas);
      const int chans = min(kTileN, p.n - t.ch0);
      for (int i = threadIdx.x; i < (r1 - r0) * (kTileN / 4); i += kThreads) {
        const int r = r0 + i / (kTileN / 4), c = i % (kTileN / 4) * 4;
        const uint32_t mine = smem_u32(smem) + (uint32_t)(r * kTileN + c) * 4u;
        int4 sum = make_int4(0, 0, 0, 0);
        for (uint32_t k = 0; k < ctas; ++k) {
          uint32_t a;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(mine), "r"(k));
          const int4 v = ld_cluster16(a);
          sum.x += v.x;
          sum.y += v.y;
          sum.z += v.z;
          sum.w += v.w;
        }
        const float sx = p.sx[t.row0 + r];
        const int acc4[4] = {sum.x, sum.y, sum.z, sum.w};
        const int64_t o = (int64_t)(t.row0 + r) * p.n + t.ch0 + c;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c + j < chans) {
            const float y = scaled_sum((float)acc4[j], sx, __ldg(p.sw + t.ch0 + c + j));
            using Elt = decltype(out_value<kOut>(y));
            static_cast<Elt *>(p.out)[o + j] = out_value<kOut>(y);
          }
      }
    }
  }
  if (kSpan == Span::kOne)
    __syncthreads();
  else
    cluster_sync();  // nothing of this CTA is read or signalled any more
  if (warp == 1) {
    tc_fence_after();
    tmem_give<kPair>(tmem_base);
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

// Stages of the ring and the kernel's shared memory.
size_t ring(I8Params &p) {
  // alignment slack, barriers, the groups' offsets
  const size_t fixed = 1024 + (2 * kMaxStages + 5) * 8 + 16 +
                       (p.offsets ? (size_t)(p.groups + 1) * sizeof(int) : 0);
  p.stages = (int)((kMaxDynSmem - fixed) / p.stage_bytes);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  return fixed + (size_t)p.stages * p.stage_bytes;
}

// cluster: CTAs per cluster; units: an upper bound on the number of tiles.
template <bool kSwiGlu, Out kOut, Span kSpan>
cudaError_t launch(const CUtensorMap &tX, const CUtensorMap &tW, const CUtensorMap &tW2,
                   I8Params p, int64_t units, int cluster, int num_sms, cudaStream_t st) {
  const size_t smem = ring(p);
  if (p.stages < 2) return cudaErrorInvalidValue;
  auto kern = k_i8_gemm<kSwiGlu, kOut, kSpan>;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kern), smem);
  if (e != cudaSuccess) return e;
  constexpr int kThreads = block_threads<kSwiGlu, kSpan>();
  const int most = num_sms / cluster;
  const int grid = (int)(kSpan == Span::kSplit || units < most ? units : most) * cluster;
  count_launches(1);
  if (cluster == 1)
    return launch_pdl(kern, dim3(grid), dim3(kThreads), smem, st, tX, tW, tW2, p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, tX, tW, tW2, p);
}

// How a product is tiled.
struct Tiling {
  bool pair;
  int bn, box, split;
};

// Rows per tile: even tiles of at most `most`, a multiple of `step`; and rows
// per TMA box.  Of one matrix the tiles are all alike and the box is a CTA's
// rows; of a group's rows, whose number is known on the device only, at most
// 64, so that a ragged tile loads no more than 63 rows past its end.
Tiling tile_rows(int64_t rows, int most, bool pair, bool grouped) {
  const int step = pair ? 32 : 16, halves = pair ? 2 : 1;
  const int64_t tiles = (rows + most - 1) / most;
  Tiling t{pair, (int)(((rows + tiles - 1) / tiles + step - 1) / step * step), 0, 1};
  t.box = t.bn / halves;
  if (grouped && t.box > 64) {
    t.box = 64;
    t.bn = (t.bn + 64 * halves - 1) / (64 * halves) * (64 * halves);
  }
  return t;
}

I8Params params(const Tiling &t, int n, int k, int num_w, unsigned *err) {
  I8Params p{};
  const int channels = t.pair ? 2 * kTileN : kTileN;
  p.groups = 1;
  p.n = n;
  p.tiles_n = (n + channels - 1) / channels;
  p.k_slices = (k + kSliceK - 1) / kSliceK;
  p.bn = t.bn;
  p.box = t.box;
  p.stage_bytes = num_w * kTileBytes + (uint32_t)(t.pair ? t.bn / 2 : t.bn) * kSliceK;
  p.bufs = num_w * t.bn <= kTmemCols / 2 ? 2 : 1;
  p.err = err;
  return p;
}

// The tiling of one matrix product that a simple cost says is the cheapest:
// waves of CTAs x (slices x time per slice + epilogue), in us.  Measured per
// slice with every SM busy: 0.43 us for 256 rows a tile, 0.34 for 128, 0.31 for
// 64 and below (what an SM takes from L2 bounds it: 48, 32, 24 KB); a split
// tile's sum costs about 2 us.  Against every other choice on 5 to 4096 tokens
// of 4096 x 14336 and 14336 x 4096 it takes the best or one within 4 %.
Tiling choose_tiling(const I8Shape &s, int num_sms) {
  // Pairs take a third less from L2 and pay a barrier between two SMs: 172 us
  // against 178 for 4096 tokens of 4096 x 14336 (12 waves), but 48 against 47
  // for 1024 tokens of 14336 x 4096 (one).
  const int64_t pair_tiles = ((s.T + 255) / 256) * (((int64_t)s.N + 255) / 256);
  if (s.T >= 2048 && 2 * pair_tiles >= 3 * (int64_t)num_sms) return tile_rows(s.T, 256, true, false);
  const int64_t channels = ((int64_t)s.N + kTileN - 1) / kTileN;
  const int slices = (s.K + kSliceK - 1) / kSliceK;
  Tiling best{};
  float best_us = 0.f;
  for (int most : {64, 128, 256}) {
    if (most > 64 && s.T <= most / 2) break;
    Tiling t = tile_rows(s.T, most, false, false);
    const int64_t tiles = ((s.T + t.bn - 1) / t.bn) * channels;
    const float slice_us = t.bn <= 64 ? 0.31f : 0.25f + 0.0007f * (float)t.bn;
    for (int split = 1; split <= kMaxSplit; split *= 2) {
      // clusters do not fill every SM: leave an eighth
      if (split > 1 && (tiles * split > num_sms * 7 / 8 || slices < 4 * split)) break;
      const float waves = (float)((tiles * split + num_sms - 1) / num_sms);
      const float us = waves * ((float)((slices + split - 1) / split) * slice_us +
                                0.004f * (float)t.bn) + (split > 1 ? 2.f : 0.f);
      if (best.bn == 0 || us < best_us) {
        best = t;
        best.split = split;
        best_us = us;
      }
    }
  }
  return best;
}
}  // namespace

cudaError_t launch_i8_gemm(const I8Shape &s, const DeviceInfo &dev, const int8_t *xq,
                           const float *sx, const int8_t *wq, const float *sw, void *y,
                           bool weights_early, cudaStream_t st) {
  const Tiling t = choose_tiling(s, dev.num_sms);
  I8Params p = params(t, s.N, s.K, 1, dev.err);
  p.rows = s.T;
  p.early = weights_early;
  p.sx = sx;
  p.sw = sw;
  p.out = y;
  CUtensorMap mX, mW;
  if (!map_i8(&mX, xq, (uint64_t)s.K, (uint64_t)s.T, (uint32_t)p.box) ||
      !map_i8(&mW, wq, (uint64_t)s.K, (uint64_t)s.N, kTileN))
    return cudaErrorInvalidValue;
  const int64_t units = (s.T + p.bn - 1) / p.bn * p.tiles_n;
  auto go = [&](auto out) {
    constexpr Out kOut = decltype(out)::value;
    if (t.pair)
      return launch<false, kOut, Span::kPair>(mX, mW, mW, p, units, 2, dev.num_sms, st);
    if (t.split > 1)
      return launch<false, kOut, Span::kSplit>(mX, mW, mW, p, units, t.split, dev.num_sms, st);
    return launch<false, kOut, Span::kOne>(mX, mW, mW, p, units, 1, dev.num_sms, st);
  };
  return s.out_bf16 ? go(std::integral_constant<Out, Out::kBF16>{})
                    : go(std::integral_constant<Out, Out::kF32>{});
}

namespace {
// Tiles of a grouped product (n channels an expert, k long, num_w matrices).
// How many rows an expert has is known on the device only; with few on average
// the tile is as wide as twice the average asks for, so that a decode batch does
// not pay for a prefill's stages and seldom reads an expert's weights twice.
// With 64 and more, pairs of 256 rows where they run long and fill the SMs one
// and a half times: of 64 experts of 4096 x 1792, 128 rows each, 346 us against
// 356 (SwiGLU) and 347 (down) with one CTA a tile; but single CTAs of 128 rows
// (SwiGLU) or 256 (down), or of 64 where those would not fill half of the SMs, for
// short products and few tiles: 64 experts of 576 x 416, 150 rows, 74 against 83
// us; 8 of 2048 x 1024, 128 rows, 40 against 44; 2 of 1712 x 224, 960 rows, 35 against
// 41.
Tiling grouped_tiling(const ExpertShape &s, int n, int k, int num_w, int num_sms) {
  const int64_t slots = s.slots(), rows = slots / s.E;
  if (rows < 32) return tile_rows(2 * rows + 16, 256, false, true);
  if (rows < 64) return tile_rows(num_w == 2 ? 64 : 2 * rows + 16, 256, false, true);
  auto tiles = [&](int bn, int channels) {  // about: an expert's last tile is half full
    const int64_t used = slots < s.E ? slots : s.E;
    return used * (2 * rows + bn) / (2 * bn) * ((n + channels - 1) / channels);
  };
  const int slices = (k + kSliceK - 1) / kSliceK;
  if (slices >= 8 && 4 * tiles(256, 2 * kTileN) >= 3 * num_sms) return tile_rows(256, 256, true, true);
  const int wide = num_w == 2 ? 128 : 256;
  return tile_rows(2 * tiles(wide, kTileN) >= num_sms ? wide : 64, 256, false, true);
}
template <bool kSwiGlu, Out kOut>
cudaError_t launch_grouped(const CUtensorMap &mX, const CUtensorMap &mW, const CUtensorMap &mW2,
                           const Tiling &t, const I8Params &p, int num_sms, cudaStream_t st) {
  const int64_t units = (int64_t)p.groups * p.tiles_n + p.rows;
  return t.pair ? launch<kSwiGlu, kOut, Span::kPair>(mX, mW, mW2, p, units, 2, num_sms, st)
                : launch<kSwiGlu, kOut, Span::kOne>(mX, mW, mW2, p, units, 1, num_sms, st);
}
}  // namespace

cudaError_t launch_i8_experts_gateup(const ExpertShape &s, const DeviceInfo &dev,
                                     const int32_t *offsets, const int8_t *xq, const float *sx,
                                     const int8_t *Wg, const float *sg, const int8_t *Wu,
                                     const float *su, uint16_t *h, cudaStream_t st) {
  const Tiling t = grouped_tiling(s, s.f, s.d, 2, dev.num_sms);
  I8Params p = params(t, s.f, s.d, 2, dev.err);
  p.rows = s.slots();
  p.offsets = offsets;
  p.groups = s.E;
  p.early = true;
  p.sx = sx;
  p.sw = sg;
  p.sw2 = su;
  p.out = h;
  CUtensorMap mX, mG, mU;
  if (!map_i8(&mX, xq, (uint64_t)s.d, (uint64_t)s.slots(), (uint32_t)p.box) ||
      !map_i8(&mG, Wg, (uint64_t)s.d, (uint64_t)s.E * s.f, kTileN) ||
      !map_i8(&mU, Wu, (uint64_t)s.d, (uint64_t)s.E * s.f, kTileN))
    return cudaErrorInvalidValue;
  return launch_grouped<true, Out::kBF16>(mX, mG, mU, t, p, dev.num_sms, st);
}

cudaError_t launch_i8_experts_down(const ExpertShape &s, const DeviceInfo &dev,
                                   const int32_t *offsets, const int8_t *hq, const float *sh,
                                   const int8_t *Wd, const float *sd, float *o,
                                   cudaStream_t st) {
  const Tiling t = grouped_tiling(s, s.d, s.f, 1, dev.num_sms);
  I8Params p = params(t, s.d, s.f, 1, dev.err);
  p.rows = s.slots();
  p.offsets = offsets;
  p.groups = s.E;
  p.early = true;
  p.sx = sh;
  p.sw = sd;
  p.out = o;
  CUtensorMap mX, mW;
  if (!map_i8(&mX, hq, (uint64_t)s.f, (uint64_t)s.slots(), (uint32_t)p.box) ||
      !map_i8(&mW, Wd, (uint64_t)s.f, (uint64_t)s.E * s.d, kTileN))
    return cudaErrorInvalidValue;
  return launch_grouped<false, Out::kF32>(mX, mW, mW, t, p, dev.num_sms, st);
}

}  // namespace sfn
