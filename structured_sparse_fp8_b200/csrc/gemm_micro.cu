// gemm_micro.cu -- the product of two block-scaled FP4 matrices:
//   Y[m, n] = bf16( xs[m] ws[n] sum_k (cx[m, k] sx[m, b(k)]) (cw[n, k] sw[n, b(k)]) )
// with E2M1 codes c, one scale s per block of 16 (nvfp4, E4M3) or 32 (mxfp4,
// a power of two) elements along K, and fp32 accumulation in tensor memory.
//
// tcgen05.mma kind::mxf4nvf4 (scale_vec::4X) and kind::mxf4 (scale_vec::2X)
// take the codes of both operands from shared memory, two per byte, and the
// block scales from tensor memory.  A pipeline stage holds 256 K of both
// operands: one 128-byte swizzled row of codes per matrix row (TMA boxes of a
// [rows, K / 2] byte map) and the block scales of each 128-row band, which lie
// in memory in the order of the copy into tensor memory: 512 bytes (128 rows x
// 4 scales) are one 32x128b copy into 4 columns, replicated to the four lane
// quarters.  Boxes past a matrix's last row, last K or last band are filled
// with zeros; MMAs past K are not issued, so what a last stage's unused scales
// hold does not matter, and a row's scales only ever reach that row's results.
//
// Two kernels:
//   narrow (up to 64 tokens, or few tiles): the weights are the MMA's A operand
//     (128 rows), the tokens its B operand (BN columns), one CTA per tile and K
//     slice.  Such calls stream the weights, so K is sliced over a cluster of
//     CTAs until the SMs are full; the slices' partial sums meet in shared
//     memory over the cluster (distributed shared memory), are added in a fixed
//     order (the owner's, then the others by slice) and written once.
//     Bound by latency next to the weights' bytes: the start, the ring's first
//     fill and the join (1 x 11008 x 4096 takes 6.0 us of its 7.2 with all
//     operands in L2).
//   wide (more tokens): an SM pair (cta_group::2) multiplies 256 tokens by 256
//     weight rows, so that each SM reads half of both operands.  Bound by the
//     tensor pipe (a stage's 256 x 256 x 256 products would take 0.37 us of its
//     0.4 at four times the measured bf16 rate; no FP4 rate is measured), in
//     long runs at the clock that the power limit leaves, and in calls of few
//     tiles by the join of K slices (3 us) and the idle pairs.
// Measured, nvfp4, cold operands: 1 x 11008 x 4096 7.3 us (3.5 TB/s), 64 x 11008
// x 4096 9.7, 256 x 4096 x 14336 16.6 (1.8 PFLOP/s), 2048 x 4096 x 4096 18.1
// (3.8), 4096 x 12288 x 4096 86 (4.8) from a cool start and 100 (4.1) after
// seconds of it, at 1490 MHz under the power limit; mxfp4, half the scales, 2 to
// 8 % less.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kernels.h"
#include "micro_common.cuh"
#include "micro_kernels.h"
#include "sm100_ptx.cuh"
#include "sp24.h"

namespace sp24 {

namespace {

constexpr int kStageK = 256;            // K elements per pipeline stage
constexpr int kRowBytes = kStageK / 2;  // one swizzled row of codes
constexpr int kStepK = 64;              // K per MMA
constexpr int kMaxSlices = 8;           // CTAs that share a narrow tile's K (a portable cluster)
constexpr int kMaxWideSlices = 3;       // SM pairs that share a wide tile's K
constexpr int kNarrowTiles = 132;       // SMs that clusters of several CTAs fill

// Instruction descriptor of kinds mxf4 / mxf4nvf4: E2M1 operands (1), both
// K-major; scale type UE4M3 (0) or UE8M0 (1) at bit 23; N >> 3 at 17, M >> 7
// at 27.  The scale ids (bytes of a 32-bit scale word) go to bits 4 (B), 29 (A).
__host__ __device__ constexpr uint32_t micro_idesc(int block, uint32_t m, uint32_t n) {
  return (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (block == 32 ? 1u << 23 : 0u) | ((m >> 7) << 27);
}

template <int BLOCK, bool PAIR>
__device__ __forceinline__ void mma_micro(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                          uint32_t accumulate) {
#define SP24_MICRO_MMA(GROUP, KIND)                                                                        \
  asm volatile(                                                                                            \
      "{\n\t.reg .pred p;\n\t"                                                                             \
      "setp.ne.b32 p, %4, 0;\n\t"                                                                          \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),    \
      "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)                                    \
      : "memory")
  if constexpr (BLOCK == 16) {
    if constexpr (PAIR)
      SP24_MICRO_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
    else
      SP24_MICRO_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
  } else {
    if constexpr (PAIR)
      SP24_MICRO_MMA("2", "mxf4.block_scale.scale_vec::2X");
    else
      SP24_MICRO_MMA("1", "mxf4.block_scale.scale_vec::2X");
  }
#undef SP24_MICRO_MMA
}

// 512 bytes of block scales (128 rows x 4) from shared memory into 4 tensor
// memory columns, the 32 lanes replicated to all four lane quarters.
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
  const uint64_t d = smem_desc(saddr, 16, 128, kSwizzleNone);
  if constexpr (PAIR)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// Bulk copy of this CTA's shared memory into another CTA of the cluster,
// counted on that CTA's mbarrier (dst and bar: shared::cluster addresses).
__device__ __forceinline__ void bulk_push(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(smem_addr(src)), "r"(bytes), "r"(bar)
               : "memory");
}

// The CTAs of a cluster order only each other's asynchronous operations here,
// never plain stores: tensor-memory reads that have returned (wait::ld) and that
// the tcgen05 fences before the arrival and behind the wait order around it;
// bulk copies counted on mbarriers; mbarriers whose initialisation is fenced.
// So their arrivals are relaxed: a release at cluster scope first waits for the
// thread's earlier stores, which took 0.6 to 0.7 us of every tile of Y.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_meet() {
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

struct MicroParams {
  int M, N, K;
  int stages;      // ceil(K / 256)
  int slices;      // CTAs (pairs) of a cluster that share a tile's K
  int tiles_m, tiles_n;
  uint16_t *y;
  const float *xs, *ws;
  int x_vec, w_vec;
  int32_t *status;
};

// ------------------------------------------------------------------ narrow

// K slices of a tile are joined in shared memory: slice i owns the tile's
// tokens [i * per, (i + 1) * per); every slice lays its fp32 sums out [token]
// [128 rows], copies each other owner's tokens into that CTA (one bulk copy
// each: plain stores into another CTA's shared memory moved about 5 bytes/ns
// per SM, which made a 128 x 256 tile's join 20 us), and the owner adds them to
// its own, slices in order.  Up to 32 tokens what arrives has room of its own; wider
// tiles take it over the ring, once every CTA has finished its main loop.

// Tokens that arrive from other slices at most: (slices - 1) * ceil(BN / slices).
constexpr uint32_t most_tokens(int bn) {
  uint32_t most = 0;
  for (int s = 2; s <= kMaxSlices; ++s) {
    const uint32_t t = (s - 1) * ((bn + s - 1) / s);
    most = t > most ? t : most;
  }
  return most;
}

template <int BLOCK, int BN>
struct Narrow {
  static constexpr int kAtoms = kStageK / BLOCK / 4;  // 512-byte scale tiles per band and stage
  static constexpr uint32_t kABytes = 128 * kRowBytes;
  static constexpr uint32_t kBBytes = BN * kRowBytes;
  static constexpr uint32_t kSfBytes = kAtoms * 512;
  static constexpr uint32_t kBOff = kABytes, kSfaOff = kBOff + kBBytes, kSfbOff = kSfaOff + kSfBytes;
  static constexpr uint32_t kStageBytes = kSfbOff + kSfBytes;
  static constexpr bool kOwnRoom = BN <= 32;
  static constexpr uint32_t kPartBytes = most_tokens(BN) * 512;
  // Two CTAs on an SM, so that one starts (barriers, tensor memory,
  // descriptors: about 1 us) while the other works.  (Four of two stages each,
  // for BN = 16, held fewer bytes in flight: 1 x 11008 x 4096 7.5 us against
  // 7.2, 1 x 4096 x 14336 9.2 against 8.5.)
  static constexpr int kPerSm = 2;
  static constexpr int kStages = (109 * 1024 - (kOwnRoom ? kPartBytes : 0)) / kStageBytes;
  // CTAs that a call is cut into, and stages of a slice at least
  static constexpr int kCtas = BN <= 16 ? 192 : 2 * kNarrowTiles;
  static constexpr int kSliceStages = BN <= 32 ? 3 : 4;
  static constexpr uint32_t kPartOff = kOwnRoom ? kStages * kStageBytes : BN * 512;
  static constexpr uint32_t kBarOff = kStages * kStageBytes + (kOwnRoom ? kPartBytes : 0);
  static constexpr uint32_t kScaleOff = kBarOff + 512;  // the tile's token scales
  static constexpr uint32_t kSmem = kScaleOff + 512 + 1024 /*align*/;
  static constexpr uint32_t kSfCols = 8 * kAtoms;  // A's and B's scales of a stage; two stages' worth
  static constexpr uint32_t kTmemNeed = BN + 2 * kSfCols;
  static constexpr uint32_t kTmemCols = kTmemNeed <= 64 ? 64 : 128;
  static_assert(kTmemNeed <= 128 && kPerSm * kTmemCols <= 512, "tensor memory");
  static_assert(kStageBytes % 1024 == 0 && BN % 16 == 0 && BN <= 64, "tile");
  static_assert(kStages >= 2 && BN * 512 + (kOwnRoom ? 0 : kPartBytes) <= kStages * kStageBytes, "sums fit the ring");
};

template <int BLOCK, int BN>
__global__ void __launch_bounds__(192, Narrow<BLOCK, BN>::kPerSm)
    narrow_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                  const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmSX,
                  const MicroParams p) {
  using C = Narrow<BLOCK, BN>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
  uint64_t *empty = full + S;
  uint64_t *done = empty + S;
  uint64_t *arrived = done + 1;  // the other slices' sums
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(arrived + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slice = static_cast<int>(blockIdx.x) % p.slices, tile = static_cast<int>(blockIdx.x) / p.slices;
  const int n0 = (tile % p.tiles_n) * 128, m0 = (tile / p.tiles_n) * BN;
  // this slice's stages, and its tokens of the tile
  const int s0 = static_cast<int>(static_cast<int64_t>(slice) * p.stages / p.slices);
  const int s1 = static_cast<int>(static_cast<int64_t>(slice + 1) * p.stages / p.slices);
  const int mvalid = min(BN, p.M - m0);
  const int per = (mvalid + p.slices - 1) / p.slices;
  const int c0 = min(mvalid, slice * per), c1 = min(mvalid, c0 + per);

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmSW);
    prefetch_tensormap(&tmSX);
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    mbar_init(arrived, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(arrived, (p.slices - 1) * (c1 - c0) * 512);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (p.slices > 1) cluster_arrive();  // this CTA runs and its barriers exist
  const uint32_t tmem = *tmem_slot;
  // Everything the kernel reads may come from the kernel before it.
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {
    const bool leader = elect_one();
    const uint64_t keep = l2_policy_evict_last();
    const uint64_t stream = p.tiles_m == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
    const int tiles_k = (p.K / BLOCK + 3) / 4;
    for (int i = 0; i < s1 - s0; ++i) {
      const int s = i % S, kb = s0 + i;
      if (i >= S && !mbar_wait_warp(&empty[s], (static_cast<uint32_t>(i / S) & 1u) ^ 1u, p.status)) break;
      uint8_t *st = smem + s * C::kStageBytes;
      if (leader) {
        mbar_arrive_expect_tx(&full[s], C::kStageBytes);
        tma_load_2d(st, &tmW, &full[s], kb * kRowBytes, n0, stream);
        tma_load_2d(st + C::kSfaOff, &tmSW, &full[s], 0, ((n0 / 128) * tiles_k + kb * C::kAtoms) * 2, stream);
        tma_load_2d(st + C::kBOff, &tmX, &full[s], kb * kRowBytes, m0, keep);
        tma_load_2d(st + C::kSfbOff, &tmSX, &full[s], 0, ((m0 / 128) * tiles_k + kb * C::kAtoms) * 2, keep);
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    const bool leader = elect_one();
    constexpr uint32_t idesc = micro_idesc(BLOCK, 128, BN);
    for (int i = 0; i < s1 - s0; ++i) {
      const int s = i % S, kb = s0 + i;
      if (!mbar_wait_warp(&full[s], static_cast<uint32_t>(i / S) & 1u, p.status)) break;
      tc_fence_after();
      const uint32_t st = smem_addr(smem + s * C::kStageBytes);
      const uint32_t sfa = tmem + BN + (i & 1) * C::kSfCols, sfb = sfa + 4 * C::kAtoms;
      // a second tile of 64 tokens starts in the middle of a band of scales
      // (32 rows to a column)
      const uint32_t sfb_m = sfb + (m0 % 128) / 32;
      const int steps = min(kStageK / kStepK, (p.K - kb * kStageK) / kStepK);
      if (leader) {
#pragma unroll
        for (int a = 0; a < C::kAtoms; ++a) {
          copy_scales<false>(sfa + 4 * a, st + C::kSfaOff + 512 * a);
          copy_scales<false>(sfb + 4 * a, st + C::kSfbOff + 512 * a);
        }
#pragma unroll
        for (int j = 0; j < kStageK / kStepK; ++j) {
          if (j >= steps) break;
          const uint64_t ad = smem_desc(st + 32 * j, 16, 8 * kRowBytes, kSwizzle128B);
          const uint64_t bd = smem_desc(st + C::kBOff + 32 * j, 16, 8 * kRowBytes, kSwizzle128B);
          const uint32_t col = BLOCK == 16 ? 4 * j : 4 * (j / 2);
          const uint32_t id = BLOCK == 16 ? 0u : 2u * (j & 1);
          mma_micro<BLOCK, false>(tmem, ad, bd, idesc | id << 4 | id << 29, sfa + col, sfb_m + col, (i | j) ? 1u : 0u);
        }
        mma_commit(&empty[s]);
      }
      __syncwarp();
    }
    if (leader) mma_commit(done);
    __syncwarp();
  }

  // ---- epilogue: warps 2-5 hold 32 weight rows each (their lanes), and lay
  // the sums out [token][128 rows]; then a warp writes one token's 128 results
  const int q = warp & 3, tid = static_cast<int>(threadIdx.x) - 64;
  const int n = n0 + 4 * lane;  // of the four results a lane writes
  float *xsm = reinterpret_cast<float *>(smem + C::kScaleOff);
  float4 wsn = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
  if (warp >= 2) {
    // the scales, fetched while the main loop runs
    if (p.ws && p.w_vec) {
      if (n < p.N) wsn = __ldg(reinterpret_cast<const float4 *>(p.ws + n));
    } else if (p.ws) {
      wsn.x = wsn.y = wsn.z = wsn.w = __ldg(p.ws);
    }
    for (int c = tid; c < mvalid; c += 128) xsm[c] = p.xs ? __ldg(p.xs + (p.x_vec ? m0 + c : 0)) : 1.0f;
    mbar_wait(done, 0u, p.status);
    tc_fence_after();
    const uint32_t t_row = tmem + (static_cast<uint32_t>(q * 32) << 16);
    float *sums = reinterpret_cast<float *>(smem) + q * 32 + lane;
#pragma unroll 1
    for (int c = 0; c < mvalid; c += 16) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(t_row + c, v);
      tmem_ld_wait();
      tmem_regs_ready(v);
#pragma unroll
      for (int k = 0; k < 16; ++k) sums[(c + k) * 128] = __uint_as_float(v[k]);
    }
    tc_fence_before();
    fence_proxy_async_smem();
    named_bar_sync(1, 128);
  }
  if (p.slices > 1) {
    __syncwarp();
    cluster_wait();
    if (!C::kOwnRoom) cluster_meet();
  }
  if (warp >= 2) {
    if (p.slices > 1) {
      if (warp == 2 && lane < p.slices && lane != slice) {
        const int o0 = min(mvalid, lane * per), o1 = min(mvalid, o0 + per), from = slice - (slice > lane ? 1 : 0);
        if (o1 > o0)
          bulk_push(mapa_shared(smem + C::kPartOff + from * per * 512, lane), smem + o0 * 512, (o1 - o0) * 512,
                    mapa_shared(arrived, lane));
      }
      __syncwarp();
      mbar_wait(arrived, 0u, p.status);
    }
    const float4 *sums = reinterpret_cast<const float4 *>(smem) + lane;
    const float4 *part = reinterpret_cast<const float4 *>(smem + C::kPartOff) + lane;
    if (n < p.N) {
#pragma unroll 2
      for (int c = c0 + warp - 2; c < c1; c += 4) {
        float4 sum = sums[c * 32];
#pragma unroll
        for (int r = 0; r < kMaxSlices - 1; ++r) {
          if (r < p.slices - 1) {
            const float4 v = part[(r * per + c - c0) * 32];
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
          }
        }
        const float x = xsm[c];
        *reinterpret_cast<uint2 *>(p.y + static_cast<int64_t>(m0 + c) * p.N + n) =
            make_uint2(pack_bf16(sum.x * (x * wsn.x), sum.y * (x * wsn.y)), pack_bf16(sum.z * (x * wsn.z), sum.w * (x * wsn.w)));
      }
    }
  }
  if (p.slices > 1) {
    __syncwarp();
    cluster_meet();  // nobody leaves while its sums are being copied
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------------ wide

// 256 tokens (A, 128 per CTA) x 256 weight rows (B, 128 per CTA's half); each
// CTA's accumulator is 128 lanes (its tokens) x 256 columns.  Both CTAs hold
// the scales of all 256 weight rows.  Tensor memory: two accumulators of 256
// columns that share 96 (0..255 and 160..415), and two stages' scales.  Four
// epilogue warps take the shared columns of a finished tile to registers and
// give them free at once, and the next tile's main loop, in the other
// accumulator, runs beside the rest of the epilogue.  Reading tensor memory
// is slow enough (an accumulator's 128 KB takes 1.2 us) that the other four
// warps, who hold the accumulator's other half, wait until the shared columns
// are read.  Y leaves through shared memory, 32 tokens x 32 columns per bulk
// tensor store.
template <int BLOCK>
struct Wide {
  static constexpr int kAtoms = kStageK / BLOCK / 4;
  static constexpr uint32_t kABytes = 128 * kRowBytes, kBBytes = 128 * kRowBytes;
  static constexpr uint32_t kSfBytes = kAtoms * 512;
  static constexpr uint32_t kBOff = kABytes, kSfaOff = kBOff + kBBytes, kSfbOff = kSfaOff + kSfBytes;
  static constexpr uint32_t kStageBytes = kSfbOff + 2 * kSfBytes;
  static constexpr uint32_t kStagePitch = (kStageBytes + 1023) / 1024 * 1024;
  static constexpr int kStages = 5;
  static constexpr int kThreads = 64 + 256;
  static constexpr uint32_t kAcc1 = 160;                    // first column of the second accumulator
  static constexpr uint32_t kSfCol = kAcc1 + 256;           // first column of the scales
  static constexpr uint32_t kYBytes = 32 * 64 * 2;          // a warp's staged Y: two passes of 32 x 32
  static constexpr uint32_t kYOff = kStages * kStagePitch;  // one per epilogue warp
  static constexpr uint32_t kWsOff = kYOff + 8 * kYBytes;   // weight scales of two tiles
  static constexpr uint32_t kBarOff = kWsOff + 2 * 256 * 4;
  static constexpr uint32_t kSmem = kBarOff + 1024 + 1024 /*align*/;
  static constexpr uint32_t kSfCols = 12 * kAtoms;  // A 4, B 8 per 512-byte tile of A
  static_assert(kSfCol + 2 * kSfCols <= 512, "scale columns");
  // K slices: six of a 128 x 256 tile's eight 32-column units leave at most,
  // and as many arrive
  static constexpr uint32_t kUnitBytes = 128 * 32 * 4;
  static constexpr uint32_t kPartOff = 6 * kUnitBytes;
  static_assert(2 * kPartOff <= kWsOff, "partial sums reuse the ring and the staged Y");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

template <int BLOCK>
__global__ void __launch_bounds__(Wide<BLOCK>::kThreads, 1)
    wide_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmSX,
                const __grid_constant__ CUtensorMap tmY, const MicroParams p) {
  using C = Wide<BLOCK>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
  uint64_t *empty = full + S;
  uint64_t *acc_full = empty + S;        // [2]: accumulator complete
  uint64_t *shared_free = acc_full + 2;  // see the epilogue
  uint64_t *arrived = shared_free + 1;   // the other slices' sums
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(arrived + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank(), rank = crank & 1u, lead = crank & ~1u;
  const int slice = static_cast<int>(crank >> 1);
  const int csize = 2 * p.slices;
  const int first = static_cast<int>(blockIdx.x) / csize, step = static_cast<int>(gridDim.x) / csize;
  const int tiles = p.tiles_m * p.tiles_n;
  const int s0 = static_cast<int>(static_cast<int64_t>(slice) * p.stages / p.slices);
  const int s1 = static_cast<int>(static_cast<int64_t>(slice + 1) * p.stages / p.slices);
  const int u0 = slice * 8 / p.slices, u1 = (slice + 1) * 8 / p.slices;  // 32-column units this slice owns

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmSW);
    prefetch_tensormap(&tmSX);
    prefetch_tensormap(&tmY);
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full[0], 1);
    mbar_init(&acc_full[1], 1);
    mbar_init(shared_free, 8);  // both CTAs' epilogue warps of half 0
    mbar_init(arrived, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(arrived, (p.slices - 1) * (u1 - u0) * C::kUnitBytes);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_meet();  // the barriers of both CTAs exist before a remote arrive or load
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {
    const bool leader = elect_one();
    const uint64_t keep = l2_policy_evict_last();
    const int tiles_k = (p.K / BLOCK + 3) / 4;
    int i = 0;
    bool ok = true;
    for (int t = first; ok && t < tiles; t += step) {
      const int m0 = (t % p.tiles_m) * 256, n0 = (t / p.tiles_m) * 256;
      const int my_m = m0 + static_cast<int>(rank) * 128, my_n = n0 + static_cast<int>(rank) * 128;
      for (int kb = s0; kb < s1; ++kb, ++i) {
        const int s = i % S;
        if (i >= S && !mbar_wait_warp(&empty[s], (static_cast<uint32_t>(i / S) & 1u) ^ 1u, p.status)) {
          ok = false;
          break;
        }
        uint8_t *st = smem + s * C::kStagePitch;
        if (leader) {
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::kStageBytes);
          const uint32_t bar = mapa_shared(&full[s], lead);
          tma_load_2d_pair(st, &tmX, bar, kb * kRowBytes, my_m, keep);
          tma_load_2d_pair(st + C::kBOff, &tmW, bar, kb * kRowBytes, my_n, keep);
          tma_load_2d_pair(st + C::kSfaOff, &tmSX, bar, 0, ((my_m / 128) * tiles_k + kb * C::kAtoms) * 2, keep);
          tma_load_2d_pair(st + C::kSfbOff, &tmSW, bar, 0, ((n0 / 128) * tiles_k + kb * C::kAtoms) * 2, keep);
          tma_load_2d_pair(st + C::kSfbOff + C::kSfBytes, &tmSW, bar, 0,
                           ((n0 / 128 + 1) * tiles_k + kb * C::kAtoms) * 2, keep);
        }
        __syncwarp();
      }
    }
    // the leader's commits release this CTA's slots too: wait for the last
    // ones, so that none lands after this CTA has left
    for (int k = i > S ? i - S : 0; ok && k < i; ++k)
      if (!mbar_wait_warp(&empty[k % S], static_cast<uint32_t>(k / S) & 1u, p.status)) break;
  } else if (warp == 1) {
    if (rank == 0) {
      const bool leader = elect_one();
      const uint16_t both = static_cast<uint16_t>(3u << lead);
      constexpr uint32_t idesc = micro_idesc(BLOCK, 256, 256);
      int i = 0, j = 0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += step, ++j) {
        if (j > 0 && !mbar_wait_warp(shared_free, static_cast<uint32_t>(j - 1) & 1u, p.status)) break;
        tc_fence_after();
        const uint32_t d = tmem + (j & 1) * C::kAcc1;
        for (int kb = s0; kb < s1; ++kb, ++i) {
          const int s = i % S;
          if (!mbar_wait_warp(&full[s], static_cast<uint32_t>(i / S) & 1u, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_addr(smem + s * C::kStagePitch);
          const uint32_t sf = tmem + C::kSfCol + (i & 1) * C::kSfCols;
          const uint32_t sfb = sf + 4 * C::kAtoms;
          const int steps = min(kStageK / kStepK, (p.K - kb * kStageK) / kStepK);
          if (leader) {
#pragma unroll
            for (int a = 0; a < C::kAtoms; ++a) {
              copy_scales<true>(sf + 4 * a, st + C::kSfaOff + 512 * a);
              copy_scales<true>(sfb + 8 * a, st + C::kSfbOff + 512 * a);
              copy_scales<true>(sfb + 8 * a + 4, st + C::kSfbOff + C::kSfBytes + 512 * a);
            }
#pragma unroll
            for (int k = 0; k < kStageK / kStepK; ++k) {
              if (k >= steps) break;
              const uint64_t ad = smem_desc(st + 32 * k, 16, 8 * kRowBytes, kSwizzle128B);
              const uint64_t bd = smem_desc(st + C::kBOff + 32 * k, 16, 8 * kRowBytes, kSwizzle128B);
              const uint32_t a = BLOCK == 16 ? k : k / 2;
              const uint32_t id = BLOCK == 16 ? 0u : 2u * (k & 1);
              mma_micro<BLOCK, true>(d, ad, bd, idesc | id << 4 | id << 29, sf + 4 * a, sfb + 8 * a,
                                     (kb > s0 || k > 0) ? 1u : 0u);
            }
            mma_commit_pair(&empty[s], both);
          }
          __syncwarp();
        }
        if (leader) mma_commit_pair(&acc_full[j & 1], both);
        __syncwarp();
      }
    }
    __syncwarp();
  } else if (p.slices == 1) {
    // The MMAs of tile j + 1 wait for the warps of the shared columns (half 0)
    // of both CTAs, which arrive once they hold tile j's.  Tile j - 1, whose
    // accumulator tile j + 1 takes, has been left by then, by the other warps
    // (half 1) too: half 0 passes tile j's first barrier only with them.  Half
    // 1 must not arrive as well: it could be a tile ahead of the other CTA's
    // half 0, and its arrival for tile j + 1 would stand in for the one that
    // tile j still lacks.  Half 0 cannot be ahead, as it arrives for tile j + 1
    // after that tile's products, which wait for tile j's arrivals.
    const int e = warp - 2, half = e >> 2, q = warp & 3;
    float *wsm = reinterpret_cast<float *>(smem + C::kWsOff);
    uint8_t *buf = smem + C::kYOff + e * C::kYBytes;
    // one arrival a warp: a thread each, they would queue
    auto arrive = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(shared_free, lead));
    };
    int j = 0;
    for (int t = first; t < tiles; t += step, ++j) {
      const int mq = (t % p.tiles_m) * 256 + static_cast<int>(rank) * 128 + q * 32, n0 = (t / p.tiles_m) * 256;
      float xsm = 1.0f;
      if (p.xs) xsm = __ldg(p.xs + (p.x_vec ? min(mq + lane, p.M - 1) : 0));
      // the tile's weight scales, in the buffer of the tile before last
      float *wt = wsm + (j & 1) * 256;
      const int k0 = static_cast<int>(threadIdx.x) - 64;
      wt[k0] = p.ws ? __ldg(p.ws + (p.w_vec ? min(n0 + k0, p.N - 1) : 0)) : 1.0f;
      named_bar_sync(1, 256);
      mbar_wait(&acc_full[j & 1], static_cast<uint32_t>(j >> 1) & 1u, p.status);
      tc_fence_after();
      // The 128 columns this warp takes, from c0 on: accumulator 0 shares its
      // last 96, accumulator 1 its first 96.  v[0..2] are the shared ones (of
      // half 0), v[3] the rest.
      const int odd = j & 1, c0 = (half == 0) == (odd == 0) ? 128 : 0;
      const int cs = c0 + (odd ? 0 : 32), cr = c0 + (odd ? 96 : 0);
      const uint32_t t_row = tmem + odd * C::kAcc1 + (static_cast<uint32_t>(q * 32) << 16);
      uint32_t v[4][32];
      if (half == 1) named_bar_sync(2, 256);
#pragma unroll
      for (int i = 0; i < 3; ++i) tmem_ld_32x32b_x32(t_row + cs + 32 * i, v[i]);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 3; ++i) tmem_regs_ready(v[i]);
      tc_fence_before();
      if (half == 0) {
        arrive();
        named_bar_sync(2, 256);
      }
      tmem_ld_32x32b_x32(t_row + cr, v[3]);
      tmem_ld_wait();
      tmem_regs_ready(v[3]);
      tc_fence_before();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = i < 3 ? cs + 32 * i : cr;
        uint8_t *box = buf + (i & 1) * 2048;
        if (lane == 0) bulk_wait_group_read<1>();  // the store before last has read the box
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
          const float4 a = *reinterpret_cast<const float4 *>(wt + c + k), b = *reinterpret_cast<const float4 *>(wt + c + k + 4);
          const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          uint32_t o[4];
#pragma unroll
          for (int l = 0; l < 4; ++l)
            o[l] = pack_bf16(__uint_as_float(v[i][k + 2 * l]) * (xsm * f[2 * l]),
                             __uint_as_float(v[i][k + 2 * l + 1]) * (xsm * f[2 * l + 1]));
          // row `lane` of the 64-byte swizzled box: 16-byte chunk i at i ^ (lane / 2 & 3)
          *reinterpret_cast<uint4 *>(box + lane * 64 + ((k / 8) ^ (lane >> 1 & 3)) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (mq < p.M && n0 + c < p.N) tma_store_2d(&tmY, box, n0 + c, mq);
          bulk_commit_group();
        }
      }
    }
    // the CTA's shared memory outlives what the stores read; the writes are
    // complete with the grid
    if (lane == 0) bulk_wait_group_read<0>();
  }
  __syncwarp();
  if (p.slices > 1) {
    // One tile per cluster.  Slice i owns the 32-column units [8 i / slices,
    // 8 (i + 1) / slices) of the tile; every slice lays the others' units out
    // [unit][4 columns][token] over its ring, copies them to their owners, and
    // adds what arrives to its own, the other slices in order.  The units are
    // shared between the two halves of the epilogue warps.
    const int half = (warp - 2) >> 2, q = warp & 3, row = q * 32 + lane;
    const int m = (first % p.tiles_m) * 256 + static_cast<int>(rank) * 128 + row, n0 = (first / p.tiles_m) * 256;
    const uint32_t t_row = tmem + (static_cast<uint32_t>(q * 32) << 16);
    float *wt = reinterpret_cast<float *>(smem + C::kWsOff);
    float xsm = 1.0f;
    if (warp >= 2) {
      if (p.xs) xsm = __ldg(p.xs + (p.x_vec ? min(m, p.M - 1) : 0));
      const int k0 = static_cast<int>(threadIdx.x) - 64;
      wt[k0] = p.ws ? __ldg(p.ws + (p.w_vec ? min(n0 + k0, p.N - 1) : 0)) : 1.0f;
      mbar_wait(&acc_full[0], 0u, p.status);
      tc_fence_after();
    }
    __syncwarp();
    cluster_meet();  // no CTA's ring is in use any more
    if (warp >= 2) {
#pragma unroll 1
      for (int i = 1; i < p.slices; ++i) {
        const int o = (slice + i) % p.slices, o0 = o * 8 / p.slices, o1 = (o + 1) * 8 / p.slices;
        uint8_t *mine = smem + (o > slice ? o0 - (u1 - u0) : o0) * C::kUnitBytes;
#pragma unroll 1
        for (int u = o0 + half; u < o1; u += 2) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(t_row + u * 32, v);
          tmem_ld_wait();
          tmem_regs_ready(v);
#pragma unroll
          for (int l = 0; l < 8; ++l)
            *reinterpret_cast<uint4 *>(mine + (u - o0) * C::kUnitBytes + (l * 128 + row) * 16) =
                make_uint4(v[4 * l], v[4 * l + 1], v[4 * l + 2], v[4 * l + 3]);
        }
        fence_proxy_async_smem();
        named_bar_sync(1, 256);
        if (threadIdx.x == 64) {
          const uint32_t to = static_cast<uint32_t>(2 * o) + rank, from = slice - (slice > o ? 1 : 0);
          const uint32_t bytes = (o1 - o0) * C::kUnitBytes;
          bulk_push(mapa_shared(smem + C::kPartOff + from * bytes, to), mine, bytes, mapa_shared(arrived, to));
        }
        __syncwarp();
      }
      mbar_wait(arrived, 0u, p.status);
#pragma unroll 1
      for (int u = u0 + half; u < u1; u += 2) {
        const float4 *part = reinterpret_cast<const float4 *>(smem + C::kPartOff + (u - u0) * C::kUnitBytes) + row;
        uint32_t v[32];
        tmem_ld_32x32b_x32(t_row + u * 32, v);
        tmem_ld_wait();
        tmem_regs_ready(v);
#pragma unroll
        for (int l = 0; l < 8; l += 2) {
          const int c = u * 32 + l * 4;
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[4 * l + i]);
#pragma unroll
          for (int r = 0; r < kMaxWideSlices - 1; ++r) {
            if (r < p.slices - 1) {
              const float4 *src = part + r * (u1 - u0) * (C::kUnitBytes / 16);
              const float4 a = src[l * 128], b = src[(l + 1) * 128];
              f[0] += a.x, f[1] += a.y, f[2] += a.z, f[3] += a.w, f[4] += b.x, f[5] += b.y, f[6] += b.z, f[7] += b.w;
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= xsm * wt[c + i];
          if (n0 + c < p.N && m < p.M)
            *reinterpret_cast<uint4 *>(p.y + static_cast<int64_t>(m) * p.N + n0 + c) =
                make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
        }
      }
      tc_fence_before();
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  // no CTA frees tensor memory or leaves while another may still use it or
  // arrive on its barriers
  cluster_meet();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------ host

// Clusters of `slices` SM pairs of the wide kernel that the current device
// runs at once (148 SMs hold 74, 33 and 22), with the kernel's shared memory
// allowed.
template <int BLOCK>
cudaError_t wide_clusters(int slices, int *clusters) {
  static DeviceNumbers<kMaxWideSlices + 1> caps;
  return caps.get(slices, clusters, [slices](int *n) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * slices, 1, 1);
    cfg.blockDim = dim3(Wide<BLOCK>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = Wide<BLOCK>::kSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2 * slices;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(n, wide_kernel<BLOCK>, &cfg);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
  });
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), unsigned grid, unsigned cluster, unsigned threads, uint32_t smem, cudaStream_t st,
                   Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Codes [rows, K / 2] as bytes in boxes of 128 bytes x `box` rows; block
// scales as rows of 256 bytes (half a 512-byte tile), a stage's tiles per box.
bool make_maps(CUtensorMap *codes, CUtensorMap *scales, const uint8_t *q, const uint8_t *b, int64_t rows, int K, int block,
               int box) {
  const uint64_t tiles = static_cast<uint64_t>((rows + 127) / 128) * ((K / block + 3) / 4);
  return make_tensor_map_2d(codes, q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K / 2, rows, kRowBytes, box,
                            CU_TENSOR_MAP_SWIZZLE_128B) &&
         make_tensor_map_2d(scales, b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 256, tiles * 2, 256, kStageK / block / 4 * 2,
                            CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <int BLOCK, int BN>
cudaError_t launch_narrow(const MicroGemmArgs &a, MicroParams p, cudaStream_t st) {
  using C = Narrow<BLOCK, BN>;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t err = allow_shared(narrow_kernel<BLOCK, BN>, C::kSmem, ready);
  if (err != cudaSuccess) return err;
  p.tiles_n = (a.N + 127) / 128;
  p.tiles_m = (a.M + BN - 1) / BN;
  // K slices, cold weights: 1 x 11008 x 4096 (86 tiles) 7.2 us with 2, 7.6 with
  // 3, 10.4 with 4 (a second wave); 1 x 4096 x 14336 (32 tiles) 8.5 with 6, 9.7
  // with 3; 64 x 11008 x 4096 9.7 with 3, 10.0 with 2; 64 x 4096 x 4096 6.7 with
  // 4 (4 stages each), 7.9 with 8.
  const int64_t tiles = static_cast<int64_t>(p.tiles_n) * p.tiles_m;
  int64_t s = C::kCtas / tiles;
  if (s > p.stages / C::kSliceStages) s = p.stages / C::kSliceStages;
  if (s > kMaxSlices) s = kMaxSlices;
  if (s < 1) s = 1;
  p.slices = static_cast<int>(s);
  CUtensorMap tm[4];
  if (!make_maps(&tm[0], &tm[2], a.wq, a.wb, a.N, a.K, BLOCK, 128) ||
      !make_maps(&tm[1], &tm[3], a.xq, a.xb, a.M, a.K, BLOCK, BN))
    return cudaErrorInvalidValue;
  return launch(narrow_kernel<BLOCK, BN>, static_cast<unsigned>(tiles * s), static_cast<unsigned>(s), 192, C::kSmem, st, tm[0],
                tm[1], tm[2], tm[3], p);
}

template <int BLOCK>
cudaError_t launch_wide(const MicroGemmArgs &a, MicroParams p, cudaStream_t st) {
  p.tiles_m = (a.M + 255) / 256;
  p.tiles_n = (a.N + 255) / 256;
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> ready{0};
  cudaError_t err = allow_shared(wide_kernel<BLOCK>, Wide<BLOCK>::kSmem, ready);
  if (err != cudaSuccess) return err;
  int pairs = 0;
  if ((err = wide_clusters<BLOCK>(1, &pairs)) != cudaSuccess) return err;
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  // few tiles: slices of K over the idle pairs.  A stage takes about 0.4 us
  // and a join about 3 us, as much as 8 stages.
  int s = 1;
  int64_t best = (tiles + pairs - 1) / pairs * p.stages;
  for (int i = 2; i <= kMaxWideSlices && i <= p.stages; ++i) {
    int cap = 0;
    if ((err = wide_clusters<BLOCK>(i, &cap)) != cudaSuccess) return err;
    if (cap < 1) break;
    const int64_t cost = (tiles + cap - 1) / cap * ((p.stages + i - 1) / i + 8);
    if (cost < best) best = cost, s = i;
  }
  p.slices = s;
  const int64_t clusters = s > 1 ? tiles : (tiles < pairs ? tiles : pairs);
  CUtensorMap tm[5];
  if (!make_maps(&tm[0], &tm[2], a.wq, a.wb, a.N, a.K, BLOCK, 128) ||
      !make_maps(&tm[1], &tm[3], a.xq, a.xb, a.M, a.K, BLOCK, 128) ||
      !make_tensor_map_2d(&tm[4], a.y, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, a.N, a.M, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  return launch(wide_kernel<BLOCK>, static_cast<unsigned>(clusters * 2 * s), static_cast<unsigned>(2 * s), Wide<BLOCK>::kThreads,
                Wide<BLOCK>::kSmem, st, tm[0], tm[1], tm[2], tm[3], tm[4], p);
}

template <int BLOCK>
cudaError_t launch_block(const MicroGemmArgs &a, cudaStream_t st) {
  MicroParams p{};
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.stages = (a.K + kStageK - 1) / kStageK;
  p.y = a.y;
  p.xs = a.xs;
  p.ws = a.ws;
  p.x_vec = a.xs ? a.x_vec : 0;
  p.w_vec = a.ws ? a.w_vec : 0;
  p.status = a.status;
  if (a.M <= 16) return launch_narrow<BLOCK, 16>(a, p, st);
  if (a.M <= 32) return launch_narrow<BLOCK, 32>(a, p, st);
  // More than 64 tokens: narrow tiles as long as two or more slices of K fit
  // and an SM gets 32 stages of them at most (nvfp4, cold, narrow / SM pairs:
  // 256 x 4096 x 4096, 128 tiles of 16 stages, 9.2 / 11.7 us; 128 x 4096 x
  // 14336, 64 of 56, 13.2 / 16.3; 256 x 4096 x 8192, 128 of 32, 12.5 / 13.4; 192
  // x 4096 x 14336, 96 of 56, 17.6 / 16.3; 384 x 4096 x 4096, 192 of 16, 12.2 /
  // 10.6).
  const int64_t tiles = static_cast<int64_t>((a.N + 127) / 128) * ((a.M + 63) / 64);
  if (a.M <= 64 || (tiles <= kNarrowTiles && tiles * p.stages <= 32 * 148)) return launch_narrow<BLOCK, 64>(a, p, st);
  return launch_wide<BLOCK>(a, p, st);
}

}  // namespace

cudaError_t launch_micro_gemm(int block, const MicroGemmArgs &a, cudaStream_t st) {
  return block == 16 ? launch_block<16>(a, st) : launch_block<32>(a, st);
}

}  // namespace sp24
