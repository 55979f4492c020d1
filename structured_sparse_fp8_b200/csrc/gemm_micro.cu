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
//   narrow (M <= 128 tokens): the weights are the MMA's A operand (128 rows),
//     the tokens its B operand (BN columns), one CTA per weight tile and K
//     slice.  Such calls stream the weights, so K is sliced over a cluster of
//     CTAs until the SMs are full; the slices' partial sums meet in shared
//     memory over the cluster (distributed shared memory), are added in slice
//     order and written once.
//   wide (more tokens): an SM pair (cta_group::2) multiplies 256 tokens by 256
//     weight rows.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

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
// per SM, which made a 128 x 256 tile's join 20 us), and the owner adds them,
// slices in order.  Up to 32 tokens what arrives has room of its own; wider
// tiles take it over the ring, once every CTA has finished its main loop.
template <int BLOCK, int BN>
struct Narrow {
  static constexpr int kAtoms = kStageK / BLOCK / 4;  // 512-byte scale tiles per band and stage
  static constexpr uint32_t kABytes = 128 * kRowBytes;
  static constexpr uint32_t kBBytes = BN * kRowBytes;
  static constexpr uint32_t kSfBytes = kAtoms * 512;
  static constexpr uint32_t kBOff = kABytes, kSfaOff = kBOff + kBBytes, kSfbOff = kSfaOff + kSfBytes;
  static constexpr uint32_t kStageBytes = kSfbOff + kSfBytes;
  static constexpr bool kOwnRoom = BN <= 32;
  // (slices - 1) * ceil(BN / slices) tokens arrive at most
  static constexpr uint32_t kPartBytes = (BN + kMaxSlices - 2) * 512;
  // two CTAs on an SM, but for the widest tile
  static constexpr int kPerSm = BN <= 64 ? 2 : 1;
  static constexpr uint32_t kBudget = (kPerSm == 2 ? 112 : 200) * 1024;
  static constexpr int kStages = (kBudget - 2048 - (kOwnRoom ? kPartBytes : 0)) / kStageBytes;
  static constexpr uint32_t kPartOff = kOwnRoom ? kStages * kStageBytes : BN * 512;
  static constexpr uint32_t kBarOff = kStages * kStageBytes + (kOwnRoom ? kPartBytes : 0);
  static constexpr uint32_t kSmem = kBarOff + 1024 /*align*/ + 1024 /*barriers*/;
  static constexpr uint32_t kSfCols = 8 * kAtoms;  // A's and B's scales of a stage; two stages' worth
  static constexpr uint32_t kTmemNeed = BN + 2 * kSfCols;
  static constexpr uint32_t kTmemCols = kTmemNeed <= 64 ? 64 : kTmemNeed <= 128 ? 128 : 256;
  static_assert(kStageBytes % 1024 == 0 && BN % 16 == 0 && BN <= 128, "tile");
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
          mma_micro<BLOCK, false>(tmem, ad, bd, idesc | id << 4 | id << 29, sfa + col, sfb + col, (i | j) ? 1u : 0u);
        }
        mma_commit(&empty[s]);
      }
      __syncwarp();
    }
    if (leader) mma_commit(done);
    __syncwarp();
  }

  // ---- epilogue: warps 2-5 hold 32 weight rows each (their lanes)
  const int q = warp & 3, row = q * 32 + lane, n = n0 + row;
  float wsn = 1.0f, x1 = 1.0f;
  if (warp >= 2) {
    if (p.ws) wsn = __ldg(p.ws + (p.w_vec ? min(n, p.N - 1) : 0));
    if (p.xs && !p.x_vec) x1 = __ldg(p.xs);
    mbar_wait(done, 0u, p.status);
    tc_fence_after();
  }
  auto store = [&](int m, float sum) {
    const float xsm = p.x_vec ? __ldg(p.xs + m) : x1;
    p.y[static_cast<int64_t>(m) * p.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(sum * (xsm * wsn)));
  };
  if (p.slices > 1) {
    __syncwarp();
    cluster_wait();
    if (!C::kOwnRoom) {
      cluster_arrive();
      cluster_wait();
    }
  }
  if (warp >= 2) {
    const uint32_t t_row = tmem + (static_cast<uint32_t>(q * 32) << 16);
    float *sums = reinterpret_cast<float *>(smem) + row;
#pragma unroll 1
    for (int c = 0; c < mvalid; c += 16) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(t_row + c, v);
      tmem_ld_wait();
      tmem_regs_ready(v);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        if (p.slices > 1) {
          sums[(c + k) * 128] = __uint_as_float(v[k]);
        } else if (c + k < mvalid && n < p.N) {
          store(m0 + c + k, __uint_as_float(v[k]));
        }
      }
    }
    tc_fence_before();
    if (p.slices > 1) {
      fence_proxy_async_smem();
      named_bar_sync(1, 128);
      if (warp == 2 && lane < p.slices && lane != slice) {
        const int o0 = min(mvalid, lane * per), o1 = min(mvalid, o0 + per), from = slice - (slice > lane ? 1 : 0);
        if (o1 > o0)
          bulk_push(mapa_shared(smem + C::kPartOff + from * per * 512, lane), smem + o0 * 512, (o1 - o0) * 512,
                    mapa_shared(arrived, lane));
      }
      __syncwarp();
      mbar_wait_cluster(arrived, 0u, p.status);
      const float *part = reinterpret_cast<const float *>(smem + C::kPartOff) + row;
      if (n < p.N) {
        for (int c = c0; c < c1; ++c) {
          float sum = sums[c * 128];
#pragma unroll
          for (int r = 0; r < kMaxSlices - 1; ++r)
            if (r < p.slices - 1) sum += part[(r * per + c - c0) * 128];
          store(m0 + c, sum);
        }
      }
    }
  }
  if (p.slices > 1) {
    __syncwarp();
    cluster_sync_all();  // nobody leaves while its sums are being copied
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
// columns that overlap in 64 (0..255 and 192..447), and 64 columns of scales.
// A tile's epilogue first takes the 64 shared columns to registers and gives
// them free; the next tile's main loop, in the other accumulator, then runs
// beside the rest of the epilogue.  Y leaves through shared memory, 32 tokens
// x 64 columns per bulk tensor store.
template <int BLOCK>
struct Wide {
  static constexpr int kAtoms = kStageK / BLOCK / 4;
  static constexpr uint32_t kABytes = 128 * kRowBytes, kBBytes = 128 * kRowBytes;
  static constexpr uint32_t kSfBytes = kAtoms * 512;
  static constexpr uint32_t kBOff = kABytes, kSfaOff = kBOff + kBBytes, kSfbOff = kSfaOff + kSfBytes;
  static constexpr uint32_t kStageBytes = kSfbOff + 2 * kSfBytes;
  static constexpr uint32_t kStagePitch = (kStageBytes + 1023) / 1024 * 1024;
  static constexpr int kStages = 5;
  static constexpr uint32_t kYBytes = 32 * 128;             // one warp's staged 32 x 64 of Y
  static constexpr uint32_t kYOff = kStages * kStagePitch;  // two per epilogue warp
  static constexpr uint32_t kWsOff = kYOff + 8 * kYBytes;   // weight scales of two tiles
  static constexpr uint32_t kBarOff = kWsOff + 2 * 256 * 4;
  static constexpr uint32_t kSmem = kBarOff + 1024 + 1024 /*align*/;
  static constexpr uint32_t kSfCols = 12 * kAtoms;                 // A 4, B 8 per 512-byte tile of A
  static constexpr uint32_t kSfSlots = kSfCols * 2 <= 64 ? 2 : 1;  // stages' scales held at once
  static_assert(kSfCols * kSfSlots <= 64, "scale columns");
  // K slices: three quarters of a 128 x 256 tile leave and as many arrive
  static constexpr uint32_t kPartOff = 3 * 128 * 64 * 4;
  static_assert(2 * kPartOff <= kWsOff, "partial sums reuse the ring and the staged Y");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

template <int BLOCK>
__global__ void __launch_bounds__(192, 1)
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
  uint64_t *shared_free = acc_full + 2;  // a tile's shared columns are in registers
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
    mbar_init(shared_free, 256);  // both CTAs' epilogue threads
    mbar_init(arrived, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(arrived, (p.slices - 1) * (64 / p.slices) * 2048);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the barriers of both CTAs exist before a remote arrive or load
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
        if (j > 0 && !mbar_wait_cluster_warp(shared_free, static_cast<uint32_t>(j - 1) & 1u, p.status)) break;
        tc_fence_after();
        const uint32_t d = tmem + (j & 1) * 192;
        for (int kb = s0; kb < s1; ++kb, ++i) {
          const int s = i % S;
          if (!mbar_wait_warp(&full[s], static_cast<uint32_t>(i / S) & 1u, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_addr(smem + s * C::kStagePitch);
          const uint32_t sf = tmem + 448 + (C::kSfSlots == 2 ? (i & 1) * C::kSfCols : 0);
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
    const int e = warp - 2, q = warp & 3;
    float *wsm = reinterpret_cast<float *>(smem + C::kWsOff);
    int j = 0;
    uint32_t pass = 0;
    for (int t = first; t < tiles; t += step, ++j) {
      const int mq = (t % p.tiles_m) * 256 + static_cast<int>(rank) * 128 + q * 32, n0 = (t / p.tiles_m) * 256;
      float xsm = 1.0f;
      if (p.xs) xsm = __ldg(p.xs + (p.x_vec ? min(mq + lane, p.M - 1) : 0));
      // the tile's weight scales, in the buffer of the tile before last
      float *wt = wsm + (j & 1) * 256;
      for (int k = static_cast<int>(threadIdx.x) - 64; k < 256; k += 128)
        wt[k] = p.ws ? __ldg(p.ws + (p.w_vec ? min(n0 + k, p.N - 1) : 0)) : 1.0f;
      named_bar_sync(1, 128);
      mbar_wait(&acc_full[j & 1], static_cast<uint32_t>(j >> 1) & 1u, p.status);
      tc_fence_after();
      const uint32_t t_row = tmem + (j & 1) * 192 + (static_cast<uint32_t>(q * 32) << 16);
      // 64 columns at a time, the shared ones first: the last of the lower
      // accumulator, the first of the upper
#pragma unroll 1
      for (int h = 0; h < 4; ++h, ++pass) {
        const int c = ((j & 1) ? h : (h + 3) & 3) * 64;
        uint32_t v[64];
        tmem_ld_32x32b_x64(t_row + c, v);
        tmem_ld_wait();
        tmem_regs_ready(v);
        if (h == 0) {
          tc_fence_before();
          if (rank == 0)
            mbar_arrive(shared_free);
          else
            mbar_arrive_cluster(mapa_shared(shared_free, lead));
        }
        uint8_t *buf = smem + C::kYOff + (2 * e + (pass & 1)) * C::kYBytes;
        if (lane == 0) bulk_wait_group_read<1>();  // the store two passes ago has read it
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 64; k += 8) {
          const float4 a = *reinterpret_cast<const float4 *>(wt + c + k), b = *reinterpret_cast<const float4 *>(wt + c + k + 4);
          const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          uint32_t o[4];
#pragma unroll
          for (int l = 0; l < 4; ++l)
            o[l] = pack_bf16(__uint_as_float(v[k + 2 * l]) * (xsm * f[2 * l]),
                             __uint_as_float(v[k + 2 * l + 1]) * (xsm * f[2 * l + 1]));
          // row `lane` of the 128-byte swizzled box: 16-byte chunk i at i ^ (lane & 7)
          *reinterpret_cast<uint4 *>(buf + lane * 128 + ((k / 8) ^ (lane & 7)) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (mq < p.M && n0 + c < p.N) tma_store_2d(&tmY, buf, n0 + c, mq);
          bulk_commit_group();
        }
      }
    }
    tc_fence_before();
    if (lane == 0) bulk_wait_group_all();
  }
  __syncwarp();
  if (p.slices > 1) {
    // One tile per cluster.  Slice i owns 256 / slices columns of the tile;
    // every slice lays the others' columns out [owner][4 columns][token] over
    // its ring, copies them to their owners, and adds what arrives to its own,
    // the other slices in order.
    const int q = warp & 3, row = q * 32 + lane;
    const int m = (first % p.tiles_m) * 256 + static_cast<int>(rank) * 128 + row, n0 = (first / p.tiles_m) * 256;
    const int quads = 64 / p.slices;
    const uint32_t t_row = tmem + (static_cast<uint32_t>(q * 32) << 16);
    if (warp >= 2) {
      mbar_wait(&acc_full[0], 0u, p.status);
      tc_fence_after();
    }
    __syncwarp();
    cluster_sync_all();  // no CTA's ring is in use any more
    if (warp >= 2) {
#pragma unroll 1
      for (int o = 0; o < p.slices; ++o) {
        if (o == slice) continue;
        uint8_t *mine = smem + (o - (o > slice ? 1 : 0)) * quads * 2048;
#pragma unroll 1
        for (int k = 0; k < quads; k += 8) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(t_row + (o * quads + k) * 4, v);
          tmem_ld_wait();
          tmem_regs_ready(v);
#pragma unroll
          for (int l = 0; l < 8; ++l)
            *reinterpret_cast<uint4 *>(mine + ((k + l) * 128 + row) * 16) =
                make_uint4(v[4 * l], v[4 * l + 1], v[4 * l + 2], v[4 * l + 3]);
        }
        fence_proxy_async_smem();
        named_bar_sync(1, 128);
        if (threadIdx.x == 64) {
          const uint32_t to = static_cast<uint32_t>(2 * o) + rank, from = slice - (slice > o ? 1 : 0);
          bulk_push(mapa_shared(smem + C::kPartOff + from * quads * 2048, to), mine, quads * 2048, mapa_shared(arrived, to));
        }
        __syncwarp();
      }
      const float xsm = p.xs ? __ldg(p.xs + (p.x_vec ? min(m, p.M - 1) : 0)) : 1.0f;
      const float w1 = p.ws && !p.w_vec ? __ldg(p.ws) : 1.0f;
      mbar_wait_cluster(arrived, 0u, p.status);
      const float4 *part = reinterpret_cast<const float4 *>(smem + C::kPartOff) + row;
#pragma unroll 1
      for (int k = 0; k < quads; k += 8) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(t_row + (slice * quads + k) * 4, v);
        tmem_ld_wait();
        tmem_regs_ready(v);
#pragma unroll
        for (int l = 0; l < 8; l += 2) {
          const int n = n0 + (slice * quads + k + l) * 4;
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[4 * l + i]);
#pragma unroll
          for (int r = 0; r < 3; ++r) {
            if (r < p.slices - 1) {
              const float4 a = part[(r * quads + k + l) * 128], b = part[(r * quads + k + l + 1) * 128];
              f[0] += a.x, f[1] += a.y, f[2] += a.z, f[3] += a.w, f[4] += b.x, f[5] += b.y, f[6] += b.z, f[7] += b.w;
            }
          }
          if (n < p.N && m < p.M) {
            float4 a = make_float4(w1, w1, w1, w1), b = a;
            if (p.w_vec) a = __ldg(reinterpret_cast<const float4 *>(p.ws + n)), b = __ldg(reinterpret_cast<const float4 *>(p.ws + n + 4));
            *reinterpret_cast<uint4 *>(p.y + static_cast<int64_t>(m) * p.N + n) = make_uint4(
                pack_bf16(f[0] * (xsm * a.x), f[1] * (xsm * a.y)), pack_bf16(f[2] * (xsm * a.z), f[3] * (xsm * a.w)),
                pack_bf16(f[4] * (xsm * b.x), f[5] * (xsm * b.y)), pack_bf16(f[6] * (xsm * b.z), f[7] * (xsm * b.w)));
          }
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
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------ host

// Clusters of `size` CTAs of the wide kernel that the device runs at once.
template <int BLOCK>
int wide_clusters(int size) {
  static int cap[3] = {0, 0, 0};
  static std::once_flag once;
  std::call_once(once, [] {
    if (cudaFuncSetAttribute(wide_kernel<BLOCK>, cudaFuncAttributeMaxDynamicSharedMemorySize, Wide<BLOCK>::kSmem) != cudaSuccess) {
      (void)cudaGetLastError();
      return;
    }
    for (int i = 0; i < 3; ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2u << i, 1, 1);
      cfg.blockDim = dim3(192, 1, 1);
      cfg.dynamicSmemBytes = Wide<BLOCK>::kSmem;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = 2u << i;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, wide_kernel<BLOCK>, &cfg) == cudaSuccess)
        cap[i] = n;
      else
        (void)cudaGetLastError();
    }
  });
  return cap[size == 2 ? 0 : size == 4 ? 1 : 2];
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), unsigned grid, unsigned cluster, uint32_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(192, 1, 1);
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
  static std::once_flag once;
  static cudaError_t err = cudaSuccess;
  std::call_once(once, [] {
    err = cudaFuncSetAttribute(narrow_kernel<BLOCK, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  if (err != cudaSuccess) return err;
  p.tiles_n = (a.N + 127) / 128;
  p.tiles_m = (a.M + BN - 1) / BN;
  // K slices: as many as leave every CTA resident at once (one
  // token tile at most 128 wide, so a tile starts at a band of 128 rows)
  const int64_t tiles = static_cast<int64_t>(p.tiles_n) * p.tiles_m;
  int64_t s = C::kPerSm * 148 / tiles;
  s = s < 1 ? 1 : s > kMaxSlices ? kMaxSlices : s;
  if (s > p.stages) s = p.stages;
  p.slices = static_cast<int>(s);
  CUtensorMap tm[4];
  if (!make_maps(&tm[0], &tm[2], a.wq, a.wb, a.N, a.K, BLOCK, 128) ||
      !make_maps(&tm[1], &tm[3], a.xq, a.xb, a.M, a.K, BLOCK, BN))
    return cudaErrorInvalidValue;
  return launch(narrow_kernel<BLOCK, BN>, static_cast<unsigned>(tiles * s), static_cast<unsigned>(s), C::kSmem, st, tm[0], tm[1],
                tm[2], tm[3], p);
}

template <int BLOCK>
cudaError_t launch_wide(const MicroGemmArgs &a, MicroParams p, cudaStream_t st) {
  p.tiles_m = (a.M + 255) / 256;
  p.tiles_n = (a.N + 255) / 256;
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  const int pairs = wide_clusters<BLOCK>(2);
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  // few tiles: slices of K over the idle pairs
  int s = 1;
  while (s < 4 && tiles * 2 * s <= pairs && 2 * s <= p.stages && wide_clusters<BLOCK>(4 * s) >= 1) s *= 2;
  p.slices = s;
  const int64_t clusters = s > 1 ? tiles : (tiles < pairs ? tiles : pairs);
  CUtensorMap tm[5];
  if (!make_maps(&tm[0], &tm[2], a.wq, a.wb, a.N, a.K, BLOCK, 128) ||
      !make_maps(&tm[1], &tm[3], a.xq, a.xb, a.M, a.K, BLOCK, 128) ||
      !make_tensor_map_2d(&tm[4], a.y, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, a.N, a.M, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  return launch(wide_kernel<BLOCK>, static_cast<unsigned>(clusters * 2 * s), static_cast<unsigned>(2 * s), Wide<BLOCK>::kSmem,
                st, tm[0], tm[1], tm[2], tm[3], tm[4], p);
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
  if (a.M <= 64) return launch_narrow<BLOCK, 64>(a, p, st);
  if (a.M <= 128) return launch_narrow<BLOCK, 128>(a, p, st);
  return launch_wide<BLOCK>(a, p, st);
}

}  // namespace

cudaError_t launch_micro_gemm(int block, const MicroGemmArgs &a, cudaStream_t st) {
  return block == 16 ? launch_block<16>(a, st) : launch_block<32>(a, st);
}

}  // namespace sp24
