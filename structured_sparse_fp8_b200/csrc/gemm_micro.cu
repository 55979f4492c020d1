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

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
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

template <int BLOCK, int BN>
struct Narrow {
  static constexpr int kAtoms = kStageK / BLOCK / 4;  // 512-byte scale tiles per band and stage
  static constexpr uint32_t kABytes = 128 * kRowBytes;
  static constexpr uint32_t kBBytes = BN * kRowBytes;
  static constexpr uint32_t kSfBytes = kAtoms * 512;
  static constexpr uint32_t kBOff = kABytes, kSfaOff = kBOff + kBBytes, kSfbOff = kSfaOff + kSfBytes;
  static constexpr uint32_t kStageBytes = kSfbOff + kSfBytes;
  // two CTAs on an SM
  static constexpr int kStages = (112 * 1024 - 2048) / kStageBytes;
  static constexpr uint32_t kSmem = kStages * kStageBytes + 1024 /*align*/ + 1024 /*barriers*/;
  static constexpr uint32_t kSfCols = 8 * kAtoms;  // A's and B's scales of a stage; two stages' worth
  static constexpr uint32_t kTmemNeed = BN + 2 * kSfCols;
  static constexpr uint32_t kTmemCols = kTmemNeed <= 64 ? 64 : kTmemNeed <= 128 ? 128 : 256;
  static_assert(kStageBytes % 1024 == 0 && BN % 16 == 0 && BN <= 128, "tile");
  static_assert(kStages >= 2 && BN * 128 * 4 <= kStages * kStageBytes, "partial sums reuse the ring");
};

template <int BLOCK, int BN>
__global__ void __launch_bounds__(192, 2)
    narrow_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                  const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmSX,
                  const MicroParams p) {
  using C = Narrow<BLOCK, BN>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S * C::kStageBytes);
  uint64_t *empty = full + S;
  uint64_t *done = empty + S;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slice = static_cast<int>(blockIdx.x) % p.slices, tile = static_cast<int>(blockIdx.x) / p.slices;
  const int n0 = (tile % p.tiles_n) * 128, m0 = (tile / p.tiles_n) * BN;
  // this slice's stages
  const int s0 = static_cast<int>(static_cast<int64_t>(slice) * p.stages / p.slices);
  const int s1 = static_cast<int>(static_cast<int64_t>(slice + 1) * p.stages / p.slices);

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
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
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
  } else {
    const int q = warp & 3, row = q * 32 + lane, n = n0 + row;
    const int mvalid = min(BN, p.M - m0);
    const float w1 = p.ws && !p.w_vec ? __ldg(p.ws) : 1.0f, x1 = p.xs && !p.x_vec ? __ldg(p.xs) : 1.0f;
    const float wsn = p.w_vec && n < p.N ? __ldg(p.ws + n) : w1;
    mbar_wait(done, 0u, p.status);
    tc_fence_after();
    const uint32_t t_row = tmem + (static_cast<uint32_t>(q * 32) << 16);
    float *part = reinterpret_cast<float *>(smem);
#pragma unroll 1
    for (int c = 0; c < mvalid; c += 16) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(t_row + c, v);
      tmem_ld_wait();
      tmem_regs_ready(v);
      if (p.slices > 1) {
#pragma unroll
        for (int k = 0; k < 16; ++k) part[(c + k) * 128 + row] = __uint_as_float(v[k]);
      } else if (n < p.N) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int m = m0 + c + k;
          if (c + k < mvalid) {
            const float xsm = p.x_vec ? __ldg(p.xs + m) : x1;
            p.y[static_cast<int64_t>(m) * p.N + n] =
                __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(v[k]) * (xsm * wsn)));
          }
        }
      }
    }
    tc_fence_before();
  }
  if (p.slices > 1) {
    __syncwarp();
    cluster_sync_all();
    if (warp >= 2) {
      const int mvalid = min(BN, p.M - m0);
      const float w1 = p.ws && !p.w_vec ? __ldg(p.ws) : 1.0f, x1 = p.xs && !p.x_vec ? __ldg(p.xs) : 1.0f;
      const int step = 128 * p.slices;
      for (int e = static_cast<int>(threadIdx.x) - 64 + 128 * slice; e < mvalid * 32; e += step) {
        const int m = m0 + e / 32, n = n0 + (e % 32) * 4;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int r = 0; r < p.slices; ++r) {  // in slice order: the same sum every time
          const float4 v = ld_cluster_f4(mapa_shared(smem + e * 16, r));
          sum.x += v.x;
          sum.y += v.y;
          sum.z += v.z;
          sum.w += v.w;
        }
        if (n < p.N) {
          const float xsm = p.x_vec ? __ldg(p.xs + m) : x1;
          const float4 w = p.w_vec ? __ldg(reinterpret_cast<const float4 *>(p.ws + n)) : make_float4(w1, w1, w1, w1);
          *reinterpret_cast<uint2 *>(p.y + static_cast<int64_t>(m) * p.N + n) =
              make_uint2(pack_bf16(sum.x * (xsm * w.x), sum.y * (xsm * w.y)),
                         pack_bf16(sum.z * (xsm * w.z), sum.w * (xsm * w.w)));
        }
      }
    }
    __syncwarp();
    cluster_sync_all();  // nobody leaves while its partial sums are read
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
// beside the rest of the epilogue.
template <int BLOCK>
struct Wide {
  static constexpr int kAtoms = kStageK / BLOCK / 4;
  static constexpr uint32_t kABytes = 128 * kRowBytes, kBBytes = 128 * kRowBytes;
  static constexpr uint32_t kSfBytes = kAtoms * 512;
  static constexpr uint32_t kBOff = kABytes, kSfaOff = kBOff + kBBytes, kSfbOff = kSfaOff + kSfBytes;
  static constexpr uint32_t kStageBytes = kSfbOff + 2 * kSfBytes;
  static constexpr uint32_t kStagePitch = (kStageBytes + 1023) / 1024 * 1024;
  static constexpr int kStages = 5;
  static constexpr uint32_t kPartPitch = 260;  // floats per token row of a partial tile
  static constexpr uint32_t kSmem = kStages * kStagePitch + 2048;
  static constexpr uint32_t kSfCols = 12 * kAtoms;                 // A 4, B 8 per 512-byte tile of A
  static constexpr uint32_t kSfSlots = kSfCols * 2 <= 64 ? 2 : 1;  // stages' scales held at once
  static_assert(kSfCols * kSfSlots <= 64, "scale columns");
  static_assert(128 * kPartPitch * 4 <= kStages * kStagePitch, "partial sums reuse the ring");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

template <int BLOCK>
__global__ void __launch_bounds__(192, 1)
    wide_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmSX,
                const MicroParams p) {
  using C = Wide<BLOCK>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S * C::kStagePitch);
  uint64_t *empty = full + S;
  uint64_t *acc_full = empty + S;      // [2]: accumulator complete
  uint64_t *shared_free = acc_full + 2;  // a tile's shared columns are in registers
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(shared_free + 1);

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
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full[0], 1);
    mbar_init(&acc_full[1], 1);
    mbar_init(shared_free, 256);  // both CTAs' epilogue threads
    fence_mbar_init();
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
  } else {
    const int q = warp & 3, row = q * 32 + lane;
    const float w1 = p.ws && !p.w_vec ? __ldg(p.ws) : 1.0f, x1 = p.xs && !p.x_vec ? __ldg(p.xs) : 1.0f;
    int j = 0;
    for (int t = first; t < tiles; t += step, ++j) {
      const int m = (t % p.tiles_m) * 256 + static_cast<int>(rank) * 128 + row, n0 = (t / p.tiles_m) * 256;
      const float xsm = p.x_vec && m < p.M ? __ldg(p.xs + m) : x1;
      if (!mbar_wait(&acc_full[j & 1], static_cast<uint32_t>(j >> 1) & 1u, p.status)) break;
      tc_fence_after();
      const uint32_t t_row = tmem + (j & 1) * 192 + (static_cast<uint32_t>(q * 32) << 16);
      // 64 columns at a time, the shared ones first: the last of the lower
      // accumulator, the first of the upper
#pragma unroll 1
      for (int h = 0; h < 4; ++h) {
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
        if (p.slices > 1) {
          float4 *dst = reinterpret_cast<float4 *>(reinterpret_cast<float *>(smem) + row * C::kPartPitch + c);
#pragma unroll
          for (int k = 0; k < 16; ++k)
            dst[k] = make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]), __uint_as_float(v[4 * k + 2]),
                                 __uint_as_float(v[4 * k + 3]));
        } else if (m < p.M) {
          uint16_t *y = p.y + static_cast<int64_t>(m) * p.N + n0 + c;
#pragma unroll
          for (int k = 0; k < 64; k += 8) {
            if (n0 + c + k < p.N) {
              float f[8];
              if (p.w_vec) {
                const float4 a = __ldg(reinterpret_cast<const float4 *>(p.ws + n0 + c + k));
                const float4 b = __ldg(reinterpret_cast<const float4 *>(p.ws + n0 + c + k + 4));
                f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
              } else {
#pragma unroll
                for (int l = 0; l < 8; ++l) f[l] = w1;
              }
#pragma unroll
              for (int l = 0; l < 8; ++l) f[l] = __uint_as_float(v[k + l]) * (xsm * f[l]);
              *reinterpret_cast<uint4 *>(y + k) =
                  make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
            }
          }
        }
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  if (p.slices > 1) {
    cluster_sync_all();  // every slice's partial tile is written
    if (warp >= 2) {
      // this CTA's columns of its own 128 tokens, over all slices
      const float w1 = p.ws && !p.w_vec ? __ldg(p.ws) : 1.0f, x1 = p.xs && !p.x_vec ? __ldg(p.xs) : 1.0f;
      const int m0 = (first % p.tiles_m) * 256 + static_cast<int>(rank) * 128, n0 = (first / p.tiles_m) * 256;
      const int quads = 64 / p.slices, c0 = quads * slice;  // of 4 columns
      const int rows = min(128, p.M - m0);
      for (int e = static_cast<int>(threadIdx.x) - 64; e < rows * quads; e += 128) {
        const int r = e / quads, c = (c0 + e % quads) * 4, m = m0 + r, n = n0 + c;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k = 0; k < p.slices; ++k) {
          const float4 v = ld_cluster_f4(mapa_shared(reinterpret_cast<float *>(smem) + r * C::kPartPitch + c, 2 * k + rank));
          sum.x += v.x;
          sum.y += v.y;
          sum.z += v.z;
          sum.w += v.w;
        }
        if (n < p.N) {
          const float xsm = p.x_vec ? __ldg(p.xs + m) : x1;
          const float4 w = p.w_vec ? __ldg(reinterpret_cast<const float4 *>(p.ws + n)) : make_float4(w1, w1, w1, w1);
          *reinterpret_cast<uint2 *>(p.y + static_cast<int64_t>(m) * p.N + n) =
              make_uint2(pack_bf16(sum.x * (xsm * w.x), sum.y * (xsm * w.y)),
                         pack_bf16(sum.z * (xsm * w.z), sum.w * (xsm * w.w)));
        }
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  // no CTA frees tensor memory or leaves while another may still use it, read
  // its partial sums or arrive on its barriers
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

template <typename Kernel>
cudaError_t launch(Kernel kernel, unsigned grid, unsigned cluster, uint32_t smem, const CUtensorMap (&tm)[4],
                   const MicroParams &p, cudaStream_t st) {
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
  return cudaLaunchKernelEx(&cfg, kernel, tm[0], tm[1], tm[2], tm[3], p);
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
  // K slices: as many as leave every CTA resident at once, two on an SM
  const int64_t tiles = static_cast<int64_t>(p.tiles_n) * p.tiles_m;
  int64_t s = 2 * 148 / tiles;
  s = s < 1 ? 1 : s > 8 ? 8 : s;
  if (s > p.stages) s = p.stages;
  p.slices = static_cast<int>(s);
  CUtensorMap tm[4];
  if (!make_maps(&tm[0], &tm[2], a.wq, a.wb, a.N, a.K, BLOCK, 128) ||
      !make_maps(&tm[1], &tm[3], a.xq, a.xb, a.M, a.K, BLOCK, BN))
    return cudaErrorInvalidValue;
  return launch(narrow_kernel<BLOCK, BN>, static_cast<unsigned>(tiles * s), static_cast<unsigned>(s), C::kSmem, tm, p, st);
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
  CUtensorMap tm[4];
  if (!make_maps(&tm[0], &tm[2], a.wq, a.wb, a.N, a.K, BLOCK, 128) ||
      !make_maps(&tm[1], &tm[3], a.xq, a.xb, a.M, a.K, BLOCK, 128))
    return cudaErrorInvalidValue;
  return launch(wide_kernel<BLOCK>, static_cast<unsigned>(clusters * 2 * s), static_cast<unsigned>(2 * s), Wide<BLOCK>::kSmem,
                tm, p, st);
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
