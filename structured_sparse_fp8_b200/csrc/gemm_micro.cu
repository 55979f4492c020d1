// gemm_micro.cu -- the product of two block-scaled FP4 matrices:
//   Y[m, n] = bf16( xs[m] ws[n] sum_k (cx[m, k] sx[m, b(k)]) (cw[n, k] sw[n, b(k)]) )
// with E2M1 codes c, one scale s per block of 16 (nvfp4, E4M3) or 32 (mxfp4,
// a power of two) elements along K, and fp32 accumulation.
//
// A 64 x 64 tile of Y per CTA: both operands' values of 32 K are decoded to
// shared memory as fp32 and multiplied on the CUDA cores.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "micro_common.cuh"
#include "micro_kernels.h"
#include "quant_common.cuh"
#include "sp24.h"

namespace sp24 {

namespace {

constexpr int kTile = 64, kStep = 32;

__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t mag = c & 7u;
  const float v = mag < 2 ? 0.5f * mag : __uint_as_float((((mag >> 1) + 126u) << 23) | (mag & 1u) << 22);
  return (c & 8u) ? -v : v;
}

template <int BLOCK>
__device__ __forceinline__ float scale_value(uint32_t b) {
  if constexpr (BLOCK == 16) return e4m3_value(b);
  return b == 0u ? 0x1p-127f : __uint_as_float(b << 23);
}

template <int BLOCK>
__global__ void __launch_bounds__(256) simple_kernel(const MicroGemmArgs p) {
  __shared__ float a[kStep][kTile + 1], b[kStep][kTile + 1];
  const int n0 = blockIdx.x * kTile, m0 = blockIdx.y * kTile;
  const int64_t tiles = (p.K / BLOCK + 3) / 4;
  float acc[4][4] = {};
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int k0 = 0; k0 < p.K; k0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
      const int r = i / kStep, k = i % kStep;
      float va = 0.0f, vb = 0.0f;
      if (m0 + r < p.M) {
        const uint8_t c = p.xq[static_cast<int64_t>(m0 + r) * (p.K / 2) + (k0 + k) / 2];
        va = e2m1_value((k & 1) ? c >> 4 : c & 15) *
             scale_value<BLOCK>(p.xb[block_scale_offset(m0 + r, (k0 + k) / BLOCK, tiles)]);
      }
      if (n0 + r < p.N) {
        const uint8_t c = p.wq[static_cast<int64_t>(n0 + r) * (p.K / 2) + (k0 + k) / 2];
        vb = e2m1_value((k & 1) ? c >> 4 : c & 15) *
             scale_value<BLOCK>(p.wb[block_scale_offset(n0 + r, (k0 + k) / BLOCK, tiles)]);
      }
      a[k][r] = va;
      b[k][r] = vb;
    }
    __syncthreads();
    for (int k = 0; k < kStep; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[k][ty + 16 * i], b[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= p.M || n >= p.N) continue;
      const float xs = p.xs ? p.xs[p.x_vec ? m : 0] : 1.0f, ws = p.ws ? p.ws[p.w_vec ? n : 0] : 1.0f;
      p.y[static_cast<int64_t>(m) * p.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[i][j] * (xs * ws)));
    }
}

}  // namespace

cudaError_t launch_micro_gemm(int block, const MicroGemmArgs &a, cudaStream_t st) {
  const dim3 grid((a.N + kTile - 1) / kTile, (a.M + kTile - 1) / kTile);
  if (block == 16)
    simple_kernel<16><<<grid, 256, 0, st>>>(a);
  else
    simple_kernel<32><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace sp24
