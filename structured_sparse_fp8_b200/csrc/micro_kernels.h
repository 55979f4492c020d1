// micro_kernels.h -- launches of the block-scaled FP4 kernels and of the
// row stages (norm, gated activation) that quantise their output: internal to
// the library (api.cu, rowquant.cu, gemm_micro.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace sp24 {

// Lets `kernel` use `bytes` of dynamic shared memory on the current device;
// `ready` has a bit for each device where that is done.
template <typename... Args>
cudaError_t allow_shared(void (*kernel)(Args...), uint32_t bytes, std::atomic<uint64_t> &ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (ready.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes));
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
  return e;
}

// Numbers that a device has, each asked for once a device; what could not be
// told is asked for again.
template <int N>
struct DeviceNumbers {
  std::atomic<int> known[64][N] = {};  // the number + 1, or 0
  template <typename Ask>  // cudaError_t ask(int *)
  cudaError_t get(int which, int *number, Ask ask) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<int> &k = known[dev & 63][which];
    *number = k.load(std::memory_order_relaxed) - 1;
    if (*number >= 0) return cudaSuccess;
    e = ask(number);
    if (e == cudaSuccess) k.store(*number + 1, std::memory_order_relaxed);
    return e;
  }
};

// ---- rowquant.cu
enum RowOut : int { kOutE4M3 = 0, kOutNvfp4 = 1, kOutMxfp4 = 2 };

struct RowQuantArgs {
  const uint16_t *x;         // bf16 [rows, cols] (the gated form: [rows, 2 cols], gate then up)
  const uint16_t *residual;  // norm: bf16 [rows, cols] or null
  const uint16_t *weight;    // norm: bf16 [cols]
  uint16_t *residual_out;    // norm: bf16 [rows, cols], null exactly when residual is
  float eps;                 // norm
  uint8_t *q;                // E4M3 codes [rows, cols], or FP4 codes [rows, cols / 2]
  uint8_t *blocks;           // FP4: block scales in tiles of 128 rows x 4 scales
  float *scales;             // E4M3 and nvfp4: one per row
  int64_t rows, cols;
  int32_t *status;
  // set by the launch
  int chunks, tiles;  // of a row: chunks of 16 elements, tiles of block scales
  bool wide;          // x, residual and residual_out are 32-byte aligned
};

cudaError_t launch_rowquant_plain(RowOut out, const RowQuantArgs &a, cudaStream_t st);
cudaError_t launch_rowquant_norm(RowOut out, const RowQuantArgs &a, cudaStream_t st);
cudaError_t launch_rowquant_gate(RowOut out, const RowQuantArgs &a, cudaStream_t st);
// E2M1 codes, two per byte, to E4M3 codes of the same values, one per byte.
cudaError_t launch_fp4_unpack(const uint8_t *q, int64_t bytes, uint8_t *out, cudaStream_t st);

// ---- gemm_micro.cu
struct MicroGemmArgs {
  const uint8_t *xq, *xb, *wq, *wb;  // codes [M or N, K / 2] and block-scale tiles
  const float *xs, *ws;              // row scales, or null (1)
  int x_vec, w_vec;                  // one per row, or one for all
  uint16_t *y;                       // bf16 [M, N]
  int M, N, K;
  int32_t *status;
};
cudaError_t launch_micro_gemm(int block, const MicroGemmArgs &a, cudaStream_t st);

}  // namespace sp24
