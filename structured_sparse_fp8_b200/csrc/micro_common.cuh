// micro_common.cuh -- device helpers of the block-scaled FP4 formats.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace sp24 {

// Scale (row, block) of a [rows, n] grid of block scales, in tiles of 128
// rows x 4 scales (512 bytes; `tiles` = ceil(n / 4) of them per row band).
__device__ __forceinline__ int64_t block_scale_offset(int64_t row, int64_t blk, int64_t tiles) {
  return ((row >> 7) * tiles + (blk >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (blk & 3);
}

// The value of a non-negative E4M3 code.
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(code)));
  return __half2float(__ushort_as_half(static_cast<uint16_t>(h2)));
}

// E2M1 codes of 8 fp32 values (nearest, ties to the even code, saturating at
// 6), element i in bits 4i .. 4i + 3.
__device__ __forceinline__ uint32_t e2m1_codes8(const float *v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// E4M3 codes of 4 fp32 values, element i in byte i.
__device__ __forceinline__ uint32_t e4m3_codes4(const float *v) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]));
  return r;
}

}  // namespace sp24
