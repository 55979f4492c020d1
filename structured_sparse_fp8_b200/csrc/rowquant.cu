// rowquant.cu -- row stages with a quantised output: the plain quantiser to
// block-scaled FP4, the root-mean-square norm with the residual's addition,
// and the gated activation.  One CTA works on one row.
//
// Value of an element before quantisation:
//   plain   y = x
//   norm    h = bf16(x + residual); y = h * rsqrt(mean(h^2) + eps) * w
//   gate    y = g / (1 + exp(-g)) * u
// Quantisation:
//   E4M3    s = max(amax|y| / 448, 2^-126) (1 for a zero row), q = E4M3(y / s)
//   nvfp4   R = max(amax|y|, 2688 * 2^-100), s = R / 2688 (1 for a zero row);
//           per block of 16: sf = E4M3(448 amax / R), q = E2M1(2688 y / (sf R))
//           (0 where sf = 0), so that a value is q * sf * s
//   mxfp4   per block of 32: e = floor(log2 amax) - 2, q = E2M1(y / 2^e)
// The norm is of the stored (bf16) sum, which is what the next block adds to.
// Sums and scales are fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "micro_common.cuh"
#include "micro_kernels.h"
#include "quant_common.cuh"
#include "sp24.h"

namespace sp24 {

namespace {

enum RowSrc : int { kSrcPlain = 0, kSrcNorm = 1, kSrcGate = 2 };

constexpr int kThreads = 256;
constexpr int kUnit = 16;                    // elements a thread takes at a time
constexpr float kRowFloor = 0x1.5p-89f;      // 2688 * 2^-100

// Largest / sum of one value per thread over the CTA.
__device__ __forceinline__ float block_max(float v, float *red) {
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < kThreads / 32; ++i) v = fmaxf(v, red[i]);
  return v;
}
__device__ __forceinline__ float block_sum(float v, float *red) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
  for (int i = 0; i < kThreads / 32; ++i) v += red[i];
  return v;
}

__device__ __forceinline__ void load_unit(const uint16_t *p, float *v) {
  const uint4 a = *reinterpret_cast<const uint4 *>(p), b = *reinterpret_cast<const uint4 *>(p + 8);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// The 16 values y of unit u.
template <int SRC>
__device__ __forceinline__ void unit_values(const RowQuantArgs &p, int64_t row, int64_t u, float rstd, float *y) {
  if constexpr (SRC == kSrcPlain) {
    load_unit(p.x + row * p.cols + u * kUnit, y);
  } else if constexpr (SRC == kSrcNorm) {
    float w[kUnit];
    load_unit((p.residual ? p.residual_out : p.x) + row * p.cols + u * kUnit, y);
    load_unit(p.weight + u * kUnit, w);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) y[i] = y[i] * rstd * w[i];
  } else {
    float up[kUnit];
    load_unit(p.x + row * 2 * p.cols + u * kUnit, y);
    load_unit(p.x + row * 2 * p.cols + p.cols + u * kUnit, up);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) y[i] = __fdividef(y[i], 1.0f + __expf(-y[i])) * up[i];
  }
}

__device__ __forceinline__ float max_abs(const float *y) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < kUnit; ++i) m = fmaxf(m, fabsf(y[i]));
  return m;
}

// fmaxf drops a NaN, so the row's sum of |y| tells whether one is there.
__device__ __forceinline__ float unit_bad(const float *y) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kUnit; ++i) s += 0.0f * y[i];
  return s;  // 0, or NaN when any is Inf or NaN
}

template <int SRC, int OUT>
__global__ void __launch_bounds__(kThreads) rowquant_kernel(const RowQuantArgs p) {
  __shared__ float red[kThreads / 32];
  const int64_t row = blockIdx.x;
  const int64_t units = p.cols / kUnit;
  const int64_t nblk = OUT == kOutMxfp4 ? units / 2 : units;
  const int64_t tiles = (nblk + 3) / 4;
  if constexpr (OUT != kOutE4M3) {
    // scales outside the matrix are zero: whole rows of the last band, and
    // the blocks past a row's last
    const int64_t from = row < p.rows ? nblk : 0;
    for (int64_t b = from + threadIdx.x; b < 4 * tiles; b += kThreads) p.blocks[block_scale_offset(row, b, tiles)] = 0;
    if (row >= p.rows) return;
  }
  float rstd = 0.0f, bad = 0.0f;
  if constexpr (SRC == kSrcNorm) {
    float sum = 0.0f;
    for (int64_t u = threadIdx.x; u < units; u += kThreads) {
      float h[kUnit];
      load_unit(p.x + row * p.cols + u * kUnit, h);
      if (p.residual) {
        float r[kUnit];
        load_unit(p.residual + row * p.cols + u * kUnit, r);
        __nv_bfloat162 o[kUnit / 2];
#pragma unroll
        for (int i = 0; i < kUnit / 2; ++i) {
          o[i] = __floats2bfloat162_rn(h[2 * i] + r[2 * i], h[2 * i + 1] + r[2 * i + 1]);
          h[2 * i] = __low2float(o[i]);
          h[2 * i + 1] = __high2float(o[i]);
        }
        uint4 *dst = reinterpret_cast<uint4 *>(p.residual_out + row * p.cols + u * kUnit);
        dst[0] = reinterpret_cast<const uint4 *>(o)[0];
        dst[1] = reinterpret_cast<const uint4 *>(o)[1];
      }
#pragma unroll
      for (int i = 0; i < kUnit; ++i) sum = fmaf(h[i], h[i], sum);
    }
    sum = block_sum(sum, red);
    const float ms = sum / static_cast<float>(p.cols) + p.eps;
    rstd = ms > 0.0f ? __frsqrt_rn(ms) : 0.0f;
    bad = 0.0f * sum;
  }
  float amax = 0.0f;
  for (int64_t u = threadIdx.x; u < units; u += kThreads) {
    float y[kUnit];
    unit_values<SRC>(p, row, u, rstd, y);
    amax = fmaxf(amax, max_abs(y));
    bad += unit_bad(y);
  }
  if (__syncthreads_or(!(bad == 0.0f)) && threadIdx.x == 0 && p.status) atomicOr(p.status, SP24_STATUS_NONFINITE);
  if constexpr (OUT != kOutMxfp4) amax = block_max(amax, red);
  float s = 1.0f, inv = 1.0f, R = 0.0f;
  if constexpr (OUT == kOutE4M3) {
    s = amax == 0.0f ? 1.0f : fmaxf(__fdiv_rn(amax, 448.0f), 0x1p-126f);
    inv = __frcp_rn(s);
  } else if constexpr (OUT == kOutNvfp4) {
    R = fmaxf(amax, kRowFloor);
    s = amax == 0.0f ? 1.0f : __fdiv_rn(R, 2688.0f);
  }
  if constexpr (OUT != kOutMxfp4) {
    if (threadIdx.x == 0) p.scales[row] = s;
  }
  // pairs of lanes hold a block of 32, so a warp's lanes stay together
  for (int64_t u0 = threadIdx.x & ~31; u0 < units; u0 += kThreads) {
    const int64_t u = u0 + (threadIdx.x & 31);
    const bool on = u < units;
    float y[kUnit];
    if (on) {
      unit_values<SRC>(p, row, u, rstd, y);
    } else {
#pragma unroll
      for (int i = 0; i < kUnit; ++i) y[i] = 0.0f;
    }
    if constexpr (OUT == kOutE4M3) {
#pragma unroll
      for (int i = 0; i < kUnit; ++i) y[i] *= inv;
      if (on)
        *reinterpret_cast<uint4 *>(p.q + row * p.cols + u * kUnit) =
            make_uint4(e4m3_codes4(y), e4m3_codes4(y + 4), e4m3_codes4(y + 8), e4m3_codes4(y + 12));
    } else {
      float top = max_abs(y), mul;
      uint32_t code;
      if constexpr (OUT == kOutNvfp4) {
        // 0.875 top, sf / 512 * R and their quotients stay in range for every
        // finite row; products with these constants are exact for bf16 values
        code = e4m3_code(__fdiv_rn(0.875f * top, R) * 512.0f);
        const float d = e4m3_value(code) * 0x1p-9f * R;
        mul = code == 0u ? 0.0f : 5.25f * __frcp_rn(d);
      } else {
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        code = static_cast<uint32_t>(max(static_cast<int>(__float_as_uint(top) >> 23) - 2, 0));
        mul = __uint_as_float((254u - code) << 23);
      }
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        float v = y[i] * mul;
        // A bf16 value over the block's divisor is a rounding boundary of E2M1
        // or at least 2^-14 away from it; v is within 2^-22 of the quotient,
        // so rounding v to 17 bits first decides ties as the exact quotient.
        if constexpr (SRC == kSrcPlain && OUT == kOutNvfp4) v = __uint_as_float((__float_as_uint(v) + 0x40u) & ~0x7Fu);
        y[i] = v;
      }
      if (on) {
        *reinterpret_cast<uint2 *>(p.q + row * (p.cols / 2) + u * 8) = make_uint2(e2m1_codes8(y), e2m1_codes8(y + 8));
        if (OUT == kOutNvfp4)
          p.blocks[block_scale_offset(row, u, tiles)] = static_cast<uint8_t>(code);
        else if ((u & 1) == 0)
          p.blocks[block_scale_offset(row, u >> 1, tiles)] = static_cast<uint8_t>(code);
      }
    }
  }
}

template <int SRC>
cudaError_t launch(RowOut out, const RowQuantArgs &a, cudaStream_t st) {
  const unsigned band = static_cast<unsigned>((a.rows + 127) / 128 * 128), rows = static_cast<unsigned>(a.rows);
  if (out == kOutE4M3) {
    if constexpr (SRC == kSrcPlain)
      return cudaErrorInvalidValue;  // fp8_quantize_pertoken does that
    else
      rowquant_kernel<SRC, kOutE4M3><<<rows, kThreads, 0, st>>>(a);
  } else if (out == kOutNvfp4) {
    rowquant_kernel<SRC, kOutNvfp4><<<band, kThreads, 0, st>>>(a);
  } else {
    rowquant_kernel<SRC, kOutMxfp4><<<band, kThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

// The E4M3 codes of two E2M1 codes (a byte): magnitude m to the code of
// 0, 0.5, 1, 1.5, 2, 3, 4, 6 by table, sign bit 3 to bit 7.
__device__ __forceinline__ uint32_t widen4(uint32_t four) {  // 4 codes in bits 0..15
  const uint32_t sel = four & 0x7777u;
  const uint32_t mag = __byte_perm(0x3C383000u, 0x4C484440u, sel);
  const uint32_t sg = (four & 0x8u) << 4 | (four & 0x80u) << 8 | (four & 0x800u) << 12 | (four & 0x8000u) << 16;
  return mag | sg;
}

__global__ void unpack_kernel(const uint8_t *q, int64_t bytes, uint8_t *out) {
  const int64_t n = bytes / 8, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) {
    const uint2 c = reinterpret_cast<const uint2 *>(q)[i];
    reinterpret_cast<uint4 *>(out)[i] =
        make_uint4(widen4(c.x & 0xFFFFu), widen4(c.x >> 16), widen4(c.y & 0xFFFFu), widen4(c.y >> 16));
  }
}

}  // namespace

cudaError_t launch_rowquant_plain(RowOut out, const RowQuantArgs &a, cudaStream_t st) { return launch<kSrcPlain>(out, a, st); }
cudaError_t launch_rowquant_norm(RowOut out, const RowQuantArgs &a, cudaStream_t st) { return launch<kSrcNorm>(out, a, st); }
cudaError_t launch_rowquant_gate(RowOut out, const RowQuantArgs &a, cudaStream_t st) { return launch<kSrcGate>(out, a, st); }

cudaError_t launch_fp4_unpack(const uint8_t *q, int64_t bytes, uint8_t *out, cudaStream_t st) {
  const int64_t want = (bytes / 8 + 255) / 256;
  unpack_kernel<<<static_cast<unsigned>(want < 148 * 8 ? want : 148 * 8), 256, 0, st>>>(q, bytes, out);
  return cudaGetLastError();
}

}  // namespace sp24
