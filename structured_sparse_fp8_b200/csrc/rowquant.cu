// rowquant.cu -- row stages with a quantised output: the plain quantiser to
// block-scaled FP4, the root-mean-square norm with the residual's addition,
// and the gated activation.
//
// Value of an element before quantisation:
//   plain   y = x
//   norm    h = bf16(x + residual); y = h * rstd * w, rstd = 1 / sqrt(mean(h^2) + eps)
//   gate    y = g / (1 + exp(-g)) * u
// Quantisation:
//   E4M3    s = max(amax|y| / 448, 2^-126) (1 for a zero row), q = E4M3(y / s)
//   nvfp4   R = max(amax|y|, 2688 * 2^-100), s = R / 2688 (1 for a zero row);
//           per block of 16: sf = E4M3(448 amax / R), q = E2M1(2688 y / (sf R))
//           (0 where sf = 0), so that a value is q * sf * s
//   mxfp4   per block of 32: e = floor(log2 amax) - 2, q = E2M1(y / 2^e)
// The norm is of the stored (bf16) sum, which is what the next block adds to.
// Sums and scales are fp32.
//
// All but the last are quotients of two values of the row, so the norm's rstd
// cancels out of its codes and block scales: z = h * w is what is quantised
// (exact in fp32), sum h^2 and amax|z| come from one pass over the row, and
// rstd enters the row's scale only.
//
// Such stages read and write each element once and are bound by memory.  A
// row is held in registers from its one read to its last write, 8 elements
// (16 bytes) per thread and load, neighbouring threads on neighbouring
// chunks: a warp per row up to 1024 columns, a CTA of as many warps as the row
// needs up to 32768, and beyond that a CTA that reads the row again for the
// second pass.  Lanes share a block's largest value and pack four block
// scales to a word by shuffles.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "micro_common.cuh"
#include "micro_kernels.h"
#include "quant_common.cuh"
#include "sm100_ptx.cuh"
#include "sp24.h"

namespace sp24 {

namespace {

enum RowSrc : int { kSrcPlain = 0, kSrcNorm = 1, kSrcGate = 2 };

constexpr int kChunk = 8;                    // elements per thread and load
constexpr int kWarpRows = 8;                 // rows of a CTA in the warp-per-row form
constexpr float kRowFloor = 0x1.5p-89f;      // 2688 * 2^-100
constexpr int64_t kFewRows = 296;             // two CTAs an SM
constexpr float kInf = __builtin_huge_valf();

// ld.global (not .nc: residual_out may be x or residual), kept out of L1
__device__ __forceinline__ uint4 ld_row(const uint16_t *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void unpack8(const uint4 &a, float *v) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// NaN wins, so that one in a row is seen in its largest value
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// max(a, |b|, |c|), a >= 0
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// 1 / v to one step, v a normal number
__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
// The largest of `so_far` (>= 0) and the chunk's magnitudes.
__device__ __forceinline__ float max_abs8(const float *y, float so_far = 0.0f) {
#pragma unroll
  for (int i = 0; i < kChunk; i += 2) so_far = max_abs3(so_far, y[i], y[i + 1]);
  return so_far;
}

// What chunk `c` of the row contributes: y, or z = h * w for the norm (then
// also its sum of squares; `first` adds the residual and stores h).
template <int SRC>
__device__ __forceinline__ void chunk_values(const RowQuantArgs &p, int64_t row, int c, bool first, float *y, float &sum) {
  const int64_t at = row * p.cols + static_cast<int64_t>(c) * kChunk;
  if constexpr (SRC == kSrcPlain) {
    unpack8(ld_row(p.x + at), y);
  } else if constexpr (SRC == kSrcNorm) {
    float w[kChunk];
    const uint4 wv = __ldg(reinterpret_cast<const uint4 *>(p.weight) + c);
    if (first && p.residual) {
      const uint4 xv = ld_row(p.x + at), rv = ld_row(p.residual + at);
      float r[kChunk];
      unpack8(xv, y);
      unpack8(rv, r);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h2 = __floats2bfloat162_rn(y[2 * i] + r[2 * i], y[2 * i + 1] + r[2 * i + 1]);
        o[i] = *reinterpret_cast<const uint32_t *>(&h2);
      }
      const uint4 ov = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4 *>(p.residual_out + at) = ov;
      unpack8(ov, y);
    } else {
      unpack8(ld_row((p.residual ? p.residual_out : p.x) + at), y);
    }
    unpack8(wv, w);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      if (first) sum = fmaf(y[i], y[i], sum);
      y[i] *= w[i];
    }
  } else {
    const int64_t g = row * 2 * p.cols + static_cast<int64_t>(c) * kChunk;
    float u[kChunk];
    const uint4 gv = ld_row(p.x + g), uv = ld_row(p.x + g + p.cols);
    unpack8(gv, y);
    unpack8(uv, u);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) y[i] = __fdividef(y[i], 1.0f + __expf(-y[i])) * u[i];
  }
}

// How a row's values become codes: one factor for the row (E4M3), or R.
struct RowScale {
  float pre;   // factor for values of a row so small that its quotients would leave fp32's range, else 1
  float mul;   // E4M3: codes are E4M3(value * mul); nvfp4: 2688 / R; mxfp4: rstd
  float sf;    // nvfp4: block scales are E4M3(amax * sf), sf = 448 / R
};

// amax of the row's values (z for the norm) and rstd (1 but for the norm) to
// the row's scale and factors.
template <int OUT>
__device__ __forceinline__ RowScale row_scale(float amax, float rstd, float &scale) {
  RowScale r;
  r.pre = amax < 0x1p-64f ? 0x1p64f : 1.0f;
  r.mul = rstd;
  r.sf = 0.0f;
  if constexpr (OUT == kOutE4M3) {
    const float s = __fdiv_rn(amax * rstd, 448.0f);
    scale = amax * rstd == 0.0f ? 1.0f : fmaxf(s, 0x1p-126f);
    r.mul = amax == 0.0f ? 0.0f : s >= 0x1p-126f ? __fdiv_rn(448.0f, amax * r.pre) : __fdiv_rn(rstd, scale) * (1.0f / r.pre);
  } else if constexpr (OUT == kOutNvfp4) {
    const float top = amax * rstd;
    scale = top == 0.0f ? 1.0f : top >= kRowFloor ? __fdiv_rn(top, 2688.0f) : 0x1p-100f;
    const float R = top >= kRowFloor ? amax * r.pre : rstd > 0.0f ? __fdiv_rn(kRowFloor, rstd) * r.pre : 1.0f;
    r.sf = __fdiv_rn(448.0f, R);
    r.mul = 6.0f * r.sf;
  } else {
    r.pre = 1.0f;
  }
  return r;
}

// Bits dropped (rounded) from a quotient of two of the row's values before it
// is rounded to a code.  Where the values have few significant bits (8 for
// plain, 16 for z) a quotient is either on a rounding boundary of the code or
// well away from it (2^-14 and 2^-20 relative), and the computed quotient,
// within 2^-22, is moved onto the boundary by rounding it to 17 (22) bits: ties
// are then decided as for the exact quotient.  (A code of nvfp4 behind the norm
// is a quotient with 20 bits below the line, as close as 2^-22 to a boundary,
// and computed to 2^-21.5: there most ties are decided so, not all.)
template <int SRC>
__device__ __forceinline__ float settle(float v) {
  if constexpr (SRC == kSrcGate) return v;
  constexpr uint32_t drop = SRC == kSrcPlain ? 7 : 2;
  return __uint_as_float((__float_as_uint(v) + (1u << (drop - 1))) & ~((1u << drop) - 1));
}

// Codes of one chunk, and its block's scale.  Every lane of the warp takes
// part; `on` lanes store.
template <int SRC, int OUT>
__device__ __forceinline__ void encode_chunk(const RowQuantArgs &p, int64_t row, int c, bool on, const RowScale &r, float *y,
                                             int64_t tiles) {
  const int lane = threadIdx.x & 31;
  if constexpr (OUT == kOutE4M3) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) y[i] = settle<SRC>(y[i] * r.mul);
    if (on) *reinterpret_cast<uint2 *>(p.q + row * p.cols + static_cast<int64_t>(c) * kChunk) = make_uint2(e4m3_codes4(y), e4m3_codes4(y + 4));
  } else {
    float mul;
    uint32_t code;
    if constexpr (OUT == kOutNvfp4) {
      float top = max_abs8(y);
      top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      code = e4m3_code(settle<SRC>(top * r.sf));
      mul = code == 0u ? 0.0f : r.mul * rcp_approx(e4m3_value(code));
    } else {
      if constexpr (SRC == kSrcNorm) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) y[i] *= r.mul;
      }
      float top = max_abs8(y);
      top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      if (!(top < kInf) && p.status) atomicOr(p.status, SP24_STATUS_NONFINITE);
      code = static_cast<uint32_t>(max(static_cast<int>(__float_as_uint(top) >> 23) - 2, 0));
      mul = __uint_as_float((254u - code) << 23);
    }
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      y[i] *= mul;
      if constexpr (OUT == kOutNvfp4) y[i] = settle<SRC>(y[i]);
    }
    if (on) *reinterpret_cast<uint32_t *>(p.q + row * (p.cols / 2) + static_cast<int64_t>(c) * 4) = e2m1_codes8(y);
    // four block scales to a word (absent blocks of a last tile are zero)
    constexpr int lanes = OUT == kOutNvfp4 ? 2 : 4;  // per block
    uint32_t word = on ? code << (8 * (lane / lanes & 3)) : 0u;
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, lanes);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2 * lanes);
    if (on && lane % (4 * lanes) == 0)
      *reinterpret_cast<uint32_t *>(p.blocks + block_scale_offset(row, c / lanes, tiles)) = word;
  }
}

__device__ __forceinline__ void flag(const RowQuantArgs &p) {
  if (p.status) atomicOr(p.status, SP24_STATUS_NONFINITE);
}

// NC: chunks a thread holds in registers; 0: the row is read twice.
// WARP: a warp per row, else a CTA, or `segs` CTAs where nothing is summed or
// compared over the row.
template <int SRC, int OUT, int NC, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : 1024) rowquant_kernel(const RowQuantArgs p, int segs) {
  constexpr int kLive = NC > 0 ? NC : 1;
  __shared__ float2 red[32];
  const int threads = WARP ? 32 : static_cast<int>(blockDim.x);
  constexpr bool kNeedMax = OUT != kOutMxfp4, kNeedSum = SRC == kSrcNorm, kSegs = !WARP && NC > 0 && !kNeedMax && !kNeedSum;
  const int seg = kSegs ? static_cast<int>(blockIdx.x % segs) : 0;
  const int t = WARP ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x) + seg * NC * threads;
  const int64_t row = WARP    ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5)
                      : kSegs ? static_cast<int64_t>(blockIdx.x / segs)
                              : static_cast<int64_t>(blockIdx.x);
  const int chunks = static_cast<int>(p.cols / kChunk);
  const int64_t tiles = OUT == kOutNvfp4 ? (p.cols + 63) / 64 : (p.cols + 127) / 128;
  grid_dependency_wait();
  grid_launch_dependents();
  if (row >= p.rows) {
    // a row past the matrix in its last band of 128: zero scales
    if (OUT != kOutE4M3 && row < (p.rows + 127) / 128 * 128)
      for (int64_t i = threadIdx.x % threads + seg * threads; i < tiles; i += threads * segs)
        *reinterpret_cast<uint32_t *>(p.blocks + block_scale_offset(row, 4 * i, tiles)) = 0u;
    return;
  }
  // ---- first pass: values, sum of squares, largest magnitude
  float y[kLive][kChunk], sum = 0.0f, amax = 0.0f;
  auto take = [&](int c, float *v) {
    chunk_values<SRC>(p, row, c, true, v, sum);
    if constexpr (kNeedMax) amax = max_abs8(v, amax);
  };
  if constexpr (NC > 0) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (t + i * threads < chunks) {
        take(t + i * threads, y[i]);
      } else {
#pragma unroll
        for (int k = 0; k < kChunk; ++k) y[i][k] = 0.0f;
      }
    }
  } else {
#pragma unroll 2
    for (int c = t; c < chunks; c += threads) take(c, y[0]);
  }
  if constexpr (kNeedMax || kNeedSum) {
    if constexpr (kNeedMax) amax = warp_max(amax);
    if constexpr (kNeedSum) sum = warp_sum(sum);
    if constexpr (!WARP) {
      const int warps = threads >> 5, lane = t & 31;
      if (lane == 0) red[t >> 5] = make_float2(amax, sum);
      __syncthreads();
      const float2 v = lane < warps ? red[lane] : make_float2(0.0f, 0.0f);
      if constexpr (kNeedMax) amax = warp_max(v.x);
      if constexpr (kNeedSum) sum = warp_sum(v.y);
    }
  }
  float rstd = 1.0f;
  if constexpr (kNeedSum) {
    const float ms = __fdiv_rn(sum, static_cast<float>(p.cols)) + p.eps;
    rstd = ms > 0.0f ? __frsqrt_rn(ms) : 0.0f;
  }
  float scale = 1.0f;
  const RowScale r = row_scale<OUT>(amax, rstd, scale);
  if (t == 0) {
    if constexpr (kNeedMax) p.scales[row] = scale;
    if ((kNeedMax && !(amax * rstd < kInf)) || (kNeedSum && !(sum < kInf))) flag(p);
  }
  // ---- second pass: codes
  auto put = [&](int c, bool on, float *v) {
    if (r.pre != 1.0f) {
#pragma unroll
      for (int k = 0; k < kChunk; ++k) v[k] *= r.pre;
    }
    encode_chunk<SRC, OUT>(p, row, c, on, r, v, tiles);
  };
  if constexpr (NC > 0) {
#pragma unroll
    for (int i = 0; i < NC; ++i) put(t + i * threads, t + i * threads < chunks, y[i]);
  } else {
    // a warp's lanes stay together: they share blocks
#pragma unroll 2
    for (int c0 = t & ~31; c0 < chunks; c0 += threads) {
      const int c = c0 + (t & 31);
      float v[kChunk] = {}, none = 0.0f;
      if (c < chunks) chunk_values<SRC>(p, row, c, false, v, none);
      put(c, c < chunks, v);
    }
  }
}

template <typename... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), unsigned grid, unsigned threads, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int SRC, int OUT, int NC, bool WARP>
cudaError_t launch_form(const RowQuantArgs &a, unsigned grid, unsigned threads, cudaStream_t st, int segs = 1) {
  return launch_dependent(rowquant_kernel<SRC, OUT, NC, WARP>, grid, threads, st, a, segs);
}

template <int SRC, int OUT>
cudaError_t launch_out(const RowQuantArgs &a, cudaStream_t st) {
  const int64_t rows = OUT == kOutE4M3 ? a.rows : (a.rows + 127) / 128 * 128;
  const int64_t chunks = a.cols / kChunk;
  if (chunks <= 128) {
    const unsigned grid = static_cast<unsigned>((rows + kWarpRows - 1) / kWarpRows);
    if (chunks <= 32) return launch_form<SRC, OUT, 1, true>(a, grid, 32 * kWarpRows, st);
    return launch_form<SRC, OUT, 4, true>(a, grid, 32 * kWarpRows, st);
  }
  const unsigned grid = static_cast<unsigned>(rows);
  if constexpr (OUT == kOutMxfp4 && SRC != kSrcNorm) {
    // nothing to reduce over the row: CTAs of up to 256 threads, two chunks
    // each (rows of over 1024 columns: far fewer CTAs than a grid may have)
    const int64_t segs = (chunks + 511) / 512;
    const unsigned threads = static_cast<unsigned>((chunks + 64 * segs - 1) / (64 * segs) * 32);
    return launch_form<SRC, OUT, 2, false>(a, static_cast<unsigned>(segs * rows), threads, st, static_cast<int>(segs));
  } else {
    if (chunks > 4 * 1024) return launch_form<SRC, OUT, 0, false>(a, grid, 1024, st);
    // few rows: as many threads on each as there are chunks; many: four (two)
    // chunks a thread, for more loads in flight
    const int nc = chunks <= 1024 && a.rows <= kFewRows ? 1 : chunks <= 2048 && a.rows <= kFewRows ? 2 : 4;
    const unsigned threads = static_cast<unsigned>((chunks + 32 * nc - 1) / (32 * nc) * 32);
    if (nc == 1) return launch_form<SRC, OUT, 1, false>(a, grid, threads, st);
    if (nc == 2) return launch_form<SRC, OUT, 2, false>(a, grid, threads, st);
    return launch_form<SRC, OUT, 4, false>(a, grid, threads, st);
  }
}

template <int SRC>
cudaError_t launch(RowOut out, const RowQuantArgs &a, cudaStream_t st) {
  if (out == kOutNvfp4) return launch_out<SRC, kOutNvfp4>(a, st);
  if (out == kOutMxfp4) return launch_out<SRC, kOutMxfp4>(a, st);
  if constexpr (SRC == kSrcPlain)
    return cudaErrorInvalidValue;  // fp8_quantize_pertoken does that
  else
    return launch_out<SRC, kOutE4M3>(a, st);
}

// The E4M3 codes of two E2M1 codes (a byte): magnitude m to the code of
// 0, 0.5, 1, 1.5, 2, 3, 4, 6 by table, sign bit 3 to bit 7.
__device__ __forceinline__ uint32_t widen4(uint32_t four) {  // 4 codes in bits 0..15
  const uint32_t sel = four & 0x7777u;
  const uint32_t mag = __byte_perm(0x3C383000u, 0x4C484440u, sel);
  const uint32_t sg = (four & 0x8u) << 4 | (four & 0x80u) << 8 | (four & 0x800u) << 12 | (four & 0x8000u) << 16;
  return mag | sg;
}

__global__ void __launch_bounds__(256) unpack_kernel(const uint8_t *q, int64_t bytes, uint8_t *out) {
  grid_dependency_wait();
  grid_launch_dependents();
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
  return launch_dependent(unpack_kernel, static_cast<unsigned>(want < 148 * 32 ? want : 148 * 32), 256u, st, q, bytes, out);
}

}  // namespace sp24
