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
// Such stages read and write each element once and are bound by memory, next
// by how many rows an SM has in flight (registers) and by instruction issue: a
// thread takes 16 elements at a time (a block of nvfp4, half one of mxfp4, a
// 32-byte access), so that a block's scale is worked out once, and calculates
// on packed pairs.  A row is held in registers from its one read to its last
// write: a warp per row up to 1024 columns, a CTA of as many warps as the row
// needs up to 32768, and beyond that a CTA that reads the row again for the
// second pass.  (8 elements a thread: norm to E4M3, 4096 x 4096, 21.4 us
// against 18.9.  Plain rows held as values, not as bf16 words: quantiser to
// nvfp4, 12288 x 4096, 29.3 us against 23.9.  Rows brought ahead into shared
// memory by bulk copies of CTAs that stay: norm 43 us against 35 at 4096 x
// 8192.)  Measured with cold inputs, bytes read and written over the time:
// norm to E4M3, 4096 x 4096, 18.9 us (6.2 TB/s), 1 x 4096 1.8 us; gate to
// mxfp4, 4096 x 14336, 39.8 us (6.7 TB/s); quantiser, 12288 x 4096, to mxfp4
// 20.4 us (6.3 TB/s), to nvfp4 23.9 (5.4).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "micro_common.cuh"
#include "micro_kernels.h"
#include "sm100_ptx.cuh"
#include "sp24.h"

namespace sp24 {

namespace {

enum RowSrc : int { kSrcPlain = 0, kSrcNorm = 1, kSrcGate = 2 };

constexpr int kChunk = 16;                   // elements a thread takes at a time
constexpr int kWarpRows = 8;                 // rows of a CTA in the warp-per-row form
constexpr float kRowFloor = 0x1.5p-89f;      // 2688 * 2^-100
constexpr float kInf = __builtin_huge_valf();

// 16 bf16 values.
struct Raw {
  uint32_t w[8];
};
// ld.global and not .nc: residual_out may be x or residual.  One 32-byte load
// where the row's address allows (all lanes alike), else two of 16 bytes,
// through L1, where they meet.
__device__ __forceinline__ Raw ld_row(const uint16_t *p, bool wide) {
  Raw r;
  if (wide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
                 : "l"(p));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r.w[4 * i]), "=r"(r.w[4 * i + 1]), "=r"(r.w[4 * i + 2]), "=r"(r.w[4 * i + 3])
                   : "l"(p + 8 * i));
  }
  return r;
}
__device__ __forceinline__ void st_row(uint16_t *p, const Raw &r, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]), "r"(r.w[3]),
                 "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7]), "l"(p)
                 : "memory");
  } else {
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
  }
}
__device__ __forceinline__ Raw raw_of(const uint4 &a, const uint4 &b) {
  return Raw{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// Two fp32 values in a register pair, and the packed operations on them: such
// stages are bound by instruction issue next to memory, and these halve it.
typedef uint64_t f2;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split2(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 both(float v) { return pack2(v, v); }

// 16 values of a chunk.
struct Chunk {
  f2 v[8];
  __device__ __forceinline__ void scale(float m) {
    const f2 mm = both(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], mm);
  }
};

__device__ __forceinline__ Chunk unpack(const Raw &r) {
  Chunk c;
#pragma unroll
  for (int i = 0; i < 8; ++i) c.v[i] = pack2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xFFFF0000u));
  return c;
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
// 1 / v to one step; results below 2^-126 are 0
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
// The largest magnitude of the chunk.
__device__ __forceinline__ float max_abs(const Chunk &c) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = split2(c.v[i]);
    m = max_abs3(m, v.x, v.y);
  }
  return m;
}

__device__ __forceinline__ float max_abs(const Raw &r) {
  __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&r.w[0]));
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&r.w[i])));
  return max_nan(__low2float(m), __high2float(m));
}

// What a thread holds of a chunk between the two passes: the values, or for
// plain rows the bf16 words as they came (half the registers).
template <int SRC>
struct Held {
  Chunk v;
  __device__ __forceinline__ Chunk values() const { return v; }
};
template <>
struct Held<kSrcPlain> {
  Raw v;
  __device__ __forceinline__ Chunk values() const { return unpack(v); }
};

// bf16(x + r): the sum of two bf16 values rounded once (fp32 holds every such
// sum that is near a rounding boundary exactly)
__device__ __forceinline__ Raw add_bf16(const Raw &x, const Raw &r) {
  Raw o;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&x.w[i]), *reinterpret_cast<const __nv_bfloat162 *>(&r.w[i]));
    o.w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return o;
}

// z = h * w, and the sum of h^2
__device__ __forceinline__ Chunk norm_values(const Raw &h, const Raw &w, f2 &sum) {
  Chunk y = unpack(h);
  const Chunk ww = unpack(w);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sum = fma2(y.v[i], y.v[i], sum);
    y.v[i] = mul2(y.v[i], ww.v[i]);
  }
  return y;
}

// g / (1 + exp(-g)) * u.  The exponential's argument is one fp32 product, so
// the result is within (1.173 |g| + 8) * 2^-23 of itself.  Codes have 3 bits at
// most, and no more of them differ from the exact value's than with a library's
// exponential (E4M3, 8.4 million normal values: 14 and 14).  The reciprocal is
// taken of (1 + exp(-g)) / 16, so that neither leaves the range of normal
// numbers while the factor is at least 2^-130 (below that, from g = -90.1 on, it
// counts as 0): u may be large.
__device__ __forceinline__ Chunk gate_values(const Raw &gv, const Raw &uv) {
  Chunk g = unpack(gv);
  const Chunk u = unpack(uv);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 a = split2(fma2(g.v[i], both(-1.4426950408889634f), both(-4.0f)));
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(a.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(a.y));
    const float2 d = split2(add2(pack2(e.x, e.y), both(0.0625f)));
    const f2 sigmoid = mul2(pack2(rcp_approx(d.x), rcp_approx(d.y)), both(0.0625f));
    g.v[i] = mul2(mul2(g.v[i], sigmoid), u.v[i]);
  }
  return g;
}

// A row's pointers (64-bit products once per row; offsets within it are 32-bit).
struct Row {
  const uint16_t *x, *residual;  // of the gated form: gate, up
  uint16_t *h;                   // the norm's sum, written and read back
  uint8_t *q, *blocks;           // blocks: scale 0 of the row; tile i is 512 i bytes on
};
template <int SRC, int OUT>
__device__ __forceinline__ Row row_of(const RowQuantArgs &p, int row) {
  Row r;
  const int64_t chunk = static_cast<int64_t>(row) * p.chunks;  // the row's first
  r.x = p.x + chunk * (kChunk * (SRC == kSrcGate ? 2 : 1));
  r.residual = SRC == kSrcGate ? r.x + p.chunks * kChunk : p.residual + chunk * kChunk;
  r.h = p.residual_out + chunk * kChunk;
  r.q = p.q + chunk * (OUT == kOutE4M3 ? kChunk : kChunk / 2);
  r.blocks = p.blocks + block_scale_offset(row, 0, p.tiles);
  return r;
}

// What chunk `c` of the row contributes: y, or z = h * w for the norm (then
// also its sum of squares; `first` adds the residual and stores h).
template <int SRC>
__device__ __forceinline__ Held<SRC> chunk_values(const RowQuantArgs &p, const Row &row, int c, bool first, f2 &sum) {
  const int at = c * kChunk;
  if constexpr (SRC == kSrcPlain) {
    return {ld_row(row.x + at, p.wide)};
  } else if constexpr (SRC == kSrcNorm) {
    const uint4 *w = reinterpret_cast<const uint4 *>(p.weight) + 2 * c;
    const uint4 w0 = __ldg(w), w1 = __ldg(w + 1);
    Raw h;
    if (first && p.residual) {
      const Raw x = ld_row(row.x + at, p.wide), r = ld_row(row.residual + at, p.wide);
      h = add_bf16(x, r);
      st_row(row.h + at, h, p.wide);
    } else {
      h = ld_row((p.residual ? row.h : row.x) + at, p.wide);
    }
    return {norm_values(h, raw_of(w0, w1), sum)};
  } else {
    const Raw g = ld_row(row.x + at, p.wide), u = ld_row(row.residual + at, p.wide);
    return {gate_values(g, u)};
  }
}

// How a row's values become codes.  Every thread works these out, so they are
// made with a refined reciprocal (within 2^-23) and not by division.
struct RowScale {
  float pre;   // factor for values of a row so small that its quotients would leave fp32's range, else 1
  float mul;   // E4M3: codes are E4M3(value * mul); nvfp4: 2688 / R; mxfp4: rstd
  float sf;    // nvfp4: block scales are E4M3(amax * sf), sf = 448 / R
};
// 1 / v: the approximation and one Newton step
__device__ __forceinline__ float rcp_refined(float v) {
  const float r = rcp_approx(v);
  return fmaf(r, fmaf(-v, r, 1.0f), r);
}

// From amax of the row's values (z for the norm) and rstd (1 but for the norm).
template <int OUT>
__device__ __forceinline__ RowScale row_scale(float amax, float rstd) {
  RowScale r;
  r.pre = 1.0f;
  r.mul = rstd;
  r.sf = 0.0f;
  if constexpr (OUT != kOutMxfp4) {
    // a row of ordinary size: its own amax decides
    const float least = OUT == kOutE4M3 ? 448.0f * 0x1p-126f : kRowFloor;
    if (amax >= 0x1p-64f && amax <= 0x1p100f && amax * rstd >= least) {
      r.sf = 448.0f * rcp_refined(amax);
    } else {
      // The row's values are multiplied by pre first, and R is scaled by it
      // before the division, which may leave fp32's range otherwise: amax is
      // at least 2^-149, so this R is at least 2^-86.
      r.pre = amax > 0x1p100f ? 0x1p-64f : 0x1p64f;
      float R = kInf;  // a row of zeros, or one whose squares all vanish: zero codes
      if (amax * rstd >= least)
        R = amax * r.pre;
      else if (amax > 0.0f && rstd > 0.0f)
        R = __fdiv_rn(least * r.pre, rstd);
      r.sf = __fdiv_rn(448.0f, R);
    }
    r.mul = OUT == kOutE4M3 ? r.sf : 6.0f * r.sf;
  }
  return r;
}
// The row's stored scale.
template <int OUT>
__device__ __forceinline__ float stored_scale(float top) {  // top = amax * rstd
  if (OUT == kOutE4M3) return top == 0.0f ? 1.0f : fmaxf(__fdiv_rn(top, 448.0f), 0x1p-126f);
  return top == 0.0f ? 1.0f : top >= kRowFloor ? __fdiv_rn(top, 2688.0f) : 0x1p-100f;
}

// Quotients of two of the row's values that are to be rounded to a code, where
// the values have few significant bits, are either on a rounding boundary of
// the code or well away from it; computed to 2^-21.5 of themselves, they are
// first rounded to fewer bits, which moves them onto the boundary, so that ties
// are decided as for the exact quotient.  That is done for plain values' block
// scales and codes and for the norm's block scales.  The norm's codes (z has 16
// bits; about 1.6 of 4096 quotients are ties) and all of the gate's quotients are
// rounded as fp32 gives them.
// Block scales, 448 amax_b / R: 17 bits for plain values (at least 2^-13 from a
// boundary otherwise), 22 for the norm's z (16 bits; 2^-20).
template <int SRC>
__device__ __forceinline__ float settle_scale(float v) {
  constexpr int drop = SRC == kSrcPlain ? 7 : SRC == kSrcNorm ? 2 : 0;
  return __uint_as_float((__float_as_uint(v) + ((1u << drop) >> 1)) & ~((1u << drop) - 1));
}
// Codes of plain values, 2688 x / (sf R), below 8: the boundaries are multiples
// of 1/4, other quotients at least 2^-13.9 from them (15 * 255 below the line);
// adding and subtracting 768 rounds to a multiple of 2^-14.
constexpr float kSettle = 768.0f;

// The E4M3 code of a value that is not negative.
__device__ __forceinline__ uint32_t e4m3_code_positive(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
  return r;
}

// Codes of one chunk whose largest magnitude is `top`, and its block's scale.
// Every lane of the warp takes part; `on` lanes store.
template <int SRC, int OUT>
__device__ __forceinline__ void encode_chunk(const RowQuantArgs &p, const Row &row, int c, bool on, const RowScale &r, Chunk y,
                                             float top) {
  const int lane = threadIdx.x & 31;
  float v[kChunk];
  auto spread = [&] {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 s = split2(y.v[i]);
      v[2 * i] = s.x, v[2 * i + 1] = s.y;
    }
  };
  if constexpr (OUT == kOutE4M3) {
    y.scale(r.mul);
    spread();
    if (on)
      *reinterpret_cast<uint4 *>(row.q + c * kChunk) =
          make_uint4(e4m3_codes4(v), e4m3_codes4(v + 4), e4m3_codes4(v + 8), e4m3_codes4(v + 12));
  } else {
    float mul;
    uint32_t code;
    if constexpr (OUT == kOutNvfp4) {
      code = e4m3_code_positive(settle_scale<SRC>(top * r.sf));
      mul = code == 0u ? 0.0f : r.mul * rcp_approx(e4m3_value(code));
    } else {
      if constexpr (SRC == kSrcNorm) {
        top *= r.mul;
        y.scale(r.mul);
      }
      top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      if (!(top < kInf) && p.status) atomicOr(p.status, SP24_STATUS_NONFINITE);
      code = static_cast<uint32_t>(max(static_cast<int>(__float_as_uint(top) >> 23) - 2, 0));
      mul = __uint_as_float((254u - code) << 23);
    }
    if constexpr (OUT == kOutNvfp4 && SRC == kSrcPlain) {
      const f2 m = both(mul), up = both(kSettle), down = both(-kSettle);
#pragma unroll
      for (int i = 0; i < 8; ++i) y.v[i] = add2(fma2(y.v[i], m, up), down);
    } else {
      y.scale(mul);
    }
    spread();
    if (on) *reinterpret_cast<uint2 *>(row.q + c * 8) = make_uint2(e2m1_codes8(v), e2m1_codes8(v + 8));
    // four block scales to a word (absent blocks of a last tile are zero)
    constexpr int lanes = OUT == kOutNvfp4 ? 1 : 2;  // per block
    uint32_t word = on ? code << (8 * (lane / lanes & 3)) : 0u;
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, lanes);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2 * lanes);
    // (c is a multiple of 4 * lanes here: tile c / (4 lanes), and one 64-bit
    // product, as tiles of a row of 2^28 columns and more pass 32-bit offsets)
    if (on && lane % (4 * lanes) == 0)
      *reinterpret_cast<uint32_t *>(row.blocks + static_cast<int64_t>(c) * (512 / (4 * lanes))) = word;
  }
}

__device__ __forceinline__ void flag(const RowQuantArgs &p) {
  if (p.status) atomicOr(p.status, SP24_STATUS_NONFINITE);
}

// NC: chunks a thread holds in registers; 0: the row is read twice.
// WARP: a warp per row, else a CTA, or gridDim.y * gridDim.z CTAs where nothing
// is summed or compared over the row.  FULL: at most 32 registers a thread, so that an
// SM's threads are all taken.
template <int SRC, int OUT, int NC, bool WARP, bool FULL>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : 1024, FULL ? 2 : 0) rowquant_kernel(const RowQuantArgs p) {
  constexpr int kLive = NC > 0 ? NC : 1;
  __shared__ float2 red[32];
  constexpr bool kNeedMax = OUT != kOutMxfp4, kNeedSum = SRC == kSrcNorm, kSegs = !WARP && NC > 0 && !kNeedMax && !kNeedSum;
  const int threads = WARP ? 32 : static_cast<int>(blockDim.x);
  const int seg = kSegs ? static_cast<int>(blockIdx.y + blockIdx.z * gridDim.y) : 0;
  const int segs = kSegs ? static_cast<int>(gridDim.y * gridDim.z) : 1;
  const int t = WARP ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x) + seg * NC * threads;
  const int row = static_cast<int>(WARP ? blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x);
  const int chunks = p.chunks;
  grid_dependency_wait();
  grid_launch_dependents();
  if (row >= static_cast<int>(p.rows)) {
    // a row past the matrix in its last band of 128: zero scales
    if (OUT != kOutE4M3 && row < (static_cast<int>(p.rows) + 127) / 128 * 128)
      for (int i = threadIdx.x % threads + seg * threads; i < p.tiles; i += threads * segs)
        *reinterpret_cast<uint32_t *>(p.blocks + block_scale_offset(row, 4 * static_cast<int64_t>(i), p.tiles)) = 0u;
    return;
  }
  // ---- first pass: values, sum of squares, largest magnitude
  const Row at = row_of<SRC, OUT>(p, row);
  Held<SRC> y[kLive];
  f2 sums = 0;
  float top[kLive], sum = 0.0f, amax = 0.0f;
  auto take = [&](int c, Held<SRC> &v, float &most) {
    v = chunk_values<SRC>(p, at, c, true, sums);
    most = max_abs(v.v);
    if constexpr (kNeedMax) amax = max_nan(amax, most);
  };
  if constexpr (NC > 0) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      y[i] = Held<SRC>{};
      top[i] = 0.0f;
      if (t + i * threads < chunks) take(t + i * threads, y[i], top[i]);
    }
  } else {
#pragma unroll 2
    for (int c = t; c < chunks; c += threads) take(c, y[0], top[0]);
  }
  if constexpr (kNeedMax || kNeedSum) {
    if constexpr (kNeedMax) amax = warp_max(amax);
    if constexpr (kNeedSum) sum = warp_sum(split2(sums).x + split2(sums).y);
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
  const RowScale r = row_scale<OUT>(amax, rstd);
  if (t == 0) {
    if constexpr (kNeedMax) p.scales[row] = stored_scale<OUT>(amax * rstd);
    if ((kNeedMax && !(amax * rstd < kInf)) || (kNeedSum && !(sum < kInf))) flag(p);
  }
  // ---- second pass: codes
  auto put = [&](int c, bool on, const Held<SRC> &held, float most) {
    Chunk v = held.values();
    if (r.pre != 1.0f) {
      most *= r.pre;
      v.scale(r.pre);
    }
    encode_chunk<SRC, OUT>(p, at, c, on, r, v, most);
  };
  if constexpr (NC > 0) {
#pragma unroll
    for (int i = 0; i < NC; ++i) put(t + i * threads, t + i * threads < chunks, y[i], top[i]);
  } else {
    // a warp's lanes stay together: they share blocks
#pragma unroll 2
    for (int c0 = t & ~31; c0 < chunks; c0 += threads) {
      const int c = c0 + (t & 31);
      Held<SRC> v{};
      f2 none = 0;
      if (c < chunks) v = chunk_values<SRC>(p, at, c, false, none);
      put(c, c < chunks, v, max_abs(v.v));
    }
  }
}

template <typename... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, unsigned threads, uint32_t smem, cudaStream_t st,
                             Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr unsigned kMaxGridY = 65535;

template <int SRC, int OUT, int NC, bool WARP, bool FULL = false>
cudaError_t launch_form(const RowQuantArgs &a, unsigned grid, unsigned threads, cudaStream_t st, unsigned segs = 1) {
  // segments along y, past its limit along z too (then the last ones may lie
  // behind the row, where they do nothing)
  const unsigned z = (segs + kMaxGridY - 1) / kMaxGridY;
  return launch_dependent(rowquant_kernel<SRC, OUT, NC, WARP, FULL>, dim3(grid, (segs + z - 1) / z, z), threads, 0, st, a);
}

template <int SRC, int OUT>
cudaError_t launch_out(const RowQuantArgs &a, cudaStream_t st) {
  const int64_t rows = OUT == kOutE4M3 ? a.rows : (a.rows + 127) / 128 * 128;
  const int chunks = a.chunks;
  if (chunks <= 64) {
    const unsigned grid = static_cast<unsigned>((rows + kWarpRows - 1) / kWarpRows);
    if (chunks <= 32) return launch_form<SRC, OUT, 1, true>(a, grid, 32 * kWarpRows, st);
    return launch_form<SRC, OUT, 2, true>(a, grid, 32 * kWarpRows, st);
  }
  const unsigned grid = static_cast<unsigned>(rows);
  if constexpr (OUT == kOutMxfp4 && SRC != kSrcNorm) {
    // nothing to reduce over the row: CTAs of up to 256 threads, a chunk each
    const int segs = (chunks + 255) / 256;
    const unsigned threads = static_cast<unsigned>((chunks + 32 * segs - 1) / (32 * segs) * 32);
    return launch_form<SRC, OUT, 1, false>(a, grid, threads, st, static_cast<unsigned>(segs));
  } else {
    // (2000 x 40000: gate to nvfp4 136 / 107 us with the registers limited, norm
    // to E4M3 118 / 120)
    if (chunks > 2 * 1024) return launch_form<SRC, OUT, 0, false, SRC == kSrcGate>(a, grid, 1024, st);
    // Two chunks a thread above 16384 columns, for plain rows (whose chunks
    // take half the registers) above 8192: quantiser to nvfp4 with two / one,
    // 2000 x 11008, 14.8 / 16.2 us; gate to E4M3, 4096 x 14336, 51.9 / 44.2,
    // norm to nvfp4 65.0 / 59.1.
    const int nc = chunks <= (SRC == kSrcPlain ? 512 : 1024) ? 1 : 2;
    const unsigned threads = static_cast<unsigned>((chunks + 32 * nc - 1) / (32 * nc) * 32);
    if (nc == 2) return launch_form<SRC, OUT, 2, false>(a, grid, threads, st);
    // Norms with a residual of up to 8192 columns, which already move 6 TB/s,
    // are better off with 38 registers than with 32 (to nvfp4, 4096 x 4096,
    // 18.0 / 18.8 us; without a residual 13.4 / 12.6).
    if constexpr (SRC == kSrcNorm && OUT != kOutMxfp4)
      if (a.residual && chunks <= 512) return launch_form<SRC, OUT, 1, false>(a, grid, threads, st);
    return launch_form<SRC, OUT, 1, false, true>(a, grid, threads, st);
  }
}

template <int SRC>
cudaError_t launch(RowOut out, RowQuantArgs a, cudaStream_t st) {
  // rows are multiples of 32 bytes, so their addresses are aligned as the bases
  const uintptr_t bases = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) |
                          reinterpret_cast<uintptr_t>(a.residual_out);
  a.wide = bases % 32 == 0;
  a.chunks = static_cast<int>(a.cols / kChunk);
  a.tiles = static_cast<int>(out == kOutNvfp4 ? (a.cols + 63) / 64 : (a.cols + 127) / 128);
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

// 16 bytes of codes a thread.  It does not release its dependents early: its
// codes may be the weights of a dense FP8 GEMM, whose loads of them do not wait
// for the kernel before.
__global__ void __launch_bounds__(256) unpack_kernel(const uint8_t *q, int64_t n, uint8_t *out) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  grid_dependency_wait();
  if (i >= n) return;
  const uint4 c = __ldcs(reinterpret_cast<const uint4 *>(q) + i);
  uint4 *o = reinterpret_cast<uint4 *>(out) + 2 * i;
  o[0] = make_uint4(widen4(c.x & 0xFFFFu), widen4(c.x >> 16), widen4(c.y & 0xFFFFu), widen4(c.y >> 16));
  o[1] = make_uint4(widen4(c.z & 0xFFFFu), widen4(c.z >> 16), widen4(c.w & 0xFFFFu), widen4(c.w >> 16));
}

}  // namespace

cudaError_t launch_rowquant_plain(RowOut out, const RowQuantArgs &a, cudaStream_t st) { return launch<kSrcPlain>(out, a, st); }
cudaError_t launch_rowquant_norm(RowOut out, const RowQuantArgs &a, cudaStream_t st) { return launch<kSrcNorm>(out, a, st); }
cudaError_t launch_rowquant_gate(RowOut out, const RowQuantArgs &a, cudaStream_t st) { return launch<kSrcGate>(out, a, st); }

cudaError_t launch_fp4_unpack(const uint8_t *q, int64_t bytes, uint8_t *out, cudaStream_t st) {
  const int64_t n = bytes / 16;  // whole: rows hold multiples of 16 bytes
  return launch_dependent(unpack_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), 256u, 0, st, q, n, out);
}

}  // namespace sp24
