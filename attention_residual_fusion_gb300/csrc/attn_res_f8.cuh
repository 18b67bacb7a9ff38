// attn_res_f8.cuh -- rows in 8 bits with a scale for each block of 128, on the
// device: group scales, element codes, the gated block's activations (see
// include/attn_res.h).
#pragma once

#include <cuda_fp8.h>

#include "attn_res.h"
#include "attn_res_common.cuh"

namespace attn_res_dev {

constexpr int kF8Block = 128;  // columns of a scale; with block scales its rows too

// A matrix as the kernels take it.  ATTN_RES_F8_ROWS: the scale of row r and
// block b of its columns is scales[b * scales_row + r]; ATTN_RES_F8_SQUARE: of
// block row i and block column b, scales[i * scales_row + b].
struct F8View {
  uint8_t* data;
  float* scales;
  int64_t row_bytes, scales_row;
  int64_t rows, cols;
};

__host__ __device__ constexpr int64_t f8_blocks(int64_t n) { return (n + kF8Block - 1) / kF8Block; }

// Bits of |x|: as integers they order like the magnitudes, with every NaN
// above infinity, so one integer maximum finds a group's amax and whether it
// holds anything that is no number.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// A group's scale from the bits of its amax, and what its codes are made with:
// its correctly rounded inverse and whether quotients may be taken with it.
struct F8Scale {
  float by, inverse;
};
__device__ __forceinline__ F8Scale f8_scale(uint32_t amax) {
  F8Scale s;
  // (at least 2^-126: below it the quotient would lose bits of the scale)
  s.by = fmaxf(__fdiv_rn(__uint_as_float(amax), 448.f), 0x1p-126f);
  if (amax == 0u) s.by = 1.f;
  s.inverse = __frcp_rn(s.by);
  if (amax >= 0x7f800000u) s.by = s.inverse = __uint_as_float(0x7fffffffu);
  return s;
}

// -(x / by) for a pair, correctly rounded: the product with the correctly
// rounded reciprocal, corrected once by its exact remainder (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990).  For a scale between 2^-96 and 2^96 nothing over- or
// underflows on the way that matters: the quotient is 448 at most, and where x
// is so small that its remainder is lost it is far below half the smallest
// code.  Negated, because so a zero keeps its sign.
__device__ __forceinline__ f32x2 f8_negated_quotient2(f32x2 x, float by, float inverse) {
  const f32x2 r = f2_make(-inverse, -inverse);
  const f32x2 q = f2_mul(x, r);
  return f2_fma(f2_fma(q, f2_make(by, by), x), r, q);
}
__device__ __forceinline__ bool f8_quotients_held(float by) { return by >= 0x1p-96f && by <= 0x1p96f; }

// Codes of four values, the first lowest.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t w;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(w)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}
// Codes of four values over one scale.
__device__ __forceinline__ uint32_t f8_codes(f32x2 lo, f32x2 hi, const F8Scale& s) {
  if (f8_quotients_held(s.by)) {
    const f32x2 a = f8_negated_quotient2(lo, s.by, s.inverse), b = f8_negated_quotient2(hi, s.by, s.inverse);
    return e4m3x4(f2_lo(a), f2_hi(a), f2_lo(b), f2_hi(b)) ^ 0x80808080u;
  }
  if (!(s.by < __int_as_float(0x7f800000))) return 0u;
  return e4m3x4(__fdiv_rn(f2_lo(lo), s.by), __fdiv_rn(f2_hi(lo), s.by), __fdiv_rn(f2_lo(hi), s.by),
                __fdiv_rn(f2_hi(hi), s.by));
}
// The values of a pair of codes (the low 16 bits), exactly.
__device__ __forceinline__ f32x2 e4m3_pair(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  return f2_make(f.x, f.y);
}

// ---- activations -------------------------------------------------------------------------

// act(g) = g / (1 + exp(-z)) with z = g (SiLU) or 2 sqrt(2 / pi) (g + 0.044715
// g^3) (GELU in its tanh form: (1 + tanh(y)) / 2 = 1 / (1 + exp(-2 y))).  The
// fast exponential is off by up to 2^-16 of itself (near |z| = 88, by a few
// units of 2^-23 for small z), the fast reciprocal by one; from z = -88.7 down
// the exponential is infinite and act(g) 0.
constexpr float kGeluScale = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

template <int ACT>
__device__ __forceinline__ float f8_gate_arg(float g) {
  if constexpr (ACT == ATTN_RES_SILU) return g;
  return kGeluScale * fmaf(kGeluCubic * g * g, g, g);
}
__device__ __forceinline__ float f8_sigmoid(float z) {
  float p;
  // (not __fdividef, which gives 0 from 2^126 on)
  asm("rcp.approx.f32 %0, %1;" : "=f"(p) : "f"(1.f + __expf(-z)));
  return p;
}

template <int ACT>
__device__ __forceinline__ float f8_act(float g) {
  return g * f8_sigmoid(f8_gate_arg<ACT>(g));
}
// act(g) and its derivative p + g p (1 - p) z'(g) of a pair.  The derivative is
// taken of g held to +-100, where it is 1 or 0, so that z' stays a number (at
// 1e19 0 x inf would come of it).
template <int ACT>
__device__ __forceinline__ void f8_act_both2(f32x2 g, f32x2& act, f32x2& slope) {
  float c[2], p[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float x = e ? f2_hi(g) : f2_lo(g);
    // (not fminf and fmaxf, which drop a NaN)
    asm("{\n\t.reg .f32 t;\n\tmin.NaN.f32 t, %1, 0f42C80000;\n\tmax.NaN.f32 %0, t, 0fC2C80000;\n\t}" : "=f"(c[e]) : "f"(x));
    p[e] = f8_sigmoid(f8_gate_arg<ACT>(c[e]));
  }
  const f32x2 c2 = f2_make(c[0], c[1]), p2 = f2_make(p[0], p[1]);
  act = f2_mul(g, p2);
  const f32x2 minus = f2_make(-1.f, -1.f), one = f2_make(1.f, 1.f);
  f32x2 t = f2_mul(f2_mul(c2, p2), f2_fma(p2, minus, one));
  if constexpr (ACT != ATTN_RES_SILU) {
    const float q = 3.f * kGeluCubic * kGeluScale;
    t = f2_mul(t, f2_fma(f2_mul(c2, f2_make(q, q)), c2, f2_make(kGeluScale, kGeluScale)));
  }
  slope = f2_fma(t, one, p2);
}

}  // namespace attn_res_dev
