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

// max(m, |a|, |b|), a NaN if there is one (its bits are then above infinity's).
__device__ __forceinline__ float amax3(float m, f32x2 v) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(f2_lo(v)), "f"(f2_hi(v)));
  return r;
}
__device__ __forceinline__ float amax3(float m, float a, float b) { return amax3(m, f2_make(a, b)); }
__device__ __forceinline__ float warp_amax(float m) {
  uint32_t r;
  asm volatile("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=r"(r) : "f"(m));
  return __uint_as_float(r);
}

// A group's scale from the bits of its amax, and its inverse, which codes are
// made with; both correctly rounded, NaN where the amax is no finite number.
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
// code; with a smaller scale the remainder may be lost, and the quotient is off
// by a unit in its last place.  Negated, because so a zero keeps its sign.
__device__ __forceinline__ f32x2 f8_negated_quotient2(f32x2 x, f32x2 by, f32x2 minus_inverse) {
  const f32x2 q = f2_mul(x, minus_inverse);
  return f2_fma(f2_fma(q, by, x), minus_inverse, q);
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
// Codes of four values over one scale that is a number (within
// f8_quotients_held those of the correctly rounded quotient).
__device__ __forceinline__ uint32_t f8_codes(f32x2 lo, f32x2 hi, float by, float inverse) {
  const f32x2 b = f2_make(by, by), r = f2_make(-inverse, -inverse);
  const f32x2 x = f8_negated_quotient2(lo, b, r), y = f8_negated_quotient2(hi, b, r);
  return e4m3x4(f2_lo(x), f2_hi(x), f2_lo(y), f2_hi(y)) ^ 0x80808080u;
}
// Over any scale (0 where that is NaN).
__device__ __forceinline__ uint32_t f8_codes(f32x2 lo, f32x2 hi, const F8Scale& s) {
  const uint32_t c = f8_codes(lo, hi, s.by, s.inverse);
  return s.by == s.by ? c : 0u;
}
// The same, correctly rounded whatever the scale.
__device__ __forceinline__ uint32_t f8_codes_far(f32x2 lo, f32x2 hi, float by) {
  const uint32_t c = e4m3x4(__fdiv_rn(f2_lo(lo), by), __fdiv_rn(f2_hi(lo), by), __fdiv_rn(f2_lo(hi), by),
                            __fdiv_rn(f2_hi(hi), by));
  return by == by ? c : 0u;
}
// The values of a pair of codes (the low 16 bits), exactly.
__device__ __forceinline__ f32x2 e4m3_pair(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  return f2_make(f.x, f.y);
}

// ---- activations -------------------------------------------------------------------------

// act(g) = g / (1 + exp(-z)) with z = g (SiLU) or 2 sqrt(2 / pi) (g + 0.044715
// g^3) (GELU in its tanh form: (1 + tanh(y)) / 2 = 1 / (1 + exp(-2 y))).
//
// The products' epilogue takes the fast exponential (f8_sigmoid), off by up to
// 2^-16 of itself near |z| = 88 and by a few units of 2^-23 for small z; from z =
// -88.7 down the exponential is infinite and act(g) 0.  The backward pass, whose
// gradients are compared with differences, has it to a few units (f8_sigmoid2).
// GELU's z comes with up to three (backward: two) units of roundings of its own,
// which exp(-z) takes |z| times: 2^-16 more near |z| = 88 on random gates.
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
// Of a pair, to a few units of 2^-23: with s = z log2(e) rounded, exp(-z) = 2^-s
// (1 + d ln 2), d what the rounding of s and of the constant took off.
__device__ __forceinline__ f32x2 f8_sigmoid2(f32x2 z) {
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr float kLog2eRest = (float)(1.4426950408889634073599 - (double)kLog2e), kLn2 = 0.69314718055994531f;
  z = f2_make(fminf(f2_lo(z), 200.f), fminf(f2_hi(z), 200.f));  // (exp(-z) is 0 there, and d a number)
  const f32x2 s = f2_mul(z, f2_make(kLog2e, kLog2e));
  const f32x2 d = f2_fma(z, f2_make(-kLog2eRest, -kLog2eRest), f2_fma(z, f2_make(-kLog2e, -kLog2e), s));
  float e[2], p[2];
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[0]) : "f"(-f2_lo(s)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[1]) : "f"(-f2_hi(s)));
  const f32x2 e2 = f2_make(e[0], e[1]), y = f2_fma(e2, f2_mul(d, f2_make(kLn2, kLn2)), e2);
  // (an infinite e may have made a NaN of it: min then gives infinity)
  const float inf = __int_as_float(0x7f800000);
  // a quarter of 1 + e, so that its reciprocal is no subnormal number
  const f32x2 q = f2_make(0.25f, 0.25f);
  const f32x2 w = f2_fma(f2_make(fminf(f2_lo(y), inf), fminf(f2_hi(y), inf)), q, q);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p[0]) : "f"(f2_lo(w)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p[1]) : "f"(f2_hi(w)));
  return f2_mul(f2_make(p[0], p[1]), q);
}

template <int ACT>
__device__ __forceinline__ float f8_act(float g) {
  return g * f8_sigmoid(f8_gate_arg<ACT>(g));
}
// act(g) and its derivative p + g p (1 - p) z'(g) of a pair.  (g^2 in z' is held
// to 10^4, where p is 1 or 0, so that z' stays a number: at g = 1e19 0 x inf would
// come of it.)
template <int ACT>
__device__ __forceinline__ void f8_act_both2(f32x2 g, f32x2& act, f32x2& slope) {
  const f32x2 one = f2_make(1.f, 1.f), minus = f2_make(-1.f, -1.f);
  f32x2 z = g, dz = one;
  if constexpr (ACT != ATTN_RES_SILU) {
    const f32x2 k = f2_make(kGeluScale, kGeluScale), kc = f2_make(kGeluScale * kGeluCubic, kGeluScale * kGeluCubic);
    const f32x2 sq = f2_mul(g, g);
    z = f2_mul(g, f2_fma(sq, kc, k));
    const f32x2 held = f2_make(fminf(f2_lo(sq), 1e4f), fminf(f2_hi(sq), 1e4f));
    dz = f2_fma(held, f2_make(3.f * kGeluScale * kGeluCubic, 3.f * kGeluScale * kGeluCubic), k);
  }
  const f32x2 p = f8_sigmoid2(z);
  act = f2_mul(g, p);
  f32x2 t = f2_mul(act, f2_fma(p, minus, one));
  slope = f2_fma(t, dz, p);
}

}  // namespace attn_res_dev
