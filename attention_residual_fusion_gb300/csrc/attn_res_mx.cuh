// attn_res_mx.cuh -- the microscaled formats on the device: group scales,
// element codes and the tiled scale layout (see include/attn_res.h).
#pragma once

#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "attn_res.h"
#include "attn_res_common.cuh"

namespace attn_res_dev {

// ---- bounded waits ----------------------------------------------------------------------

// The bounded waits of these kernels: as wait_or_flag, with the clock (whose
// reading takes longer than a stage's wait) looked at only from the 256th try
// on.  PEERS: the barrier is arrived on by other CTAs of the cluster too.
template <bool PEERS = false>
__device__ __forceinline__ bool phase_done(uint32_t bar, uint32_t parity) {
  if constexpr (!PEERS) return mbar_try_wait(bar, parity);
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
template <bool PEERS = false>
__device__ __forceinline__ bool phase_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns = kWaitLimitNs) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (phase_done<PEERS>(bar, parity)) return true;
    if ((it & 255u) == 0) {
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit_ns) return false;
    }
  }
}
template <bool PEERS = false>
__device__ __forceinline__ void phase_or_flag(uint32_t bar, uint32_t parity, bool& failed, unsigned* err,
                                              unsigned bit, uint64_t limit_ns = kWaitLimitNs) {
  if (failed || phase_wait<PEERS>(bar, parity, limit_ns)) return;
  failed = true;
  atomicOr(err, bit);
}

// ---- formats ------------------------------------------------------------------------------

template <int FMT>
struct Mx {
  static constexpr bool FP8 = FMT == ATTN_RES_MXFP8;
  static constexpr bool NV = FMT == ATTN_RES_NVFP4;
  static constexpr int GROUP = NV ? 16 : 32;
  static constexpr int LANES = GROUP / 8;        // lanes of one group, 8 elements each
  static constexpr int ATOM_LANES = 4 * LANES;   // lanes of four groups (one scale word)
  static constexpr int BITS = FP8 ? 8 : 4;
  static constexpr int TOP_EXP = FP8 ? 8 : 2;    // 448 = 1.75 * 2^8, 6 = 1.5 * 2^2
  static constexpr uint32_t TOP_MANT = FP8 ? 0x600000u : 0x400000u;
};

__host__ __device__ constexpr int mx_group(int fmt) { return fmt == ATTN_RES_NVFP4 ? 16 : 32; }
__host__ __device__ constexpr int mx_bits(int fmt) { return fmt == ATTN_RES_MXFP8 ? 8 : 4; }
// Tiles of four groups along a row.
__host__ __device__ constexpr int64_t mx_group_tiles(int fmt, int64_t cols) {
  return (cols / mx_group(fmt) + 3) / 4;
}

// Bits of |x|: as integers they order like the magnitudes, with every NaN
// above infinity, so one integer maximum finds the group's amax and its
// non-finite members at once.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3);
  return __half2float(__half(h));
}
// 2^(code - 127); 255 is NaN, 0 the subnormal 2^-127.
__device__ __forceinline__ float e8m0_value(uint32_t code) {
  return __uint_as_float(code == 0u ? 0x00400000u : code == 255u ? 0x7fffffffu : code << 23);
}

// The scale of a group from the bits of its amax: the code, what turns the
// elements into code values, and a mask that clears the codes of a group
// without a usable scale (not finite, or a product of scales of 0).
template <int FMT>
struct GroupScale {
  uint32_t code;
  float by;       // MX: times this power of two; NVFP4: divided by this
  float inverse;  // NVFP4: 1 / by, correctly rounded
  uint32_t keep;
};

template <int FMT>
__device__ __forceinline__ GroupScale<FMT> group_scale(uint32_t amax, float g, float g6) {
  using M = Mx<FMT>;
  GroupScale<FMT> s;
  const bool bad = amax >= 0x7f800000u;
  if constexpr (M::NV) {
    const uint32_t c = (uint32_t)__nv_cvt_float_to_fp8(__uint_as_float(amax) / g6, __NV_SATFINITE, __NV_E4M3);
    s.code = bad ? 0x7fu : c;
    s.by = e4m3_value(c) * g;
    s.inverse = 1.f / s.by;
    s.keep = !bad && s.by > 0.f ? 0xffffffffu : 0u;
  } else {
    // amax = m * 2^E with 1 <= m < 2: the smallest 2^e with amax <= TOP * 2^e
    // has e = E - TOP_EXP, or one more where m is above TOP's mantissa (the
    // sum below then carries into the exponent)
    const int c = max((int)((amax + (0x7fffffu - M::TOP_MANT)) >> 23) - M::TOP_EXP, 0);
    s.code = bad ? 255u : (uint32_t)c;
    s.by = __uint_as_float((uint32_t)(254 - c) << 23);
    s.inverse = 0.f;
    s.keep = bad ? 0u : 0xffffffffu;
  }
  return s;
}

// -(x / by) for a pair, correctly rounded: the product with the correctly
// rounded reciprocal, corrected once by its exact remainder (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990): 3 instructions a pair in place of two divisions.  Nothing
// over- or underflows on the way that matters: the divisor is between 2^-96
// and 2^96, the quotient below 9 (the group's scale is not saturated: 6 times
// what its rounding takes off, 17/16 at most for a normal e4m3 scale and below
// 1.5 for the subnormal ones; the conversion saturates what is above 6), and
// where x is so small that its remainder is lost, the quotient is far below
// half the smallest code.  Negated, because so a zero keeps its sign (0 - 0 is
// +0 only in the remainder).
__device__ __forceinline__ f32x2 negated_quotient2(f32x2 x, float by, float inverse) {
  const f32x2 r = f2_make(-inverse, -inverse);
  const f32x2 q = f2_mul(x, r);
  return f2_fma(f2_fma(q, f2_make(by, by), x), r, q);
}

// Codes of eight elements: 8 bytes (MXFP8) or 4 (e2m1, the even column low).
template <int FMT>
struct Codes {
  uint32_t w[Mx<FMT>::FP8 ? 2 : 1];
};

// x: four pairs of neighbouring elements.
template <int FMT>
__device__ __forceinline__ Codes<FMT> encode8(const f32x2 (&x)[4], const GroupScale<FMT>& s) {
  using M = Mx<FMT>;
  f32x2 v[4];
  if constexpr (M::NV) {
    if (s.code < 0x7eu && s.by >= 0x1p-96f && s.by <= 0x1p96f) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = negated_quotient2(x[i], s.by, s.inverse);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = f2_make(-(f2_lo(x[i]) / s.by), -(f2_hi(x[i]) / s.by));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_mul(x[i], f2_make(s.by, s.by));
  }
  Codes<FMT> c;
  if constexpr (M::FP8) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm("{\n\t.reg .b16 a, b;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
          "mov.b32 %0, {a, b};\n\t}"
          : "=r"(c.w[h])
          : "f"(f2_lo(v[2 * h])), "f"(f2_hi(v[2 * h])), "f"(f2_lo(v[2 * h + 1])), "f"(f2_hi(v[2 * h + 1])));
    c.w[0] &= s.keep;
    c.w[1] &= s.keep;
  } else {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(c.w[0])
        : "f"(f2_lo(v[0])), "f"(f2_hi(v[0])), "f"(f2_lo(v[1])), "f"(f2_hi(v[1])), "f"(f2_lo(v[2])),
          "f"(f2_hi(v[2])), "f"(f2_lo(v[3])), "f"(f2_hi(v[3])));
    if constexpr (M::NV) c.w[0] ^= 0x88888888u;  // the codes' signs
    c.w[0] &= s.keep;
  }
  return c;
}

template <int FMT>
__device__ __forceinline__ void decode8(const Codes<FMT>& c, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2_raw h;
    if constexpr (Mx<FMT>::FP8)
      h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c.w[i / 2] >> (16 * (i % 2))), __NV_E4M3);
    else
      h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(c.w[0] >> (8 * i)), __NV_E2M1);
    const float2 f = __half22float2(__half2(h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// The largest magnitudes of eight bf16 values each of two rows, as 16-bit
// patterns (a's low), which order like the magnitudes too: two at a time.
__device__ __forceinline__ uint32_t amax_pair(const uint4& a, const uint4& b) {
  constexpr uint32_t kAbs = 0x7fff7fffu;
  const uint32_t ma = __vmaxu2(__vmaxu2(a.x & kAbs, a.y & kAbs), __vmaxu2(a.z & kAbs, a.w & kAbs));
  const uint32_t mb = __vmaxu2(__vmaxu2(b.x & kAbs, b.y & kAbs), __vmaxu2(b.z & kAbs, b.w & kAbs));
  return __vmaxu2(__byte_perm(ma, mb, 0x5410), __byte_perm(ma, mb, 0x7632));
}
template <int LANES>
__device__ __forceinline__ uint32_t group_max2(uint32_t v) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) v = __vmaxu2(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The scale word of four neighbouring groups, in the first lane of every
// ATOM_LANES lanes (the other lanes' results are not used).
template <int FMT>
__device__ __forceinline__ uint32_t scale_word(uint32_t code) {
  constexpr int L = Mx<FMT>::LANES;
  code |= __shfl_down_sync(0xffffffffu, code, L) << 8;
  code |= __shfl_down_sync(0xffffffffu, code, 2 * L) << 16;
  return code;
}
// The same for four rows at once, whose codes are the bytes of `codes`: the
// words of the rows, a 4 x 4 transpose of bytes over four lanes.
template <int FMT>
__device__ __forceinline__ uint4 scale_words(uint32_t codes) {
  constexpr int L = Mx<FMT>::LANES;
  const uint32_t b = __shfl_down_sync(0xffffffffu, codes, L);
  const uint32_t lo = __byte_perm(codes, b, 0x5140);  // rows 0, 1 of two groups
  const uint32_t hi = __byte_perm(codes, b, 0x7362);  // rows 2, 3
  const uint32_t lo2 = __shfl_down_sync(0xffffffffu, lo, 2 * L);
  const uint32_t hi2 = __shfl_down_sync(0xffffffffu, hi, 2 * L);
  return make_uint4(__byte_perm(lo, lo2, 0x5410), __byte_perm(lo, lo2, 0x7632), __byte_perm(hi, hi2, 0x5410),
                    __byte_perm(hi, hi2, 0x7632));
}

template <int FMT>
__device__ __forceinline__ void st_codes(uint8_t* row, int64_t vec, const Codes<FMT>& c) {
  if constexpr (Mx<FMT>::FP8)
    *reinterpret_cast<uint2*>(row + vec * 8) = make_uint2(c.w[0], c.w[1]);
  else
    *reinterpret_cast<uint32_t*>(row + vec * 4) = c.w[0];
}
template <int FMT>
__device__ __forceinline__ Codes<FMT> ld_codes(const uint8_t* row, int64_t vec) {
  Codes<FMT> c;
  if constexpr (Mx<FMT>::FP8) {
    const uint2 v = *reinterpret_cast<const uint2*>(row + vec * 8);
    c.w[0] = v.x;
    c.w[1] = v.y;
  } else {
    c.w[0] = *reinterpret_cast<const uint32_t*>(row + vec * 4);
  }
  return c;
}

// Microscaled matrix as the kernels take it.
struct MxView {
  uint8_t* data;
  uint8_t* scales;
  const float* tensor_scale;  // may be null (1)
  int64_t row_bytes;
  int64_t rows, cols;
  int64_t group_tiles;  // scale tiles along a row
};

__device__ __forceinline__ float tensor_scale_of(const float* g) { return g ? __ldg(g) : 1.f; }

}  // namespace attn_res_dev
