// attn_res_mx.cuh -- the microscaled formats on the device: group scales,
// element codes and the tiled scale layout (see include/attn_res.h).
#pragma once

#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "attn_res.h"
#include "attn_res_common.cuh"

namespace attn_res_dev {

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

// The scale of a group from the bits of its amax: the code, and what the
// elements are multiplied (MX: the exact reciprocal of a power of two) or
// divided (NVFP4) by; 0 where they all become zero.
template <int FMT>
struct GroupScale {
  uint32_t code;
  float by;
};

template <int FMT>
__device__ __forceinline__ GroupScale<FMT> group_scale(uint32_t amax, float g, float g6) {
  using M = Mx<FMT>;
  GroupScale<FMT> s;
  const bool bad = amax >= 0x7f800000u;
  if constexpr (M::NV) {
    const float t = __uint_as_float(amax) / g6;
    s.code = bad ? 0x7fu : (uint32_t)__nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
    s.by = bad ? 0.f : e4m3_value(s.code) * g;
  } else {
    // amax = m * 2^E with 1 <= m < 2: the smallest 2^e with amax <= TOP * 2^e
    // has e = E - TOP_EXP, or one more where m is above TOP's mantissa
    int c = (int)(amax >> 23) - M::TOP_EXP + ((amax & 0x7fffffu) > M::TOP_MANT ? 1 : 0);
    c = c < 0 ? 0 : c;
    s.code = bad ? 255u : (uint32_t)c;
    s.by = bad ? 0.f : __uint_as_float((uint32_t)(254 - c) << 23);
  }
  return s;
}

template <int FMT>
__device__ __forceinline__ float scaled_element(float x, float by) {
  if constexpr (Mx<FMT>::NV) {
    return by > 0.f ? x / by : 0.f;
  } else {
    return x * by;
  }
}

// Codes of eight elements: 8 bytes (MXFP8) or 4 (e2m1, the even column low).
template <int FMT>
struct Codes {
  uint32_t w[Mx<FMT>::FP8 ? 2 : 1];
};

template <int FMT>
__device__ __forceinline__ Codes<FMT> encode8(const float (&x)[8], float by) {
  Codes<FMT> c;
  // by == 0: a group without a usable scale has zero elements (x itself may be NaN)
  if (by == 0.f) {
    c.w[0] = 0u;
    if constexpr (Mx<FMT>::FP8) c.w[1] = 0u;
    return c;
  }
  if constexpr (Mx<FMT>::FP8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 v = make_float2(scaled_element<FMT>(x[4 * h + 2 * i], by),
                                     scaled_element<FMT>(x[4 * h + 2 * i + 1], by));
        w |= (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3) << (16 * i);
      }
      c.w[h] = w;
    }
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = make_float2(scaled_element<FMT>(x[2 * i], by),
                                   scaled_element<FMT>(x[2 * i + 1], by));
      w |= (uint32_t)__nv_cvt_float2_to_fp4x2(v, __NV_E2M1, cudaRoundNearest) << (8 * i);
    }
    c.w[0] = w;
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

__device__ __forceinline__ void widen8(const uint4& v, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = bf_lo(vword(v, k));
    x[2 * k + 1] = bf_hi(vword(v, k));
  }
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
