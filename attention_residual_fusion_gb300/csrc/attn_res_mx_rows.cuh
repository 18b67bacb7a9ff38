// attn_res_mx_rows.cuh -- rows to and from the microscaled formats:
// quantisation, its inverse, and the residual addition + RMSNorm whose result
// is quantised.  All three are bound by memory: a group's scale needs only
// its 16 or 32 elements (two or four lanes of eight), so a row is read once
// and its codes and scales are written from the registers it was read into.
#pragma once

#include "attn_res_mx.cuh"

namespace attn_res_dev {

// ---- quantisation -------------------------------------------------------------------
//
// A warp takes 256 columns of the four rows r, r + 32, r + 64, r + 96 of a
// 128-row tile: those rows' scales of four groups are the 16 consecutive
// bytes of one entry of a scale tile, so a lane stores them at once, and the
// entries of rows and groups that do not exist come out as zeros by the same
// stores.  Four 16-byte loads per lane are in flight, and six CTAs an SM: on
// 8192 x 7168 28.2 us to mxfp8, 25.4 to mxfp4 (86 % of the copy rate), 34.4 to
// nvfp4, whose quotients bound it and which spills 16 bytes a thread (with 8
// CTAs 30.6, 26.2 and 36.1: all three spill, and more).
constexpr int kMxThreads = 256;
constexpr int kMxWarpCols = 256;

struct MxRowsParams {
  const uint16_t* x;  // quantise: source
  uint16_t* out;      // dequantise: result
  int64_t x_row;
  MxView q;
  uint32_t col_chunks;  // ceil(padded cols / 256)
  uint32_t jobs;        // row tiles * 32 * col_chunks
};

template <int FMT>
__global__ void __launch_bounds__(kMxThreads, 6) attn_res_mx_quantize_kernel(const MxRowsParams p) {
  using M = Mx<FMT>;
  const int lane = threadIdx.x & 31;
  const uint32_t job = blockIdx.x * (kMxThreads / 32) + (threadIdx.x >> 5);
  grid_dep_wait();
  const float g = M::NV ? tensor_scale_of(p.q.tensor_scale) : 1.f;
  const float g6 = 6.f * g;
  if (job < p.jobs) {
    const uint32_t rest = job / p.col_chunks;
    const int r = (int)(rest & 31);
    const int64_t tile = rest >> 5;
    const int64_t vec = (int64_t)(job - rest * p.col_chunks) * 32 + lane;
    const bool in_row = vec * 8 < p.q.cols;
    uint4 v[4];
    bool ok[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t row = tile * 128 + 32 * u + r;
      ok[u] = in_row && row < p.q.rows;
      v[u] = ok[u] ? ld_row(p.x + row * p.x_row + vec * 8) : make_uint4(0, 0, 0, 0);
    }
    uint32_t codes = 0;
#pragma unroll
    for (int u = 0; u < 4; u += 2) {
      const uint32_t am = group_max2<M::LANES>(amax_pair(v[u], v[u + 1]));
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const GroupScale<FMT> s = group_scale<FMT>(e == 0 ? am << 16 : am & 0xffff0000u, g, g6);
        f32x2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = bf2_widen(vword(v[u + e], i));
        if (ok[u + e]) {
          st_codes<FMT>(p.q.data + (tile * 128 + 32 * (u + e) + r) * p.q.row_bytes, vec, encode8<FMT>(x, s));
          codes |= s.code << (8 * (u + e));
        }
      }
    }
    const uint4 words = scale_words<FMT>(codes);
    const int64_t atom = vec / M::ATOM_LANES;
    if (lane % M::ATOM_LANES == 0 && atom < p.q.group_tiles)
      *reinterpret_cast<uint4*>(p.q.scales + ((tile * p.q.group_tiles + atom) * 512 + r * 16)) = words;
  }
  grid_dep_launch_dependents();
}

// ---- the inverse ---------------------------------------------------------------------

template <int FMT>
__global__ void __launch_bounds__(kMxThreads) attn_res_mx_dequantize_kernel(const MxRowsParams p) {
  using M = Mx<FMT>;
  const int lane = threadIdx.x & 31;
  const uint32_t job = blockIdx.x * (kMxThreads / 32) + (threadIdx.x >> 5);
  grid_dep_wait();
  const float g = M::NV ? tensor_scale_of(p.q.tensor_scale) : 1.f;
  if (job < p.jobs) {
    const uint32_t rest = job / p.col_chunks;
    const int r = (int)(rest & 31);
    const int64_t tile = rest >> 5;
    const int64_t vec = (int64_t)(job - rest * p.col_chunks) * 32 + lane;
    if (vec * 8 < p.q.cols) {
      const int64_t group = vec / M::LANES;
      const uint4 sc = *reinterpret_cast<const uint4*>(
          p.q.scales + ((tile * p.q.group_tiles + group / 4) * 512 + r * 16));
      Codes<FMT> c[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t row = tile * 128 + 32 * u + r;
        if (row < p.q.rows) c[u] = ld_codes<FMT>(p.q.data + row * p.q.row_bytes, vec);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t row = tile * 128 + 32 * u + r;
        if (row >= p.q.rows) break;
        const uint32_t code = (vword(sc, u) >> (8 * (int)(group % 4))) & 0xffu;
        const float s = M::NV ? e4m3_value(code) : e8m0_value(code);
        float x[8];
        decode8<FMT>(c[u], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = M::NV ? x[i] * s * g : x[i] * s;
        st_row(p.out + row * p.x_row + vec * 8,
               make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                          pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])));
      }
    }
  }
  grid_dep_launch_dependents();
}

// ---- residual addition + RMSNorm + quantisation ---------------------------------------
//
// One CTA per token row, the row in registers (VPT 16-byte vectors per
// thread); the sum of c^2 takes one CTA barrier.  CTAs behind the last row
// write the zero scale entries of the rows that pad the last 128-row tile,
// kMxPadRows of them each.  With WARP_ROWS, for many narrow rows, a warp takes
// a row (or one of the padding rows) and no barrier is needed.
constexpr int kMxNormMaxThreads = 1024;
constexpr int kMxPadRows = 8;
constexpr int kMxWarpRows = 8;  // warps of a CTA with WARP_ROWS

struct MxNormParams {
  uint16_t* prefix;
  const uint16_t* delta;
  const uint16_t* weight;
  uint16_t* norm_out;
  int64_t prefix_row, delta_row, norm_row;
  float eps, width;  // width: H
  MxView q;
};

// Eight elements of a normalised row (vector i, its eight products y) into q,
// with the group's scale; every lane takes part, those past the row's end too.
template <int FMT>
__device__ __forceinline__ void norm_store(const MxNormParams& p, int64_t t, int i, bool in_row, const f32x2 (&y)[4],
                                           float g, float g6) {
  using M = Mx<FMT>;
  uint32_t am = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) am = max(am, max(abs_bits(f2_lo(y[k])), abs_bits(f2_hi(y[k]))));
  // past the row's end nothing counts, whatever the row's statistics make of 0
  if (!in_row) am = 0;
  const GroupScale<FMT> s = group_scale<FMT>(group_max<M::LANES>(am), g, g6);
  if (in_row) {
    st_codes<FMT>(p.q.data + t * p.q.row_bytes, i, encode8<FMT>(y, s));
    if (p.norm_out)
      st_row(p.norm_out + t * p.norm_row + (int64_t)i * 8,
             make_uint4(pack_bf16x2(f2_lo(y[0]), f2_hi(y[0])), pack_bf16x2(f2_lo(y[1]), f2_hi(y[1])),
                        pack_bf16x2(f2_lo(y[2]), f2_hi(y[2])), pack_bf16x2(f2_lo(y[3]), f2_hi(y[3]))));
  }
  const uint32_t word = scale_word<FMT>(in_row ? s.code : 0u);
  const int atom = i / M::ATOM_LANES;
  if ((threadIdx.x & 31) % M::ATOM_LANES == 0 && atom < p.q.group_tiles)
    *reinterpret_cast<uint32_t*>(p.q.scales + ((t / 128) * p.q.group_tiles + atom) * 512 + (t % 32) * 16 +
                                 (t % 128) / 32 * 4) = word;
}

// A row whose mean square (with eps) fp32 does not hold: it overflows, from
// values of 2^64 / sqrt(H) on, or lies below this, where squares lose bits to
// underflow.
constexpr float kMxLeastMean = 0x1p-100f;

// Such a row, from memory again: scaled by the power of two that brings its
// largest value to 2^30 (less where eps counts) before the statistics are
// taken.  y is the same function of the scaled row and of eps times the
// scale's square, and the scaled values are exact but for those whose y lies
// below 2^-156 times the weight.  (Reading the row again costs the other rows
// no registers; with the scaling in the registers' copy 8192 x 7168 took 64.7
// us to mxfp8 instead of 63.4.)  `part` is shared by the row's threads.
template <int FMT, bool WARP_ROWS>
__device__ __forceinline__ void norm_scaled_row(const MxNormParams& p, int64_t t, float* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = WARP_ROWS ? 32 : blockDim.x;
  const int tid = WARP_ROWS ? lane : threadIdx.x;
  const int nv = (int)(p.q.cols / 8);
  const float g = Mx<FMT>::NV ? tensor_scale_of(p.q.tensor_scale) : 1.f;
  uint16_t* const prow = p.prefix + t * p.prefix_row;
  auto current = [&](int i) {
    if (i >= nv) return make_uint4(0, 0, 0, 0);
    const uint4 c = ld_row(prow + (int64_t)i * 8);
    return p.delta ? add_bf16x8(c, ld_row(p.delta + t * p.delta_row + (int64_t)i * 8)) : c;
  };
  uint32_t am = 0;  // largest |c|, as a bf16 pattern
#pragma unroll 1
  for (int i = tid; i < nv; i += team) {
    const uint4 c = current(i);
    const uint32_t m = amax_pair(c, c);
    am = max(am, max(m & 0xffffu, m >> 16));
  }
  am = __reduce_max_sync(0xffffffffu, am);
  if constexpr (!WARP_ROWS) {
    __syncthreads();
    if (lane == 0) part[warp] = __uint_as_float(am);
    __syncthreads();
    am = __reduce_max_sync(0xffffffffu, lane < (int)(blockDim.x >> 5) ? __float_as_uint(part[lane]) : 0u);
  }
  float by = 1.f;
  if (am != 0) {  // (infinities and NaN stay what they are)
    const int e = am >= 0x80u ? (int)(am >> 7) - 127 : 31 - __clz(am) - 133;  // 2^e <= largest |c| < 2^(e + 1)
    int k = min(30 - e, 126);
    if (p.eps > 0.f) k = min(k, (100 - ilogbf(p.eps)) >> 1);
    by = __uint_as_float((uint32_t)(k + 127) << 23);
  }
  float tot = 0.f;
#pragma unroll 1
  for (int i = tid; i < nv; i += team) {
    const uint4 c = current(i);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float lo = bf_lo(vword(c, k)) * by, hi = bf_hi(vword(c, k)) * by;
      tot += lo * lo + hi * hi;
    }
  }
  tot = warp_sum(tot);
  if constexpr (!WARP_ROWS) {
    __syncthreads();
    if (lane == 0) part[warp] = tot;
    __syncthreads();
    tot = warp_sum(lane < (int)(blockDim.x >> 5) ? part[lane] : 0.f);
  }
  const float rstd = __frsqrt_rn(tot / p.width + p.eps * by * by);
  // every lane as long as any has a group (the last scale tile's among them)
  const int last = (int)(p.q.group_tiles * Mx<FMT>::ATOM_LANES);
#pragma unroll 1
  for (int i0 = 0; i0 < last; i0 += team) {
    const int i = i0 + tid;
    const uint4 c = current(i);
    const uint4 w = i < nv ? ld_weight(p.weight + (int64_t)i * 8) : make_uint4(0, 0, 0, 0);
    f32x2 y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      y[k] = f2_mul(f2_mul(f2_mul(bf2_widen(vword(c, k)), f2_make(by, by)), bf2_widen(vword(w, k))),
                    f2_make(rstd, rstd));
    norm_store<FMT>(p, t, i, i < nv, y, g, 6.f * g);
    if (p.delta && i < nv) st_row(prow + (int64_t)i * 8, c);
  }
}

template <int FMT, int VPT, int MAX_THREADS, int MIN_CTAS, bool WARP_ROWS>
__global__ void __launch_bounds__(MAX_THREADS, MIN_CTAS)
    attn_res_mx_norm_kernel(const MxNormParams p) {
  using M = Mx<FMT>;
  __shared__ float part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = WARP_ROWS ? 32 : blockDim.x;  // threads of a row
  const int tid = WARP_ROWS ? lane : threadIdx.x;
  const int64_t t = WARP_ROWS ? (int64_t)blockIdx.x * kMxWarpRows + warp : (int64_t)blockIdx.x;
  const int nv = (int)(p.q.cols / 8);
  if (t >= p.q.rows) {
    grid_dep_wait();
    grid_dep_launch_dependents();
    constexpr int kRows = WARP_ROWS ? 1 : kMxPadRows;
    const int64_t first = p.q.rows + (t - p.q.rows) * kRows;
    const int64_t last = (p.q.rows + 127) / 128 * 128;
    for (int64_t row = first; row < first + kRows && row < last; ++row)
      for (int64_t a = tid; a < p.q.group_tiles; a += team)
        *reinterpret_cast<uint32_t*>(p.q.scales + ((row / 128) * p.q.group_tiles + a) * 512 +
                                     (row % 32) * 16 + (row % 128) / 32 * 4) = 0u;
    return;
  }
  uint4 w[VPT], c[VPT];
  grid_dep_wait();
  const float g = M::NV ? tensor_scale_of(p.q.tensor_scale) : 1.f;
  const float g6 = 6.f * g;
  uint16_t* const prow = p.prefix + t * p.prefix_row;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = tid + v * team;
    c[v] = i < nv ? ld_row(prow + (int64_t)i * 8) : make_uint4(0, 0, 0, 0);
  }
  if (p.delta) {
    uint4 d[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = tid + v * team;
      d[v] = i < nv ? ld_row(p.delta + t * p.delta_row + (int64_t)i * 8) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) c[v] = add_bf16x8(c[v], d[v]);
  }
  grid_dep_launch_dependents();
  // after the addend, whose registers they take
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = tid + v * team;
    w[v] = i < nv ? ld_weight(p.weight + (int64_t)i * 8) : make_uint4(0, 0, 0, 0);
  }
  f32x2 sq2 = f2_make(0.f, 0.f);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const f32x2 x = bf2_widen(vword(c[v], k));
      sq2 = f2_fma(x, x, sq2);
    }
  }
  float tot = warp_sum(f2_lo(sq2) + f2_hi(sq2));
  if constexpr (!WARP_ROWS) {
    if (lane == 0) part[warp] = tot;
    __syncthreads();
    tot = warp_sum(lane < (int)(blockDim.x >> 5) ? part[lane] : 0.f);
  }
  // (the quotient itself: 1 / H as a factor would put its rounding into every row)
  const float mean = tot / p.width + p.eps;
  // (the same in every thread of the row)
  if (!(mean >= kMxLeastMean && mean < __int_as_float(0x7f800000))) {
    norm_scaled_row<FMT, WARP_ROWS>(p, t, part);
    return;
  }
  const float rstd = __frsqrt_rn(mean);
  // The widened elements of the sum are not kept for the products below, where
  // registers are scarce: kept, 8192 x 7168 took 72.1 us to nvfp4 instead of
  // 65.4 and 512 x 65536 75.1 to mxfp8 instead of 55.2 (spills); with up to two
  // vectors a thread and power-of-two scales they are (512 x 4096 to mxfp4 3.03
  // instead of 3.12).
  if constexpr (VPT > 2 || M::NV) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) asm("" : "+r"(c[v].x), "+r"(c[v].y), "+r"(c[v].z), "+r"(c[v].w));
  }
  const f32x2 r2 = f2_make(rstd, rstd);
  uint8_t* const qrow = p.q.data + t * p.q.row_bytes;
  uint8_t* const srow =
      p.q.scales + (t / 128) * p.q.group_tiles * 512 + (t % 32) * 16 + (t % 128) / 32 * 4;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = tid + v * team;
    const bool in_row = i < nv;
    f32x2 y[4];
    uint32_t am = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // c * w is exact in fp32 (two 8-bit significands), so y is rounded once
      y[k] = f2_mul(f2_mul(bf2_widen(vword(c[v], k)), bf2_widen(vword(w[v], k))), r2);
      am = max(am, max(abs_bits(f2_lo(y[k])), abs_bits(f2_hi(y[k]))));
    }
    // past the row's end nothing counts, whatever the row's statistics make of 0
    if (!in_row) am = 0;
    const GroupScale<FMT> s = group_scale<FMT>(group_max<M::LANES>(am), g, g6);
    if (in_row) {
      st_codes<FMT>(qrow, i, encode8<FMT>(y, s));
      if (p.norm_out)
        st_row(p.norm_out + t * p.norm_row + (int64_t)i * 8,
               make_uint4(pack_bf16x2(f2_lo(y[0]), f2_hi(y[0])), pack_bf16x2(f2_lo(y[1]), f2_hi(y[1])),
                          pack_bf16x2(f2_lo(y[2]), f2_hi(y[2])), pack_bf16x2(f2_lo(y[3]), f2_hi(y[3]))));
      if (p.delta) st_row(prow + (int64_t)i * 8, c[v]);
    }
    const uint32_t word = scale_word<FMT>(in_row ? s.code : 0u);
    const int atom = i / M::ATOM_LANES;
    if (lane % M::ATOM_LANES == 0 && atom < p.q.group_tiles)
      *reinterpret_cast<uint32_t*>(srow + (int64_t)atom * 512) = word;
  }
}

}  // namespace attn_res_dev
