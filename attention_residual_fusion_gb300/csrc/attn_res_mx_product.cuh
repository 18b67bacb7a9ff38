// attn_res_mx_product.cuh -- products of two microscaled matrices on the
// block-scaled tensor-core instructions (tcgen05.mma ... block_scale).
#pragma once

#include <type_traits>

#include "attn_res_mx.cuh"
#include "attn_res_tcgen05.cuh"

namespace attn_res_dev {

// ---- tcgen05, block scaled ------------------------------------------------------------

// 512 bytes of scales (32 rows of 16 bytes) to four TMEM columns, the 32
// lanes repeated in every quarter of the lanes (G = 2: in each CTA from its
// own shared memory).
template <int G>
__device__ __forceinline__ void scales_to_tmem(uint32_t tmem, uint64_t desc) {
  if constexpr (G == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

#define ATTN_RES_MMA_SCALED(GROUP, KIND)                                                         \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"                                 \
               "tcgen05.mma.cta_group::" #GROUP ".kind::" KIND                                   \
               " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                \
               "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                   \
               : "memory")
template <int FMT, int G>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (FMT == ATTN_RES_MXFP8) {
    if constexpr (G == 1) ATTN_RES_MMA_SCALED(1, "mxf8f6f4.block_scale.scale_vec::1X");
    else ATTN_RES_MMA_SCALED(2, "mxf8f6f4.block_scale.scale_vec::1X");
  } else if constexpr (FMT == ATTN_RES_MXFP4) {
    if constexpr (G == 1) ATTN_RES_MMA_SCALED(1, "mxf4.block_scale.scale_vec::2X");
    else ATTN_RES_MMA_SCALED(2, "mxf4.block_scale.scale_vec::2X");
  } else {
    if constexpr (G == 1) ATTN_RES_MMA_SCALED(1, "mxf4nvf4.block_scale.scale_vec::4X");
    else ATTN_RES_MMA_SCALED(2, "mxf4nvf4.block_scale.scale_vec::4X");
  }
}
#undef ATTN_RES_MMA_SCALED

// Scales: 32 rows of 16 bytes, not swizzled, eight rows (128 bytes) apart.
constexpr uint32_t kScalesHi = (128u >> 4) | 1u << 14;
// A 128-byte block of a K-major row: 128 e4m3 elements or 256 e2m1, taken by
// the tensor cores 32 bytes at a time.
template <int FMT>
struct ProductFmt {
  static constexpr int GROUPS = FMT == ATTN_RES_MXFP8 ? 4 : FMT == ATTN_RES_MXFP4 ? 8 : 16;
  static constexpr int ATOMS = GROUPS / 4;       // scale tiles of four groups in a block
  static constexpr int STEPS_PER_ATOM = 4 / ATOMS;  // 32-byte steps that share a scale tile
  // instruction descriptor: element types and scale type
  static constexpr uint32_t TYPE = FMT == ATTN_RES_MXFP8 ? 0u : 1u;  // e4m3 (8-bit kind), e2m1 (4-bit kinds)
  static constexpr uint32_t IDESC = TYPE << 7 | TYPE << 10 |
                                    (FMT == ATTN_RES_NVFP4 ? 0u : 1u) << 23;
  __host__ __device__ static constexpr uint32_t idesc(uint32_t m, uint32_t n) { return IDESC | (n >> 3) << 17 | (m >> 4) << 24; }
};
// The instruction's choice of scale bytes for step j of a scale tile: one,
// two or four of its four groups.
template <int FMT>
__device__ __forceinline__ uint32_t step_idesc(uint32_t idesc, int j) {
  const uint32_t id = FMT == ATTN_RES_MXFP8 ? j & 3 : FMT == ATTN_RES_MXFP4 ? (j & 1) * 2 : 0;
  return idesc | id << 4 | id << 29;
}

// The tensor cores' work on one 128-byte block of K, issued by one thread;
// addresses are its first CTA's.  P is the operand on the instruction's M side
// (128 rows a CTA), Q the one on its N side, whose scales come in QT tiles of
// 128 rows.  STEPS: the block's 32-byte steps, 4 but for the last block.
//
// The scales, to TMEM from column `sf` on: P's group tiles, then Q's, the row
// tiles of one group tile side by side.
template <int FMT, int G, int QT, int STEPS>
__device__ __forceinline__ void block_scales(uint32_t sf, uint32_t psf_lo, uint32_t qsf_lo) {
  using F = ProductFmt<FMT>;
  constexpr int ATOMS = (STEPS + F::STEPS_PER_ATOM - 1) / F::STEPS_PER_ATOM;
  constexpr uint32_t TILE = 512 >> 4;  // a scale tile, in descriptor units
#pragma unroll
  for (int t = 0; t < ATOMS; ++t) {
    scales_to_tmem<G>(sf + 4 * t, desc_of(psf_lo + TILE * t, kScalesHi));
#pragma unroll
    for (int h = 0; h < QT; ++h)
      scales_to_tmem<G>(sf + F::ATOMS * 4 + 4 * (QT * t + h),
                        desc_of(qsf_lo + TILE * (F::ATOMS * h + t), kScalesHi));
  }
}
// The products with Q rows whose scales begin `q_col` columns into Q's.
template <int FMT, int G, int QT, int STEPS>
__device__ __forceinline__ void block_steps(uint32_t acc, uint32_t sf, uint32_t q_col, uint32_t p_lo,
                                            uint32_t q_lo, uint32_t idesc, uint32_t accumulate) {
  using F = ProductFmt<FMT>;
#pragma unroll
  for (int j = 0; j < STEPS; ++j) {
    const int t = j / F::STEPS_PER_ATOM;
    mma_scaled<FMT, G>(acc, desc_of(p_lo + 2 * j, kOperandHi), desc_of(q_lo + 2 * j, kOperandHi),
                       step_idesc<FMT>(idesc, j), sf + 4 * t, sf + F::ATOMS * 4 + 4 * QT * t + q_col,
                       j > 0 ? 1u : accumulate);
  }
}
// f(integral constant) with the steps of a block of `bytes` bytes (any number
// from 128 on is a whole block).
template <class Fn>
__device__ __forceinline__ void with_steps(int bytes, Fn f) {
  if (bytes > 96) f(std::integral_constant<int, 4>());
  else if (bytes > 64) f(std::integral_constant<int, 3>());
  else if (bytes > 32) f(std::integral_constant<int, 2>());
  else f(std::integral_constant<int, 1>());
}

struct ProductParams {
  const uint8_t* a_scales;
  const uint8_t* w_scales;
  const float* a_g;
  const float* w_g;
  uint16_t* out;
  int64_t out_row;
  int64_t m, n;          // rows of a and of w
  int64_t group_tiles;   // scale tiles along a row
  int row_bytes_used;    // bytes of a row's codes
  bool early_weights;    // w may be read before the preceding kernel is complete
  unsigned* err;
};

// The two tensor scales, for the sums (x * first * second): 1 and their product.
// Where fp32 does not hold the product (scales of 1e-24 and 1e-20, say, under
// which a result may well be a number) they are the larger and the smaller:
// a product below 2^-126 has a larger scale of 2^23 at most, one above 2^128 a
// smaller of 1 at least, so a sum is out of range between the two
// multiplications only if the result is.
struct TensorScales {
  float first, second;
};
template <int FMT>
__device__ __forceinline__ TensorScales tensor_scales(const ProductParams& p) {
  const float a = tensor_scale_of(p.a_g), w = tensor_scale_of(p.w_g), both = a * w;
  if constexpr (FMT != ATTN_RES_NVFP4) return {1.f, both};
  const bool held = fabsf(both) >= 0x1p-126f && fabsf(both) < __int_as_float(0x7f800000);
  const bool w_larger = fabsf(a) < fabsf(w);  // (not fmaxf and fminf: a NaN stays one)
  return {held ? 1.f : w_larger ? w : a, held ? both : w_larger ? a : w};
}
// (a branch, as 64 more products a thread took 1-3 % of a large product's time)
template <int N>
__device__ __forceinline__ void scale_first(const TensorScales& s, uint32_t (&r)[N]) {
  if (s.first != 1.f) {
#pragma unroll
    for (int k = 0; k < N; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * s.first);
  }
}

// The limit of a wait for the products of `blocks` blocks of K, each of which
// takes less than 0.5 us: with the longest rows they take seconds themselves.
__device__ __forceinline__ uint64_t products_limit_ns(int blocks) { return kWaitLimitNs + 4000ull * (uint32_t)blocks; }

// ---- few tokens: weight rows on the instruction's M side, K split over a cluster -----------
//
// A CTA makes a part of the sums of 128 output columns (weight rows, the
// instruction's M) for TN tokens (its N): the part of its range of K.  The
// CTAs of a cluster share one tile and split K evenly; their parts meet in
// shared memory (over the stages, which are done with) and every CTA adds up,
// in an order fixed by the tile, a share of the sums, read from its peers.
// (Sent instead -- st.async or bulk copies to the adding CTA -- the parts took
// longer from 32 tokens on: 64 tokens x 7168 x 7168 10.9 us against 8.8.)
// TN < 128 only with a single token tile: a tile's token scales then start at
// the first of their scale tile's columns.
constexpr int kMaxSplit = 6;
constexpr int kItems = 4;  // of the joining, per thread and pass

template <int FMT, int TN>
struct NarrowCfg {
  using F = ProductFmt<FMT>;
  static constexpr uint32_t W_BYTES = 128 * 128;
  static constexpr uint32_t A_BYTES = TN * 128;
  static constexpr uint32_t SF_BYTES = F::ATOMS * 512;
  static constexpr uint32_t STAGE = W_BYTES + A_BYTES + 2 * SF_BYTES;
  // two CTAs an SM, each with as many stages as half of its shared memory
  // and half of TMEM hold
  static constexpr int STAGES = (112 * 1024 - 1024) / STAGE;
  // TMEM columns: the accumulator, then for each stage its scales (so that a
  // stage's scales are replaced only after the products that read them)
  static constexpr int SF_COLS = F::ATOMS * 4;
  static constexpr int COLS_USED = TN + STAGES * 2 * SF_COLS;
  static constexpr int COLS = pow2_at_least(COLS_USED < 32 ? 32 : COLS_USED);
  static_assert(STAGES >= 3 && COLS <= 256, "two CTAs an SM");
  static_assert(STAGES * STAGE >= TN * 128 * 4, "the parts fit over the stages");
  static constexpr uint32_t SMEM = STAGES * STAGE + 1024;
  static constexpr int THREADS = 192;
};

// One output column of four tokens, as far as they exist.
__device__ __forceinline__ void store_quad(const ProductParams& p, int64_t m, int64_t n, float a, float b, float c,
                                           float d, bool failed) {
  if (n >= p.n) return;
  const uint32_t lo = pack_bf16x2(a, b), hi = pack_bf16x2(c, d);
  if (failed) return;
  uint16_t* const o = p.out + m * p.out_row + n;
  if (m < p.m) o[0] = (uint16_t)lo;
  if (m + 1 < p.m) o[p.out_row] = (uint16_t)(lo >> 16);
  if (m + 2 < p.m) o[2 * p.out_row] = (uint16_t)hi;
  if (m + 3 < p.m) o[3 * p.out_row] = (uint16_t)(hi >> 16);
}

template <int FMT, int TN>
__global__ void __launch_bounds__(192, 2)
    attn_res_mx_product_narrow_kernel(const ProductParams p, const __grid_constant__ CUtensorMap map_a,
                                      const __grid_constant__ CUtensorMap map_w) {
  using C = NarrowCfg<FMT, TN>;
  using F = ProductFmt<FMT>;
  constexpr int S = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) unsigned long long bars[2 * S + 1];
  __shared__ uint32_t tmem_slot;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), split = (int)cluster_nctarank();
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t full = smem_addr(bars), empty = full + 8 * S, done = empty + 8 * S;
  const uint32_t w_at = base, a_at = base + S * C::W_BYTES, sf_at = base + S * (C::W_BYTES + C::A_BYTES);
  const int n0 = (int)(blockIdx.x / split) * 128, m0 = (int)blockIdx.y * TN;
  const int all_blocks = (p.row_bytes_used + 127) / 128;
  const int kb0 = (int)((int64_t)all_blocks * rank / split);
  const int blocks = (int)((int64_t)all_blocks * (rank + 1) / split) - kb0;
  bool failed = false;

  const uint8_t* const wsf = p.w_scales + (int64_t)(n0 / 128) * p.group_tiles * 512;
  const uint8_t* const asf = p.a_scales + (int64_t)(m0 / 128) * p.group_tiles * 512;
  const int ahead = blocks < S ? blocks : S;
  auto sf_bytes = [&](int kb) {
    const int64_t left = p.group_tiles - (int64_t)kb * F::ATOMS;
    return (uint32_t)(left < F::ATOMS ? left : F::ATOMS) * 512u;
  };
  auto load_w = [&](int i, int s) {
    const int kb = kb0 + i;
    const uint32_t bar = full + 8 * s, sf = sf_bytes(kb);
    mbar_arrive_expect_tx(bar, C::W_BYTES + C::A_BYTES + 2 * sf);
    tma_load_2d(w_at + s * C::W_BYTES, &map_w, kb * 128, n0, bar);
    bulk_load(sf_at + s * 2 * C::SF_BYTES, wsf + (int64_t)kb * F::ATOMS * 512, sf, bar);
  };
  auto load_a = [&](int i, int s) {
    const int kb = kb0 + i;
    const uint32_t bar = full + 8 * s;
    tma_load_2d(a_at + s * C::A_BYTES, &map_a, kb * 128, m0, bar);
    bulk_load(sf_at + s * 2 * C::SF_BYTES + C::SF_BYTES, asf + (int64_t)kb * F::ATOMS * 512, sf_bytes(kb), bar);
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * S + 1; ++i) mbar_init(full + 8 * i, 1);
    fence_mbar_init();
    // with ATTN_RES_FLAG_PDL the weights do not depend on the preceding kernel:
    // the first stages' are on their way before the wait for it
    if (p.early_weights)
      for (int i = 0; i < ahead; ++i) load_w(i, i);
  }
  grid_dep_wait();
  if (threadIdx.x == 0)
    for (int i = 0; i < ahead; ++i) {
      if (!p.early_weights) load_w(i, i);
      load_a(i, i);
    }
  // (TMEM only now: while the preceding kernel runs it may need it itself)
  if (warp == 1) tmem_alloc<1>(smem_addr(&tmem_slot), C::COLS);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);  // uniform for the compiler
  // (early: read behind the last product, its way from L2 would show)
  const TensorScales scale = FMT == ATTN_RES_NVFP4 ? tensor_scales<FMT>(p) : TensorScales{1.f, 1.f};
  const float one = scale.first, by = scale.second;

  if (warp == 0 && lane == 0) {
    int issued = ahead;
    for (int i = ahead; i < blocks; ++i) {
      const int s = i % S;
      phase_or_flag(empty + 8 * s, (i / S - 1) & 1, failed, p.err, kErrStageTimeout);
      if (failed) break;
      load_w(i, s);
      load_a(i, s);
      issued = i + 1;
    }
    if (failed)  // copies still in flight land before the CTA ends
      for (int i = issued > S ? issued - S : 0; i < issued; ++i) (void)phase_wait(full + 8 * (i % S), (i / S) & 1);
  } else if (warp == 1) {
    constexpr uint32_t idesc = F::idesc(128, TN);
    const bool issuer = elect_one();
    const uint32_t w_lo = desc_lo(w_at), a_lo = desc_lo(a_at), sf_lo = desc_lo(sf_at);
    for (int i = 0; i < blocks; ++i) {
      const int s = i % S;
      phase_or_flag(full + 8 * s, (i / S) & 1, failed, p.err, kErrStageTimeout);
      failed = __any_sync(0xffffffffu, failed);
      if (failed) {
        drain_stages<S>(full, s, i / S);
        break;
      }
      tmem_fence_after();
      if (issuer) {
        const uint32_t sfs = sf_lo + s * (2 * C::SF_BYTES >> 4);
        const uint32_t sf = tmem + TN + s * 2 * C::SF_COLS;
        with_steps(p.row_bytes_used - (kb0 + i) * 128, [&](auto steps) {
          block_scales<FMT, 1, 1, decltype(steps)::value>(sf, sfs, sfs + (C::SF_BYTES >> 4));
          block_steps<FMT, 1, 1, decltype(steps)::value>(tmem, sf, 0, w_lo + s * (C::W_BYTES >> 4), a_lo + s * (C::A_BYTES >> 4),
                                          idesc, i > 0);
        });
        mma_commit<1>(empty + 8 * s);
      }
      __syncwarp();
    }
    if (issuer) mma_commit<1>(done);
    __syncwarp();
  }
  if (warp >= 2) {
    // warp w reads the TMEM lanes 32 (w % 4) .., that is the weight rows n0 + those
    const int row = 32 * (warp % 4) + lane;
    phase_or_flag(done, 0, failed, p.err, kErrStageTimeout, products_limit_ns(blocks));
    failed = __any_sync(0xffffffffu, failed);
    tmem_fence_after();
    grid_dep_launch_dependents();
    constexpr int CH = TN >= 64 ? 64 : 16;  // tokens at a time
    for (int c = 0; c < TN; c += CH) {
      if (m0 + c >= p.m) break;  // no token there
      uint32_t r[CH];
      const uint32_t at = tmem + ((uint32_t)(32 * (warp % 4)) << 16) + c;
      if constexpr (CH == 64) tmem_ld64(at, r);
      else tmem_ld16(at, r);
      tmem_ld_wait(r);
#pragma unroll
      for (int j = 0; j < CH; j += 4) {
        if (split == 1) {
          store_quad(p, m0 + c + j, n0 + row, __uint_as_float(r[j]) * one * by, __uint_as_float(r[j + 1]) * one * by,
                     __uint_as_float(r[j + 2]) * one * by, __uint_as_float(r[j + 3]) * one * by, failed);
        } else {
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(base + (uint32_t)((c + j) * 32 + row) * 16u),
                       "r"(r[j]), "r"(r[j + 1]), "r"(r[j + 2]), "r"(r[j + 3])
                       : "memory");
        }
      }
    }
    tmem_fence_before();
  }
  __syncwarp();
  if (split > 1) {
    cluster_sync();
    // a thread's items are quadruples of tokens of one column; the loads of all
    // parts of kItems of them are in flight together
    const int64_t left = p.m - m0;
    const int items = ((left < TN ? (int)left : TN) + 3) / 4 * 128;
    const int stride = split * C::THREADS;
    for (int i0 = rank * C::THREADS + (int)threadIdx.x; i0 < items; i0 += kItems * stride) {
      float4 part[kItems][kMaxSplit];  // [.][k]: of rank (rank + k) % split, the own one from here
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const int i = i0 + k * stride;
        const uint32_t at = base + (uint32_t)i * 16u;
        if (i >= items || n0 + i % 128 >= p.n) continue;
        asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(part[k][0].x), "=f"(part[k][0].y), "=f"(part[k][0].z), "=f"(part[k][0].w)
                     : "r"(at)
                     : "memory");
#pragma unroll
        for (int r = 1; r < kMaxSplit; ++r)
          if (r < split)
            asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(part[k][r].x), "=f"(part[k][r].y), "=f"(part[k][r].z), "=f"(part[k][r].w)
                         : "r"(map_rank(at, (uint32_t)(rank + r < split ? rank + r : rank + r - split)))
                         : "memory");
      }
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const int i = i0 + k * stride;
        if (i >= items || n0 + i % 128 >= p.n) continue;
        float4 sum = part[k][0];
#pragma unroll
        for (int r = 1; r < kMaxSplit; ++r)
          if (r < split) {
            sum.x += part[k][r].x;
            sum.y += part[k][r].y;
            sum.z += part[k][r].z;
            sum.w += part[k][r].w;
          }
        store_quad(p, m0 + i / 128 * 4, n0 + i % 128, sum.x * one * by, sum.y * one * by, sum.z * one * by,
                   sum.w * one * by, failed);
      }
    }
    // No CTA ends while its part is being read.  Every load's value has been
    // used by then, so the arrival orders nothing (releasing the results'
    // stores with it took some 2000 clocks more).
    __syncwarp();
    cluster_arrive_relaxed();
  }
  __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    tmem_free<1>(tmem, C::COLS);
  }
  if (split > 1) {
    __syncwarp();
    cluster_wait_acquire();
  }
}

// ---- many tokens: CTA pairs ----------------------------------------------------------------
//
// A pair of CTAs (cta_group::2) makes 256 tokens x TN output columns: each
// holds 128 tokens' rows, half of the weight rows (the instruction reads the
// other half from the peer) and the scales of its tokens and of all TN weight
// rows.  Persistent pairs walk the tiles; warp 0 loads, warp 1 of the first
// CTA issues the MMAs of both, the warps from 4 on drain the accumulators
// through registers to global memory.
//
// What bounds a tile is what an SM takes in (measured: 60 bytes a clock of
// the 64 its port has) more than the tensor cores, so wide tiles:
//   HALVES = 2: 384 columns, as two instructions of 192 with an accumulator
//     each.  The first half of the next tile's products waits only for the
//     first accumulator's draining.
//   HALVES = 1: 256 columns, for products that make too few of the wide ones.
//     Two accumulators of 256 columns and the scales do not fit TMEM's 512
//     columns, so those of successive tiles share 128: the first at columns
//     0.., the second at 128..  A tile's shared columns are drained first, and
//     the next tile's products begin as soon as they are.
template <int FMT, int HALVES>
struct WideCfg {
  using F = ProductFmt<FMT>;
  static constexpr int HN = HALVES == 1 ? 256 : 192;  // columns of an instruction
  static constexpr int TM = 256, TN = HN * HALVES;
  static constexpr int QT = TN / 128;  // scale tiles of 128 weight rows
  static constexpr uint32_t A_BYTES = 128 * 128, W_BYTES = TN / 2 * 128, WH_BYTES = HN / 2 * 128;
  static constexpr uint32_t SF_BYTES = F::ATOMS * 512;  // of 128 rows
  static constexpr uint32_t STAGE = A_BYTES + W_BYTES + (1 + QT) * SF_BYTES;
  static constexpr int STAGES = (226 * 1024 - 1024) / STAGE;
  static constexpr uint32_t SMEM = STAGES * STAGE + 1024;
  // TMEM: accumulators, then the scales in a ring of SF_RING blocks
  static constexpr int COLS = 512, SF_AT = 384;
  static constexpr int ACC_STEP = HALVES == 1 ? 128 : 192;  // between the two accumulators
  static constexpr int SF_COLS = (1 + QT) * F::ATOMS * 4;
  static constexpr int SF_RING = (COLS - SF_AT) / SF_COLS < STAGES ? (COLS - SF_AT) / SF_COLS : STAGES;
  static_assert(SF_RING >= 2 && SMEM <= 227 * 1024, "TMEM and shared memory");
  static constexpr int EPI_WARPS = HALVES == 1 ? 8 : 12;  // four for each 64 columns of an accumulator
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
};

struct WideMaps {
  CUtensorMap a, w, a_sf, w_sf;
};

template <int FMT, int HALVES>
__global__ void __launch_bounds__(WideCfg<FMT, HALVES>::THREADS, 1)
    attn_res_mx_product_wide_kernel(const ProductParams p, const TileWalk walk,
                                    const __grid_constant__ WideMaps maps) {
  using C = WideCfg<FMT, HALVES>;
  using F = ProductFmt<FMT>;
  constexpr int S = C::STAGES, R = C::SF_RING;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) unsigned long long bars[2 * S + 2 * HALVES + 1];
  __shared__ uint32_t tmem_slot;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t full = smem_addr(bars), empty = full + 8 * S, acc_full = empty + 8 * S,
                 acc_empty = acc_full + 8 * HALVES, drained = acc_empty + 8 * HALVES;
  const uint32_t a_at = base, w_at = base + S * C::A_BYTES;
  const uint32_t sf_at = base + S * (C::A_BYTES + C::W_BYTES);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * S + HALVES; ++i) mbar_init(full + 8 * i, 1);
    for (int i = 0; i < HALVES; ++i) mbar_init(acc_empty + 8 * i, 2 * C::EPI_WARPS);
    mbar_init(drained, 1);
    fence_mbar_init();
  }
  grid_dep_wait();
  // (TMEM only now: while the preceding kernel runs it may need it itself)
  if (warp == 1) tmem_alloc<2>(smem_addr(&tmem_slot), C::COLS);
  tmem_fence_before();
  __syncwarp();
  cluster_sync();  // both CTAs' barriers and TMEM are there
  tmem_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);  // uniform for the compiler
  const int tiles = walk.m_tiles * walk.n_tiles;
  const int first = blockIdx.x / 2, step = gridDim.x / 2;
  const int blocks = (p.row_bytes_used + 127) / 128;

  if (warp == 0 && lane == 0) {
    bool failed = false;
    int s = 0;
    uint32_t use = 0, issued = 0;
    const int tiles_k = (int)p.group_tiles;
    for (int i = first; i < tiles && !failed; i += step) {
      int mt, nt;
      tile_at(walk, i, mt, nt);
      const int a_row = mt * C::TM + (int)rank * 128, w_row = nt * C::TN + (int)rank * (C::HN / 2);
      for (int kb = 0; kb < blocks; ++kb) {
        if (use > 0) phase_or_flag(empty + 8 * s, (use - 1) & 1, failed, p.err, kErrStageTimeout);
        if (failed) break;
        const uint32_t bar = full + 8 * s, bar0 = map_rank(bar, 0);
        if (rank == 0) mbar_arrive_expect_tx(bar, 2 * C::STAGE);
        const int sf_row = kb * F::ATOMS;
        const uint32_t sf = sf_at + s * (1 + C::QT) * C::SF_BYTES;
        tma_load_2d_pair(a_at + s * C::A_BYTES, &maps.a, kb * 128, a_row, bar0);
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
          tma_load_2d_pair(w_at + s * C::W_BYTES + h * C::WH_BYTES, &maps.w, kb * 128, w_row + h * C::HN, bar0);
        tma_load_2d_pair(sf, &maps.a_sf, 0, a_row / 128 * tiles_k + sf_row, bar0);
#pragma unroll
        for (int h = 0; h < C::QT; ++h)
          tma_load_2d_pair(sf + (1 + h) * C::SF_BYTES, &maps.w_sf, 0, (nt * C::QT + h) * tiles_k + sf_row, bar0);
        ++issued;
        if (++s == S) {
          s = 0;
          ++use;
        }
      }
    }
    if (failed && rank == 0)  // copies still in flight (the peer's too) land before the CTAs end
      for (uint32_t b = issued > S ? issued - S : 0; b < issued; ++b)
        (void)phase_wait(full + 8 * (b % S), (b / S) & 1);
  } else if (warp == 1 && rank == 0) {
    bool failed = false;
    int s = 0, ring = 0, ring_s = 0;  // stage, scale slot, the stage that last used the slot
    uint32_t use = 0, tile = 0, count = 0, ring_use = 0;
    constexpr uint32_t idesc = F::idesc(256, C::HN);
    const bool issuer = elect_one();
    const uint32_t a_lo = desc_lo(a_at), w_lo = desc_lo(w_at), sf_lo = desc_lo(sf_at);
    for (int i = first; i < tiles && !failed; i += step, ++tile) {
      const uint32_t acc = HALVES == 1 ? tmem + (tile & 1) * C::ACC_STEP : tmem;
      for (int kb = 0; kb < blocks; ++kb) {
        phase_or_flag(full + 8 * s, use & 1, failed, p.err, kErrStageTimeout);
        if constexpr (R < S) {  // the products that read this slot's scales are complete
          if (count >= R) {
            phase_or_flag(empty + 8 * ring_s, ring_use & 1, failed, p.err, kErrStageTimeout);
            if (++ring_s == S) {
              ring_s = 0;
              ++ring_use;
            }
          }
          ++count;
        }
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          if (kb == 0 && tile > 0)
            phase_or_flag<true>(acc_empty + 8 * h, (tile - 1) & 1, failed, p.err, kErrExchangeTimeout);
          if (h == 0 || kb == 0) {
            failed = __any_sync(0xffffffffu, failed);
            tmem_fence_after();
          }
          if (issuer && !failed) {
            const uint32_t sfs = sf_lo + s * ((1 + C::QT) * C::SF_BYTES >> 4);
            const uint32_t sf = tmem + C::SF_AT + ring * C::SF_COLS;
            with_steps(p.row_bytes_used - kb * 128, [&](auto steps) {
              if (h == 0) block_scales<FMT, 2, C::QT, decltype(steps)::value>(sf, sfs, sfs + (C::SF_BYTES >> 4));
              block_steps<FMT, 2, C::QT, decltype(steps)::value>(acc + h * C::ACC_STEP, sf, h * (C::HN / 32),
                                                  a_lo + s * (C::A_BYTES >> 4),
                                                  w_lo + (s * C::W_BYTES + h * C::WH_BYTES >> 4), idesc, kb > 0);
            });
            if (kb == blocks - 1) mma_commit<2>(acc_full + 8 * h);
          }
        }
        if (failed) break;
        if (issuer) mma_commit<2>(empty + 8 * s);
        __syncwarp();
        if (++ring == R) ring = 0;
        if (++s == S) {
          s = 0;
          ++use;
        }
      }
    }
    if (failed) {  // what was issued ends before the CTAs do
      if (issuer) mma_commit<2>(drained);
      __syncwarp();
      (void)phase_wait(drained, 0);
      drain_stages<S>(full, s, use);
    }
  } else if (warp >= 4) {
    bool failed = false;
    uint32_t tile = 0;
    const int q = warp % 4, part = (warp - 4) / 4;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
    const TensorScales scale = tensor_scales<FMT>(p);
    const bool wide = p.out_row % 16 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
    for (int i = first; i < tiles && !failed; i += step, ++tile) {
      int mt, nt;
      tile_at(walk, i, mt, nt);
      const int64_t row = (int64_t)mt * C::TM + rank * 128 + 32 * q + lane;
      // HALVES = 2: both accumulators into registers, each released, before the
      // stores (with each accumulator's stores at once the second was released
      // 2500 clocks later: 8192 x 7168 x 7168 mxfp4 114 us instead of 109)
      uint32_t v[2][32];
      int local[2] = {};
      auto store = [&](int h) {
        const int col = nt * C::TN + local[h];
        store_row(p.out + row * p.out_row + col, v[h], (int)p.n - col, wide);
      };
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (HALVES == 2 || h == 0) {
          phase_or_flag(acc_full + 8 * h, tile & 1, failed, p.err, kErrStageTimeout, products_limit_ns(blocks));
          failed = __any_sync(0xffffffffu, failed);
          tmem_fence_after();
        }
        // 64 columns: of accumulator h, or first of the 128 that successive
        // accumulators share (the upper of the first, the lower of the second)
        local[h] = HALVES == 2 ? h * C::HN + 64 * part
                               : ((tile & 1) == (h == 0 ? 0u : 1u) ? 128 : 0) + 64 * part;
        uint32_t r[64];
        tmem_ld64(lanes + (HALVES == 2 ? 0 : (tile & 1) * C::ACC_STEP) + local[h], r);
        tmem_ld_wait(r);
        tmem_fence_before();
        __syncwarp();
        if ((HALVES == 2 || h == 0) && lane == 0) mbar_arrive_remote(map_rank(acc_empty + 8 * h, 0));
        scale_first(scale, r);
        pack64(r, scale.second, v[h]);
        if (HALVES == 1 && !failed && row < p.m) store(h);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (HALVES == 2 && !failed && row < p.m) store(h);
      if (i + step >= tiles) grid_dep_launch_dependents();
    }
  }
  __syncwarp();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tmem_fence_after();
    tmem_free<2>(tmem, C::COLS);
  }
}

}  // namespace attn_res_dev
