// attn_res_f8_product.cuh -- products of two matrices in 8 bits with scales for
// blocks of 128, and the gated block's two products, on the tensor cores
// (tcgen05.mma kind::f8f6f4).
//
// The scales are fp32 and change every 128 columns of K, so the sums of a
// block of K leave the tensor cores, are scaled and added up in registers:
// sum_b sa[m, b] sw[n, b] (sum over block b of codes a x codes w), a block's
// sum and the sums over blocks in fp32.
#pragma once

#include "attn_res_f8.cuh"
#include "attn_res_tcgen05.cuh"

namespace attn_res_dev {

// ---- instructions -------------------------------------------------------------------------

template <int G>
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (G == 1)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
  else
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}
// e4m3 x e4m3 into fp32, both operands K-major.
__host__ __device__ constexpr uint32_t f8_idesc(uint32_t m, uint32_t n) {
  return 1u << 4 | (n >> 3) << 17 | (m >> 4) << 24;
}
// One block of K: four instructions of 32 columns.
template <int G>
__device__ __forceinline__ void f8_block(uint32_t acc, uint32_t p_lo, uint32_t q_lo, uint32_t idesc) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    mma_f8<G>(acc, desc_of(p_lo + 2 * j, kOperandHi), desc_of(q_lo + 2 * j, kOperandHi), idesc, j > 0);
}

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// ---- scales -------------------------------------------------------------------------------

// The product of two scales where fp32 does not hold it (scales of 1e-30 and
// 1e-20, say, under which a sum may well be a number, or of 1e25 both, and a
// sum of 0): mantissas and exponents apart, applied to x as three factors, none
// of which takes it out of range unless the result is (|x| is 0 or between
// 2^-18 and 2^26).
struct FarScale {
  float mantissa, first, second;
  __device__ __forceinline__ FarScale(float a, float w) {
    int ea, ew;
    mantissa = frexpf(a, &ea) * frexpf(w, &ew);
    const bool number = fabsf(mantissa) < __int_as_float(0x7f800000);
    const int e = number ? ea + ew : 0;  // (an infinity's or a NaN's exponent says nothing)
    const int e1 = min(max(e, -100), 100), e2 = min(max(e - e1, -149), 127);
    first = ldexpf(1.f, e1);
    second = ldexpf(1.f, e2);
  }
  __device__ __forceinline__ float of(float x) const { return x * mantissa * first * second; }
};
__device__ __forceinline__ bool scale_held(float f) {
  return fabsf(f) >= 0x1p-126f && fabsf(f) < __int_as_float(0x7f800000);
}

// ---- parameters ---------------------------------------------------------------------------

constexpr int kF8OutBf16 = 0, kF8OutF32 = 1, kF8GatedCodes = 2, kF8GatedBf16 = 3;

struct F8Scales {
  const float* at;
  int64_t row;  // between blocks of columns (row scales) or rows of blocks
};

struct F8ProductParams {
  // Products of two terms at most: out = sum over terms of a[t] w[t]^T.  The
  // gated block has one term with w[0] the gate and w[1] the up-projection.
  F8Scales a[2], w[2];
  int blocks[2];  // blocks of K of each term
  int64_t m, n;   // rows of a and of w
  void* out;      // bf16 or fp32 rows
  int64_t out_row;
  bool add;       // fp32: to what is there
  F8View h, g, u;  // gated: the results in codes; data null: not wanted
  unsigned* err;
};

struct F8ProductMaps {
  CUtensorMap a[2], w[2], w_sf[2];
};

// ---- many tokens: CTA pairs ----------------------------------------------------------------
//
// A pair of CTAs (cta_group::2) makes 256 tokens x 256 columns (of the gated
// block: 128 of the gate and the same 128 of the up-projection); each holds 128
// tokens' rows and half of the weight rows.  Persistent pairs walk the tiles;
// warp 0 loads, warp 1 of the first CTA issues the MMAs of both, warp 2 loads
// column scales, and eight warps scale and add: each block of K gets an
// accumulator of 256 TMEM columns of its own, two of which take turns, so that
// one is read while the tensor cores fill the other.  A thread holds 128 sums:
// 64 columns of the tile's first half and the same 64 of its second.
struct F8WideCfg {
  static constexpr int TM = 256, TN = 256;
  static constexpr uint32_t A_BYTES = 128 * 128, W_BYTES = 128 * 128, STAGE = A_BYTES + W_BYTES;
  static constexpr int STAGES = 6;
  static constexpr int SF_RING = 8;  // blocks of column scales
  static constexpr uint32_t SF_BYTES = TN * 4;
  static constexpr uint32_t SMEM = STAGES * STAGE + SF_RING * SF_BYTES + 1024;
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  static constexpr int COLS = 512, ACC_STEP = 256;
  // registers: 168 a thread at launch, 64512 in all, of which the first
  // warpgroup gives 96 a thread to the other two
  static constexpr int REGS_FEW = 72, REGS_MANY = 216;
  static_assert(128 * REGS_FEW + 256 * REGS_MANY <= 168 * THREADS, "the split of the registers");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// 64 fp32 columns of a lane's row, `left` of which exist; `whole`: every row
// starts on a 32-byte boundary.
__device__ __forceinline__ void store_f32_64(float* o, const f32x2* v, int left, bool whole, bool add) {
  if (whole && left >= 64) {
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      float e[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        e[2 * j] = f2_lo(v[k + j]);
        e[2 * j + 1] = f2_hi(v[k + j]);
      }
      if (add) {
        float s[8];
        asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(s[0]), "=f"(s[1]), "=f"(s[2]), "=f"(s[3]), "=f"(s[4]), "=f"(s[5]), "=f"(s[6]), "=f"(s[7])
                     : "l"(o + 2 * k)
                     : "memory");
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] += s[j];
      }
      asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(o + 2 * k), "f"(e[0]), "f"(e[1]),
                   "f"(e[2]), "f"(e[3]), "f"(e[4]), "f"(e[5]), "f"(e[6]), "f"(e[7])
                   : "memory");
    }
  } else {
#pragma unroll
    for (int k = 0; k < 64; ++k)
      if (k < left) o[k] = (k % 2 ? f2_hi(v[k / 2]) : f2_lo(v[k / 2])) + (add ? o[k] : 0.f);
  }
}

// 64 values of a lane's row in codes, over the scale of all 128 columns of the
// row, whose other half another warp holds: `other` exchanges the bits of the
// amax.  Columns behind the last hold 0 (or, with their whole row, NaN).
template <class Other>
__device__ __forceinline__ void store_f8_64(const F8View& q, int64_t row, int64_t col, bool stores, const f32x2* v,
                                            Other other) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 32; ++k) m = max(m, max(magnitude(f2_lo(v[k])), magnitude(f2_hi(v[k]))));
  const F8Scale s = f8_scale(max(m, other(m)));
  if (!stores || row >= q.rows) return;
  if (col % kF8Block == 0) q.scales[col / kF8Block * q.scales_row + row] = s.by;
  uint8_t* const o = q.data + row * q.row_bytes + col;
  const int64_t left = q.cols - col;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = f8_codes(v[8 * k + 2 * j], v[8 * k + 2 * j + 1], s);
    if (16 * k + 16 <= left) {
      *reinterpret_cast<uint4*>(o + 16 * k) = make_uint4(c[0], c[1], c[2], c[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (16 * k + e < left) o[16 * k + e] = (uint8_t)(c[e / 4] >> (8 * (e % 4)));
    }
  }
}

template <int OUT, int ACT, bool ROWS_W>
__global__ void __launch_bounds__(F8WideCfg::THREADS, 1)
    attn_res_f8_wide_kernel(const __grid_constant__ F8ProductParams p, const TileWalk walk,
                            const __grid_constant__ F8ProductMaps maps) {
  using C = F8WideCfg;
  constexpr int S = C::STAGES, R = C::SF_RING;
  constexpr bool GATED = OUT == kF8GatedCodes || OUT == kF8GatedBf16;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) unsigned long long bars[2 * S + 5 + 2 * R];
  __shared__ uint32_t tmem_slot;
  __shared__ uint32_t xch[2][2][128];  // [turn][half][row]: amaxes that two warps share
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t full = smem_addr(bars), empty = full + 8 * S, acc_full = empty + 8 * S, acc_empty = acc_full + 16,
                 drained = acc_empty + 16, sf_full = drained + 8, sf_empty = sf_full + 8 * R;
  const uint32_t a_at = base, w_at = base + S * C::A_BYTES, sf_at = base + S * C::STAGE;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * S + 2; ++i) mbar_init(full + 8 * i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(acc_empty + 8 * i, 2 * C::EPI_WARPS);
    mbar_init(drained, 1);
    for (int i = 0; i < R; ++i) {
      mbar_init(sf_full + 8 * i, 1);
      mbar_init(sf_empty + 8 * i, C::EPI_WARPS);
    }
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
  const int blocks0 = p.blocks[0], blocks = blocks0 + p.blocks[1];

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_FEW));
    if (warp == 0 && lane == 0) {
      bool failed = false;
      int s = 0;
      uint32_t use = 0, issued = 0;
      for (int i = first; i < tiles && !failed; i += step) {
        int mt, nt;
        tile_at(walk, i, mt, nt);
        const int a_row = mt * C::TM + (int)rank * 128;
        const int w_row = GATED ? nt * 128 : nt * C::TN + (int)rank * 128;
        for (int k = 0; k < blocks; ++k) {
          if (use > 0) phase_or_flag(empty + 8 * s, (use - 1) & 1, failed, p.err, kErrStageTimeout);
          if (failed) break;
          const uint32_t bar = full + 8 * s, bar0 = map_rank(bar, 0);
          const int t = k < blocks0 ? 0 : 1, kb = k < blocks0 ? k : k - blocks0;
          if (rank == 0) mbar_arrive_expect_tx(bar, 2 * C::STAGE);
          tma_load_2d_pair(a_at + s * C::A_BYTES, &maps.a[t], kb * 128, a_row, bar0);
          tma_load_2d_pair(w_at + s * C::W_BYTES, &maps.w[GATED ? (int)rank : t], kb * 128, w_row, bar0);
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
      int s = 0;
      uint32_t use = 0, it = 0;
      constexpr uint32_t idesc = f8_idesc(C::TM, C::TN);
      const bool issuer = elect_one();
      const uint32_t a_lo = desc_lo(a_at), w_lo = desc_lo(w_at);
      for (int i = first; i < tiles && !failed; i += step) {
        for (int k = 0; k < blocks; ++k, ++it) {
          const uint32_t b = it & 1;
          phase_or_flag(full + 8 * s, use & 1, failed, p.err, kErrStageTimeout);
          if (it >= 2) phase_or_flag<true>(acc_empty + 8 * b, ((it >> 1) - 1) & 1, failed, p.err, kErrExchangeTimeout);
          failed = __any_sync(0xffffffffu, failed);
          if (failed) break;
          tmem_fence_after();
          if (issuer) {
            f8_block<2>(tmem + b * C::ACC_STEP, a_lo + s * (C::A_BYTES >> 4), w_lo + s * (C::W_BYTES >> 4), idesc);
            mma_commit<2>(empty + 8 * s);
            mma_commit<2>(acc_full + 8 * b);
          }
          __syncwarp();
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
    } else if (ROWS_W && warp == 2 && lane == 0) {
      bool failed = false;
      uint32_t it = 0;
      for (int i = first; i < tiles && !failed; i += step) {
        int mt, nt;
        tile_at(walk, i, mt, nt);
        for (int k = 0; k < blocks; ++k, ++it) {
          const uint32_t r = it % R;
          if (it >= R) phase_or_flag(sf_empty + 8 * r, (it / R - 1) & 1, failed, p.err, kErrStageTimeout);
          if (failed) break;
          const int t = k < blocks0 ? 0 : 1, kb = k < blocks0 ? k : k - blocks0;
          mbar_arrive_expect_tx(sf_full + 8 * r, C::SF_BYTES);
          tma_load_2d(sf_at + r * C::SF_BYTES, &maps.w_sf[t], nt * C::TN, kb, sf_full + 8 * r);
        }
      }
      if (failed)
        for (uint32_t b = it > R ? it - R : 0; b < it; ++b) (void)phase_wait(sf_full + 8 * (b % R), (b / R) & 1);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_MANY));
    bool failed = false;
    const int q = warp % 4, part = (warp - 4) / 4;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + 64 * part;
    const uint32_t release = map_rank(acc_empty, 0);
    uint32_t it = 0, turn = 0;
    // (a warp whose wait has given up goes on through the tiles, without waits
    // or stores: another warp meets it at the exchanges)
    for (int i = first; i < tiles; i += step) {
      int mt, nt;
      tile_at(walk, i, mt, nt);
      const int64_t row = (int64_t)mt * C::TM + rank * 128 + 32 * q + lane;
      // the scales of this lane's row (1 past the last) and of the tile's
      // halves, for block k of K
      auto row_scale = [&](int k) {
        const bool one = k < blocks0;
        const F8Scales& s = p.a[one ? 0 : 1];
        return row < p.m && k < blocks ? s.at[(int64_t)(one ? k : k - blocks0) * s.row + row] : 1.f;
      };
      auto block_scale = [&](int k, int half) {
        const bool one = k < blocks0;
        const F8Scales& s = p.w[GATED ? half : one ? 0 : 1];
        const int64_t at = GATED ? nt : 2 * (int64_t)nt + half;
        return at * 128 < p.n && k < blocks ? s.at[at * s.row + (one ? k : k - blocks0)] : 1.f;
      };
      f32x2 sum[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) sum[j] = f2_make(0.f, 0.f);
      float ahead[4], sw[2], sw_ahead[2] = {1.f, 1.f};
#pragma unroll
      for (int j = 0; j < 4; ++j) ahead[j] = row_scale(j);
      if (!ROWS_W)
#pragma unroll
        for (int h = 0; h < 2; ++h) sw_ahead[h] = block_scale(lane, h);
      for (int k4 = 0; k4 < blocks && !failed; k4 += 4) {
        float sa[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sa[j] = ahead[j];
          ahead[j] = row_scale(k4 + 4 + j);
        }
        if (!ROWS_W && k4 % 32 == 0)  // lane l holds those of block k4 + l
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            sw[h] = sw_ahead[h];
            sw_ahead[h] = block_scale(k4 + 32 + lane, h);
          }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = k4 + j;
          if (k >= blocks) break;
          const uint32_t b = it & 1, r = it % R;
          if (ROWS_W) phase_or_flag(sf_full + 8 * r, (it / R) & 1, failed, p.err, kErrStageTimeout);
          phase_or_flag(acc_full + 8 * b, (it >> 1) & 1, failed, p.err, kErrStageTimeout);
          failed = __any_sync(0xffffffffu, failed);
          tmem_fence_after();
          float f[2] = {1.f, 1.f};
          float w_of[2] = {1.f, 1.f};
          bool far = false;
          if constexpr (!ROWS_W) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              w_of[h] = __shfl_sync(0xffffffffu, sw[h], k & 31);
              f[h] = sa[j] * w_of[h];
              far |= !scale_held(f[h]);
            }
          } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              float s;
              const uint32_t at = sf_at + r * C::SF_BYTES + (64 * part + (h / 2) * 128 + (h % 2) * 32 + lane) * 4;
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s) : "r"(at) : "memory");
              // (0: past the last column)
              far |= !(fabsf(s) >= 0x1p-100f && fabsf(s) <= 0x1p100f) && s != 0.f;
            }
          }
          far = __any_sync(0xffffffffu, far);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int h = c / 2;
            uint32_t v[32];
            tmem_ld32(lanes + b * C::ACC_STEP + 128 * h + 32 * (c % 2), v);
            tmem_ld_wait(v);
            if (c == 3) {
              tmem_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_remote(release + 8 * b);
            }
            const uint32_t sf = sf_at + r * C::SF_BYTES + (64 * part + 128 * h + 32 * (c % 2)) * 4;
            if (!far) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const f32x2 x = f2_make(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                if constexpr (!ROWS_W) {
                  sum[16 * c + e] = f2_fma(x, f2_make(f[h], f[h]), sum[16 * c + e]);
                } else {
                  f32x2 s;
                  asm volatile("ld.shared.b64 %0, [%1];" : "=l"(s) : "r"(sf + 8 * e) : "memory");
                  sum[16 * c + e] = f2_fma(f2_mul(x, s), f2_make(sa[j], sa[j]), sum[16 * c + e]);
                }
              }
            } else {
              FarScale fs(sa[j], w_of[h]);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float y[2];
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                  if constexpr (ROWS_W) {
                    float s;
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s) : "r"(sf + 8 * e + 4 * o) : "memory");
                    fs = FarScale(sa[j], s);
                  }
                  y[o] = fs.of(__uint_as_float(v[2 * e + o]));
                }
                sum[16 * c + e] = f2_make(f2_lo(sum[16 * c + e]) + y[0], f2_hi(sum[16 * c + e]) + y[1]);
              }
            }
          }
          if (ROWS_W) {
            __syncwarp();
            if (lane == 0) mbar_arrive(sf_empty + 8 * r);
          }
          ++it;
        }
      }
      if (i + step >= tiles) grid_dep_launch_dependents();
      if constexpr (OUT == kF8OutBf16 || OUT == kF8OutF32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t col = (int64_t)nt * C::TN + 128 * h + 64 * part;
          if (failed || row >= p.m || col >= p.n) continue;
          const int left = (int)(p.n - col < 64 ? p.n - col : 64);
          if constexpr (OUT == kF8OutBf16) {
            const bool wide = p.out_row % 16 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
            uint32_t v[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = pack_bf16x2(f2_lo(sum[32 * h + e]), f2_hi(sum[32 * h + e]));
            store_row64(static_cast<uint16_t*>(p.out) + row * p.out_row + col, v, left, wide);
          } else {
            const bool whole = p.out_row % 8 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
            store_f32_64(static_cast<float*>(p.out) + row * p.out_row + col, sum + 32 * h, left, whole, p.add);
          }
        }
      } else {
        const int64_t col = (int64_t)nt * 128 + 64 * part;
        // the other half's amax of the same row
        auto other = [&](uint32_t m) {
          uint32_t(&x)[2][128] = xch[turn++ & 1];
          x[part][32 * q + lane] = m;
          asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
          return x[1 - part][32 * q + lane];
        };
        const bool stores = !failed && col < p.n;
        if (p.g.data) store_f8_64(p.g, row, col, stores, sum, other);
        if (p.u.data) store_f8_64(p.u, row, col, stores, sum + 32, other);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float lo = f8_act<ACT>(f2_lo(sum[e])), hi = f8_act<ACT>(f2_hi(sum[e]));
          sum[e] = f2_mul(f2_make(lo, hi), sum[32 + e]);
        }
        if constexpr (OUT == kF8GatedCodes) {
          store_f8_64(p.h, row, col, stores, sum, other);
        } else if (stores && row < p.m) {
          const bool wide = p.out_row % 16 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
          uint32_t v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = pack_bf16x2(f2_lo(sum[e]), f2_hi(sum[e]));
          store_row64(static_cast<uint16_t*>(p.out) + row * p.out_row + col, v,
                      (int)(p.n - col < 64 ? p.n - col : 64), wide);
        }
      }
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
