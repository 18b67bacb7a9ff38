// attn_res_f8_product.cuh -- products of two matrices in 8 bits with scales for
// blocks of 128, and the gated block's two products, on the tensor cores
// (tcgen05.mma kind::f8f6f4).
//
// The scales are fp32 and change every 128 columns of K, so the sums of a
// block of K leave the tensor cores, are scaled and added up in registers:
// sum_b sa[m, b] sw[n, b] (sum over block b of codes a x codes w), a block's
// sum and the sums over blocks in fp32.
#pragma once

#include <type_traits>

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

__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[16]) { tmem_ld16(addr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[32]) {
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

// ---- parameters ---------------------------------------------------------------------------

constexpr int kF8OutBf16 = 0, kF8OutF32 = 1, kF8GatedCodes = 2, kF8GatedBf16 = 3;

// Four neighbours' scales from `at` on (a multiple of 4; 16-byte aligned), 1 past
// the last.
__device__ __forceinline__ void ld_scales4(const float* s, int64_t at, int64_t n, float* v) {
  if (at + 4 <= n) {
    const float4 x = *reinterpret_cast<const float4*>(s + at);
    v[0] = x.x;
    v[1] = x.y;
    v[2] = x.z;
    v[3] = x.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = at + k < n ? s[at + k] : 1.f;
  }
}
__device__ __forceinline__ void st_shared4(uint32_t at, float a, float b, float c, float d) {
  asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(at), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
__device__ __forceinline__ float ld_shared(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void ld_shared_pairs(uint32_t at, f32x2 (&v)[2]) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[0]), "=l"(v[1]) : "r"(at) : "memory");
}

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
  CUtensorMap a[2], w[2];
};

// ---- many tokens: CTA pairs ----------------------------------------------------------------
//
// A pair of CTAs (cta_group::2) makes 256 tokens x 256 columns (of the gated
// block: 128 of the gate and the same 128 of the up-projection); each holds 128
// tokens' rows and half of the weight rows.  Persistent pairs walk the tiles;
// warp 0 loads, warp 1 of the first CTA issues the MMAs of both, warps 2 and 3
// make the scales in turn, and eight warps scale and add.
//
// Each block of K gets an accumulator of 256 columns of its own, read while the
// tensor cores fill the other one.  A thread holds 128 sums: of 128 neighbouring
// columns (part 0 or 1 of the tile's two blocks of columns) or, gated, of 64 of
// the gate and the same 64 of the up-projection.
//
// The eight warps' way through a block bounds this, not the tensor cores: a block
// takes some 970 clocks (471 ns), the tensor cores 515 of them (with the loads from
// TMEM and the additions taken out, in a copy, 8192 x 7168 x 4096 took 142 us, with
// both 217, now 192).  By itself a warp takes about 80 clocks for a look at a
// barrier, 40 for an arrival, 60 for the loads of 64 columns and 70 for their
// additions, but two warps share a scheduler: with clocks read on the way (in a
// copy, which that slowed to 1280 clocks a block) a block's additions took 480, its
// loads' waits 120, the release 130, barriers and scales 420 and the rest 120, one
// after the other.  Code that is longer is fetched more slowly (two blocks
// unrolled: 222 us).  So a block has one wait and one
// arrival, scales come for four blocks at a time from two warps of their own, the
// next loads are under way while columns are added, and the next block's barrier
// is looked at meanwhile.  Tried and not kept: accumulators of 128 columns, four
// in turn (244 us); sixteen warps of 64 columns (214); 16 columns at a time (304).
struct F8WideCfg {
  static constexpr int TM = 256, TN = 256;
  static constexpr uint32_t A_BYTES = 128 * 128, W_BYTES = 128 * 128, STAGE = A_BYTES + W_BYTES;
  static constexpr int STAGES = 6;
  // Scales, a ring of groups of four blocks of K, each made by a warp of its own:
  // for each block the products of the rows' scales and those of the tile's two
  // blocks of columns (128 each) or, w with row scales, the rows' scales and
  // those of 256 columns.
  static constexpr int GROUP = 4, SF_RING = 2;
  static constexpr uint32_t SF_BLOCK = (128 + TN) * 4, SF_BYTES = GROUP * SF_BLOCK;
  static constexpr uint32_t SMEM = STAGES * STAGE + SF_RING * SF_BYTES + 1024;
  static constexpr int PARTS = 2;        // warps that share a row
  static constexpr int CW = TN / PARTS;  // a thread's columns
  static constexpr int CH = CW / 4;      // of them at a time
  static constexpr int EPI_WARPS = 4 * PARTS;
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  static constexpr int ACCS = 2, ACC_COLS = 256, COLS = ACCS * ACC_COLS;
  // registers: 168 a thread at launch, 64512 in all, of which the first
  // warpgroup gives 112 a thread to the other two
  static constexpr int REGS_FEW = 56, REGS_MANY = 224;
  static_assert(128 * REGS_FEW + 32 * EPI_WARPS * REGS_MANY <= 168 * THREADS, "the split of the registers");
  static_assert(SMEM <= 227 * 1024 && SF_RING == 2, "shared memory; a slot of the ring for each of two warps");
};

// 64 bf16 columns of a lane's row, `left` of which exist; `whole`: every row
// starts on a 32-byte boundary.
__device__ __forceinline__ void store_bf16(uint16_t* o, const f32x2* x, int left, bool whole) {
  uint32_t v[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) v[e] = pack_bf16x2(f2_lo(x[e]), f2_hi(x[e]));
  store_row(o, v, left, whole);
}
// N fp32 columns; `add`: to what is there.
template <int N>
__device__ __forceinline__ void store_f32(float* o, const f32x2* v, int left, bool whole, bool add) {
  if (whole && left >= N) {
#pragma unroll
    for (int k = 0; k < N / 2; k += 4) {
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
    for (int k = 0; k < N; ++k)
      if (k < left) o[k] = (k % 2 ? f2_hi(v[k / 2]) : f2_lo(v[k / 2])) + (add ? o[k] : 0.f);
  }
}

// N values of a lane's row in codes, over the scale of all 128 columns of the
// row, whose other parts other warps hold: `other` gives the bits of the amax of
// them all.  Columns behind the last hold 0 (or, with their whole row, NaN).
template <int N, class Other>
__device__ __forceinline__ void store_f8(const F8View& q, int64_t row, int64_t col, bool stores, const f32x2* v,
                                         Other other) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < N / 2; ++k) m = amax3(m, v[k]);
  const F8Scale s = f8_scale(other(__float_as_uint(m)));
  if (!stores || row >= q.rows) return;
  if (col % kF8Block == 0) q.scales[col / kF8Block * q.scales_row + row] = s.by;
  uint8_t* const o = q.data + row * q.row_bytes + col;
  const int64_t left = q.cols - col;
#pragma unroll
  for (int k = 0; k < N / 16; ++k) {
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
  constexpr int S = C::STAGES, R = C::SF_RING, A = C::ACCS;
  constexpr bool GATED = OUT == kF8GatedCodes || OUT == kF8GatedBf16;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) unsigned long long bars[2 * S + 2 * A + 1 + 2 * R];
  __shared__ uint32_t tmem_slot;
  __shared__ uint32_t xch[2][C::PARTS][128];  // [turn][part][row]: amaxes of the warps that share a row
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t full = smem_addr(bars), empty = full + 8 * S, acc_full = empty + 8 * S, acc_empty = acc_full + 8 * A,
                 drained = acc_empty + 8 * A, sf_full = drained + 8, sf_empty = sf_full + 8 * R;
  const uint32_t a_at = base, w_at = base + S * C::A_BYTES, sf_at = base + S * C::STAGE;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * S + A; ++i) mbar_init(full + 8 * i, 1);
    for (int i = 0; i < A; ++i) mbar_init(acc_empty + 8 * i, 2 * C::EPI_WARPS);
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
      constexpr uint32_t idesc = f8_idesc(C::TM, C::ACC_COLS);
      const bool issuer = elect_one();
      const uint32_t a_lo = desc_lo(a_at), w_lo = desc_lo(w_at);
      for (int i = first; i < tiles && !failed; i += step) {
        for (int k = 0; k < blocks; ++k, ++it) {
          const uint32_t acc = it & 1;
          phase_or_flag(full + 8 * s, use & 1, failed, p.err, kErrStageTimeout);
          if (it >= 2) phase_or_flag<true>(acc_empty + 8 * acc, ((it >> 1) - 1) & 1, failed, p.err, kErrExchangeTimeout);
          failed = __any_sync(0xffffffffu, failed);
          if (failed) break;
          tmem_fence_after();
          if (issuer) {
            f8_block<2>(tmem + acc * C::ACC_COLS, a_lo + s * (C::A_BYTES >> 4), w_lo + s * (C::W_BYTES >> 4), idesc);
            mma_commit<2>(acc_full + 8 * acc);
            mma_commit<2>(empty + 8 * s);
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
    } else if (warp >= 2) {
      bool failed = false;
      uint32_t group = 0;
      const uint32_t r = warp - 2, slot = sf_at + r * C::SF_BYTES + 16 * lane;
      for (int i = first; i < tiles && !failed; i += step) {
        int mt, nt;
        tile_at(walk, i, mt, nt);
        const int64_t row = (int64_t)mt * C::TM + rank * 128 + 4 * lane, col = (int64_t)nt * C::TN + 4 * lane;
        for (int k4 = 0; k4 < blocks; k4 += C::GROUP, ++group) {
          if (group % R != r) continue;
          if (group >= R) phase_or_flag(sf_empty + 8 * r, (group / R - 1) & 1, failed, p.err, kErrStageTimeout);
          failed = __any_sync(0xffffffffu, failed);
          if (failed) break;
#pragma unroll 1
          for (int j2 = 0; j2 < C::GROUP && k4 + j2 < blocks; j2 += 2) {  // the loads of two blocks together
            float a[2][4], w[2][ROWS_W ? 8 : 2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int k = k4 + j2 + j;
              const bool one = k < blocks0, in = k < blocks;
              const int64_t kb = one ? k : k - blocks0;
              const F8Scales& sa = p.a[one ? 0 : 1];
              const F8Scales& sw = p.w[one ? 0 : 1];
              ld_scales4(sa.at + kb * sa.row, row, in ? p.m : 0, a[j]);
              if constexpr (ROWS_W) {
                ld_scales4(sw.at + kb * sw.row, col, in ? p.n : 0, &w[j][0]);
                ld_scales4(sw.at + kb * sw.row, col + 128, in ? p.n : 0, &w[j][4]);
              } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const F8Scales& sh = GATED ? p.w[h] : sw;
                  const int64_t at = GATED ? nt : 2 * (int64_t)nt + h;
                  w[j][h] = in && at * 128 < p.n ? sh.at[at * sh.row + kb] : 1.f;
                }
              }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t at = slot + (j2 + j) * C::SF_BLOCK;
              if constexpr (ROWS_W) {
                st_shared4(at, a[j][0], a[j][1], a[j][2], a[j][3]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  st_shared4(at + 512 + 512 * h, w[j][4 * h], w[j][4 * h + 1], w[j][4 * h + 2], w[j][4 * h + 3]);
              } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  st_shared4(at + 512 * h, a[j][0] * w[j][h], a[j][1] * w[j][h], a[j][2] * w[j][h], a[j][3] * w[j][h]);
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(sf_full + 8 * r);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_MANY));
    bool failed = false;
    const int q = warp % 4, part = (warp - 4) / 4;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + (GATED ? C::CW / 2 : C::CW) * part;
    const uint32_t release = map_rank(acc_empty, 0);
    // whole sectors: every row starts on a 32-byte boundary
    const bool wide = p.out_row % (OUT == kF8OutF32 ? 8 : 16) == 0 && (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
    uint32_t it = 0, group = 0, turn = 0;
    // (a warp whose wait has given up goes on through the tiles, without waits
    // or stores: another warp meets it at the exchanges)
    for (int i = first; i < tiles; i += step) {
      int mt, nt;
      tile_at(walk, i, mt, nt);
      const int64_t row = (int64_t)mt * C::TM + rank * 128 + 32 * q + lane;
      f32x2 sum[C::CW / 2];
#pragma unroll
      for (int e = 0; e < C::CW / 2; ++e) sum[e] = f2_make(0.f, 0.f);
      // A wait is one look in the common case, and nothing else lies on the way.
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (phase_done(bar, parity) || failed) return;
        if (!phase_wait(bar, parity)) {
          failed = true;
          atomicOr(p.err, kErrStageTimeout);
        }
      };
      // this row's factors of a block (gated: gate's, and behind them up's)
      const uint32_t mine = sf_at + 4 * (32 * q + lane) + (ROWS_W || GATED ? 0 : 512 * (C::CW * part / 128));
      uint32_t v[2][C::CH];
      float f[2], f_next[2];
      auto load = [&](uint32_t block, int piece) {
        tmem_ld(lanes + (block & 1) * C::ACC_COLS + (GATED ? 128 * (piece / 2) + C::CH * (piece % 2) : C::CH * piece),
                v[piece % 2]);
      };
      auto loaded = [&]() {
        tmem_ld_wait(v[0]);
        tmem_ld_wait(v[1]);
      };
      auto factors = [&](uint32_t in_group) {
        if (in_group == 0) wait(sf_full + 8 * (group & 1), (group >> 1) & 1);
        const uint32_t at = mine + (group & 1) * C::SF_BYTES + in_group * C::SF_BLOCK;
        f_next[0] = ld_shared(at);
        f_next[1] = GATED ? ld_shared(at + 512) : f_next[0];
      };
      if (blocks > 0) {
        factors(0);
        wait(acc_full + 8 * (it & 1), (it >> 1) & 1);
        __syncwarp();
        tmem_fence_after();
        load(it, 0);
        load(it, 1);
      }
#pragma unroll 1
      for (int k = 0; k < blocks; ++k) {
        const uint32_t in_group = k % C::GROUP;
        const bool last = k == blocks - 1, leaves = in_group == C::GROUP - 1 || last;
        const uint32_t columns = sf_at + (group & 1) * C::SF_BYTES + in_group * C::SF_BLOCK + 512 + 4 * C::CW * part;
        f[0] = f_next[0];
        f[1] = f_next[1];
        auto add = [&](int piece) {
          const f32x2 by = f2_make(f[piece / 2], f[piece / 2]);
#pragma unroll
          for (int e = 0; e < C::CH / 2; e += 2) {
            f32x2 s[2] = {};
            if constexpr (ROWS_W) ld_shared_pairs(columns + 4 * C::CH * piece + 8 * e, s);
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const uint32_t* const x = &v[piece % 2][2 * (e + o)];
              const f32x2 y = f2_make(__uint_as_float(x[0]), __uint_as_float(x[1]));
              f32x2& to = sum[C::CH / 2 * piece + e + o];
              to = f2_fma(y, ROWS_W ? f2_mul(s[o], by) : by, to);
            }
          }
        };
        loaded();
        add(0);
        load(it, 2);
        add(1);
        load(it, 3);
        loaded();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_remote(release + 8 * (it & 1));
          if (!ROWS_W && leaves) mbar_arrive(sf_empty + 8 * (group & 1));
        }
        ++it;
        if (!ROWS_W) group += leaves;
        // the next block's look at its barrier and its first loads lie among
        // the additions (with the columns' own scales the look comes when it is
        // needed, or registers run out: 4096 x 7168 x 8190 320 us, else 330)
        const uint32_t next = acc_full + 8 * (it & 1);
        [[maybe_unused]] bool there = true;
        if (!ROWS_W && !last) {
          factors((k + 1) % C::GROUP);
          there = phase_done(next, (it >> 1) & 1);
        }
        add(2);
        if (!last) {
          if (ROWS_W || !there) wait(next, (it >> 1) & 1);
          __syncwarp();
          tmem_fence_after();
          load(it, 0);
        }
        add(3);
        if (!last) load(it, 1);
        if constexpr (ROWS_W) {
          __syncwarp();
          if (lane == 0 && leaves) mbar_arrive(sf_empty + 8 * (group & 1));
          group += leaves;
          if (!last) factors((k + 1) % C::GROUP);
        }
      }
      failed = __any_sync(0xffffffffu, failed);
      if (i + step >= tiles) grid_dep_launch_dependents();
      if constexpr (!GATED) {
#pragma unroll
        for (int h = 0; h < C::CW / 64; ++h) {
          const int64_t col = (int64_t)nt * C::TN + C::CW * part + 64 * h;
          if (failed || row >= p.m || col >= p.n) continue;
          const int left = (int)(p.n - col < 64 ? p.n - col : 64);
          if constexpr (OUT == kF8OutBf16)
            store_bf16(static_cast<uint16_t*>(p.out) + row * p.out_row + col, sum + 32 * h, left, wide);
          else
            store_f32<64>(static_cast<float*>(p.out) + row * p.out_row + col, sum + 32 * h, left, wide, p.add);
        }
      } else {
        constexpr int N = C::CW / 2;
        const int64_t col = (int64_t)nt * 128 + N * part;
        // the amax of this row's values and the other parts'
        auto other = [&](uint32_t m) {
          uint32_t(&x)[C::PARTS][128] = xch[turn++ & 1];
          x[part][32 * q + lane] = m;
          asm volatile("bar.sync %0, %1;" ::"r"(1 + q), "n"(32 * C::PARTS) : "memory");
#pragma unroll
          for (int o = 1; o < C::PARTS; ++o) m = max(m, x[(part + o) % C::PARTS][32 * q + lane]);
          return m;
        };
        const bool stores = !failed && col < p.n;
        if (p.g.data) store_f8<N>(p.g, row, col, stores, sum, other);
        if (p.u.data) store_f8<N>(p.u, row, col, stores, sum + N / 2, other);
        f32x2* const h = sum;
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          const float lo = f8_act<ACT>(f2_lo(h[e])), hi = f8_act<ACT>(f2_hi(h[e]));
          h[e] = f2_mul(f2_make(lo, hi), h[N / 2 + e]);
        }
        if constexpr (OUT == kF8GatedCodes) {
          store_f8<N>(p.h, row, col, stores, h, other);
        } else if (stores && row < p.m) {
          store_bf16(static_cast<uint16_t*>(p.out) + row * p.out_row + col, h, (int)(p.n - col < N ? p.n - col : N), wide);
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

// ---- few tokens: weight rows on the instruction's M side, K split over a cluster -----------
//
// A CTA makes a part of the sums of 128 output columns (weight rows, the
// instruction's M; gated: 128 of the gate and the same 128 of the
// up-projection) for TN tokens (its N): the part of its range of K.  The CTAs of
// a cluster share one tile and split K evenly.  Two CTAs an SM, whose first
// warpgroup loads, issues and makes scales; a thread of the second holds the
// sums of its weight row, TN (gated 2 TN) of them, each block of K's scaled and
// added as above.  Then the parts meet in shared memory (over the stages, which
// are done with), a row of 128 floats for each token, and every CTA adds up and
// stores a share of the tokens, a warp a token: the gated block's scale of a
// token's 128 values is then one warp's maximum.
constexpr int kF8MaxSplit = 8;

template <int TN, bool GATED, bool ROWS_W>
struct F8NarrowCfg {
  static constexpr int WT = GATED ? 2 : 1;  // weight tiles
  static constexpr uint32_t W_BYTES = 128 * 128 * WT, A_BYTES = TN * 128, STAGE = W_BYTES + A_BYTES;
  // scales of four blocks: TN products with the block's (gated: gate's, then
  // up's); ROWS_W: the TN tokens' scales and the 128 weight rows'
  static constexpr int GROUP = 4, SF_RING = 2;
  static constexpr uint32_t SF_BLOCK = (ROWS_W ? TN + 128 : WT * TN) * 4, SF_BYTES = GROUP * SF_BLOCK;
  static constexpr int STAGES_FIT = (112 * 1024 - 1024 - SF_RING * (int)SF_BYTES) / (int)STAGE;
  static constexpr int STAGES = STAGES_FIT < 6 ? STAGES_FIT : 6;
  static constexpr uint32_t SMEM = STAGES * STAGE + SF_RING * SF_BYTES + 1024;
  static constexpr int ACC_COLS = WT * TN;
  static constexpr int COLS = pow2_at_least(2 * ACC_COLS < 32 ? 32 : 2 * ACC_COLS);
  static constexpr int THREADS = 256;
  static constexpr int REGS_FEW = 40, REGS_MANY = 208;
  static_assert(128 * (REGS_FEW + REGS_MANY) <= 128 * THREADS, "the split of the registers");
  static_assert(STAGES >= 2 && COLS <= 256 && SMEM <= 113 * 1024, "two CTAs an SM");
  static_assert(STAGES * STAGE >= WT * TN * 128 * 4, "the parts fit over the stages");
  static_assert(WT * TN <= 128, "sums in registers");
};

// Four neighbouring columns of a token's row, from column n on.
__device__ __forceinline__ void store_four(const F8ProductParams& p, int out_type, int64_t m, int64_t n, const float4& x) {
  const float v[4] = {x.x, x.y, x.z, x.w};
  if (out_type == ATTN_RES_OUT_BF16) {
    uint16_t* const o = static_cast<uint16_t*>(p.out) + m * p.out_row + n;
    const uint32_t lo = pack_bf16x2(x.x, x.y), hi = pack_bf16x2(x.z, x.w);
    if (n + 4 <= p.n) {
      *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (n + e < p.n) o[e] = (uint16_t)((e < 2 ? lo : hi) >> (16 * (e % 2)));
    }
  } else {
    float* const o = static_cast<float*>(p.out) + m * p.out_row + n;
    if (n + 4 <= p.n) {
      float4 y = x;
      if (p.add) {
        const float4 b = *reinterpret_cast<const float4*>(o);
        y = make_float4(x.x + b.x, x.y + b.y, x.z + b.z, x.w + b.w);
      }
      *reinterpret_cast<float4*>(o) = y;
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (n + e < p.n) o[e] = v[e] + (p.add ? o[e] : 0.f);
    }
  }
}
// The same in codes; the warp's lanes hold all 128 columns from n - 4 lane on.
__device__ __forceinline__ void store_four_codes(const F8View& q, int64_t m, int64_t n, const float4& x) {
  const F8Scale s = f8_scale(__float_as_uint(warp_amax(amax3(amax3(0.f, x.x, x.y), x.z, x.w))));
  if (n % kF8Block == 0) q.scales[n / kF8Block * q.scales_row + m] = s.by;
  const uint32_t c = f8_codes(f2_make(x.x, x.y), f2_make(x.z, x.w), s);
  uint8_t* const o = q.data + m * q.row_bytes + n;
  if (n + 4 <= q.cols) {
    *reinterpret_cast<uint32_t*>(o) = c;
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (n + e < q.cols) o[e] = (uint8_t)(c >> (8 * e));
  }
}

template <int TN, bool GATED, bool ROWS_W>
__global__ void __launch_bounds__(256, 2)
    attn_res_f8_narrow_kernel(const __grid_constant__ F8ProductParams p, const int out_type, const int act,
                              const bool early_weights, const __grid_constant__ F8ProductMaps maps) {
  using C = F8NarrowCfg<TN, GATED, ROWS_W>;
  constexpr int S = C::STAGES, R = C::SF_RING, WT = C::WT;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) unsigned long long bars[2 * S + 4 + 2 * R];
  __shared__ uint32_t tmem_slot;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), split = (int)cluster_nctarank();
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t full = smem_addr(bars), empty = full + 8 * S, acc_full = empty + 8 * S, acc_empty = acc_full + 16,
                 sf_full = acc_empty + 16, sf_empty = sf_full + 8 * R;
  const uint32_t w_at = base, a_at = base + S * C::W_BYTES, sf_at = base + S * C::STAGE;
  const int n0 = (int)(blockIdx.x / split) * 128, m0 = (int)blockIdx.y * TN;
  const int blocks0 = p.blocks[0], all_blocks = blocks0 + p.blocks[1];
  const int k0 = (int)((int64_t)all_blocks * rank / split);
  const int blocks = (int)((int64_t)all_blocks * (rank + 1) / split) - k0;
  const int ahead = blocks < S ? blocks : S;
  bool failed = false;

  auto load_w = [&](int i, int s) {
    const int k = k0 + i, t = k < blocks0 ? 0 : 1, kb = k < blocks0 ? k : k - blocks0;
    const uint32_t bar = full + 8 * s;
    mbar_arrive_expect_tx(bar, C::STAGE);
    tma_load_2d(w_at + s * C::W_BYTES, &maps.w[GATED ? 0 : t], kb * 128, n0, bar);
    if constexpr (GATED) tma_load_2d(w_at + s * C::W_BYTES + 128 * 128, &maps.w[1], kb * 128, n0, bar);
  };
  auto load_a = [&](int i, int s) {
    const int k = k0 + i, t = k < blocks0 ? 0 : 1, kb = k < blocks0 ? k : k - blocks0;
    tma_load_2d(a_at + s * C::A_BYTES, &maps.a[t], kb * 128, m0, full + 8 * s);
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * S + 2; ++i) mbar_init(full + 8 * i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(acc_empty + 8 * i, 4);
    for (int i = 0; i < R; ++i) {
      mbar_init(sf_full + 8 * i, 1);
      mbar_init(sf_empty + 8 * i, 4);
    }
    fence_mbar_init();
    // with ATTN_RES_FLAG_PDL the weights do not depend on the preceding kernel:
    // the first stages' are on their way before the wait for it
    if (early_weights)
      for (int i = 0; i < ahead; ++i) load_w(i, i);
  }
  grid_dep_wait();
  if (threadIdx.x == 0)
    for (int i = 0; i < ahead; ++i) {
      if (!early_weights) load_w(i, i);
      load_a(i, i);
    }
  // (TMEM only now: while the preceding kernel runs it may need it itself)
  if (warp == 1) tmem_alloc<1>(smem_addr(&tmem_slot), C::COLS);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);  // uniform for the compiler

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_FEW));
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
      constexpr uint32_t idesc = f8_idesc(128, TN);
      const bool issuer = elect_one();
      const uint32_t w_lo = desc_lo(w_at), a_lo = desc_lo(a_at);
      for (int i = 0; i < blocks; ++i) {
        const int s = i % S, acc = i & 1;
        phase_or_flag(full + 8 * s, (i / S) & 1, failed, p.err, kErrStageTimeout);
        if (i >= 2) phase_or_flag(acc_empty + 8 * acc, ((i >> 1) - 1) & 1, failed, p.err, kErrStageTimeout);
        failed = __any_sync(0xffffffffu, failed);
        if (failed) {
          drain_stages<S>(full, s, i / S);
          break;
        }
        tmem_fence_after();
        if (issuer) {
#pragma unroll
          for (int t = 0; t < WT; ++t)
            f8_block<1>(tmem + acc * C::ACC_COLS + t * TN, w_lo + (s * C::W_BYTES + t * 128 * 128 >> 4),
                        a_lo + s * (C::A_BYTES >> 4), idesc);
          mma_commit<1>(acc_full + 8 * acc);
          mma_commit<1>(empty + 8 * s);
        }
        __syncwarp();
      }
    } else if (warp == 2) {
      for (int k4 = 0, group = 0; k4 < blocks; k4 += C::GROUP, ++group) {
        const uint32_t r = group % R, slot = sf_at + r * C::SF_BYTES;
        // (a lane's tokens of a block, and four weight rows)
        constexpr int PER = (TN + 31) / 32;
        float v[C::GROUP][PER], w[C::GROUP][ROWS_W ? 4 : WT];
#pragma unroll
        for (int j = 0; j < C::GROUP; ++j) {
          const int k = k0 + k4 + j;
          const bool one = k < blocks0, in = k4 + j < blocks;
          const int64_t kb = one ? k : k - blocks0;
          const F8Scales& sa = p.a[one ? 0 : 1];
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            const int64_t m = m0 + 32 * e + lane;
            v[j][e] = in && m < p.m ? sa.at[kb * sa.row + m] : 1.f;
          }
          if constexpr (ROWS_W) {
            const F8Scales& sw = p.w[one ? 0 : 1];
            ld_scales4(sw.at + kb * sw.row, n0 + 4 * lane, in ? p.n : 0, w[j]);
          } else {
#pragma unroll
            for (int t = 0; t < WT; ++t) {
              const F8Scales& sw = p.w[GATED ? t : one ? 0 : 1];
              w[j][t] = in ? sw.at[n0 / 128 * sw.row + kb] : 1.f;
            }
          }
        }
        if (group >= R) phase_or_flag(sf_empty + 8 * r, (group / R - 1) & 1, failed, p.err, kErrStageTimeout);
        failed = __any_sync(0xffffffffu, failed);
        if (failed) break;
#pragma unroll
        for (int j = 0; j < C::GROUP; ++j) {
          const uint32_t at = slot + j * C::SF_BLOCK;
#pragma unroll
          for (int e = 0; e < PER; ++e)
            if (32 * e + lane < TN) {
#pragma unroll
              for (int t = 0; t < WT; ++t)
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 4 * (t * TN + 32 * e + lane)),
                             "f"(ROWS_W ? v[j][e] : v[j][e] * w[j][ROWS_W ? 0 : t])
                             : "memory");
            }
          if constexpr (ROWS_W) st_shared4(at + 4 * TN + 16 * lane, w[j][0], w[j][1], w[j][2], w[j][3]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sf_full + 8 * r);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_MANY));
    const int q = warp % 4;  // warp w reads the TMEM lanes 32 (w % 4) .., that is the weight rows n0 + those
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
    constexpr int CH = TN >= 32 ? 32 : 16, PIECES = C::ACC_COLS / CH;  // columns at a time
    f32x2 sum[C::ACC_COLS / 2];
#pragma unroll
    for (int e = 0; e < C::ACC_COLS / 2; ++e) sum[e] = f2_make(0.f, 0.f);
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (phase_done(bar, parity) || failed) return;
      if (!phase_wait(bar, parity)) {
        failed = true;
        atomicOr(p.err, kErrStageTimeout);
      }
    };
#pragma unroll 1
    for (int i = 0; i < blocks; ++i) {
      const int acc = i & 1, group = i / C::GROUP, in_group = i % C::GROUP, r = group % R;
      if (in_group == 0) wait(sf_full + 8 * r, (group / R) & 1);
      const uint32_t at = sf_at + r * C::SF_BYTES + in_group * C::SF_BLOCK;
      float mine = 1.f;  // ROWS_W: this weight row's scale
      if constexpr (ROWS_W) mine = ld_shared(at + 4 * (TN + 32 * q + lane));
      wait(acc_full + 8 * acc, (i >> 1) & 1);
      __syncwarp();
      tmem_fence_after();
#pragma unroll
      for (int c = 0; c < PIECES; ++c) {
        uint32_t v[CH];
        tmem_ld(lanes + acc * C::ACC_COLS + CH * c, v);
        tmem_ld_wait(v);
        if (c == PIECES - 1) {
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty + 8 * acc);
        }
#pragma unroll
        for (int e = 0; e < CH / 2; e += 2) {
          f32x2 s[2];
          ld_shared_pairs(at + 4 * (CH * c + 2 * e), s);
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const f32x2 x = f2_make(__uint_as_float(v[2 * (e + o)]), __uint_as_float(v[2 * (e + o) + 1]));
            f32x2& to = sum[CH / 2 * c + e + o];
            to = f2_fma(x, ROWS_W ? f2_mul(s[o], f2_make(mine, mine)) : s[o], to);
          }
        }
      }
      if (in_group == C::GROUP - 1 || i == blocks - 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(sf_empty + 8 * r);
      }
    }
    failed = __any_sync(0xffffffffu, failed);
    grid_dep_launch_dependents();
    // The parts, over the stages: every product that read these is complete, and
    // so is every copy into them (unless a wait has given up).
    if (!failed) {
#pragma unroll
      for (int e = 0; e < C::ACC_COLS; ++e)
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + 4 * (128 * e + 32 * q + lane)),
                     "f"(e % 2 ? f2_hi(sum[e / 2]) : f2_lo(sum[e / 2]))
                     : "memory");
    }
    __syncwarp();
    if (split > 1) cluster_sync();
    else asm volatile("bar.sync 1, 128;" ::: "memory");
    const int64_t left = p.m - m0;
    const int tokens = left < TN ? (int)left : TN;
    const int64_t n = n0 + 4 * lane;
#pragma unroll 1
    for (int t = rank * 4 + q; t < tokens; t += split * 4) {
      float4 x[WT];
#pragma unroll
      for (int y = 0; y < WT; ++y) {
        const uint32_t at = base + 4 * (128 * (TN * y + t) + 4 * lane);
        float4 part[kF8MaxSplit];  // the loads of all parts together; added in the ranks' order
#pragma unroll
        for (int k = 0; k < kF8MaxSplit; ++k)
          if (k < split)
            asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(part[k].x), "=f"(part[k].y), "=f"(part[k].z), "=f"(part[k].w)
                         : "r"(map_rank(at, (uint32_t)k))
                         : "memory");
        x[y] = part[0];
#pragma unroll
        for (int k = 1; k < kF8MaxSplit; ++k)
          if (k < split)
            x[y] = make_float4(x[y].x + part[k].x, x[y].y + part[k].y, x[y].z + part[k].z, x[y].w + part[k].w);
      }
      if (failed) continue;
      const int64_t m = m0 + t;
      if constexpr (!GATED) {
        store_four(p, out_type, m, n, x[0]);
      } else {
        if (p.g.data) store_four_codes(p.g, m, n, x[0]);
        if (p.u.data) store_four_codes(p.u, m, n, x[WT - 1]);
        auto one = [&](float g, float u) {
          return (act == ATTN_RES_SILU ? f8_act<ATTN_RES_SILU>(g) : f8_act<ATTN_RES_GELU>(g)) * u;
        };
        const float4& u = x[WT - 1];
        const float4 h = make_float4(one(x[0].x, u.x), one(x[0].y, u.y), one(x[0].z, u.z), one(x[0].w, u.w));
        if (p.h.data) store_four_codes(p.h, m, n, h);
        else store_four(p, ATTN_RES_OUT_BF16, m, n, h);
      }
    }
  }
  __syncwarp();
  if (warp < 4 && split > 1) cluster_sync();  // (the parts' way, which the other four go)
  // No CTA ends while its parts are being read: every load's value has been used
  // by then, so the arrival orders nothing.
  __syncwarp();
  if (split > 1) cluster_arrive_relaxed();
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

}  // namespace attn_res_dev
