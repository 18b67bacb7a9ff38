// attn_res_mx_product.cuh -- products of two microscaled matrices on the
// block-scaled tensor-core instructions (tcgen05.mma ... block_scale).
#pragma once

#include <cuda.h>

#include "attn_res_mx.cuh"

namespace attn_res_dev {

// ---- tcgen05 ---------------------------------------------------------------------------

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}
__device__ __forceinline__ void tmem_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
// 512 bytes of scales (32 rows of 16 bytes) to four TMEM columns, the 32
// lanes repeated in every quarter of the lanes.
__device__ __forceinline__ void scales_to_tmem(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

template <int FMT>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (FMT == ATTN_RES_MXFP8) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  } else if constexpr (FMT == ATTN_RES_MXFP4) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  }
}

// Shared-memory descriptor of a K-major operand in 128-byte swizzled rows
// (eight rows of 128 bytes = 1024 bytes between row groups).
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3fffu) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// Of a 32 x 16-byte scale tile, not swizzled (128 bytes between groups of
// eight rows).
__device__ __forceinline__ uint64_t scales_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3fffu) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

// A 128-byte block of a K-major row: 128 e4m3 elements or 256 e2m1, taken by
// the tensor cores 32 bytes at a time.
template <int FMT>
struct ProductFmt {
  static constexpr int GROUPS = FMT == ATTN_RES_MXFP8 ? 4 : FMT == ATTN_RES_MXFP4 ? 8 : 16;
  static constexpr int ATOMS = GROUPS / 4;       // scale tiles of four groups in a block
  static constexpr int STEPS_PER_ATOM = 4 / ATOMS;  // 32-byte steps that share a scale tile
  // instruction descriptor: element types, scale type, M = 128
  static constexpr uint32_t TYPE = FMT == ATTN_RES_MXFP8 ? 0u : 1u;  // e4m3 (8-bit kind), e2m1 (4-bit kinds)
  static constexpr uint32_t IDESC = TYPE << 7 | TYPE << 10 |
                                    (FMT == ATTN_RES_NVFP4 ? 0u : 1u) << 23 | (128u >> 4) << 24;
};
// The instruction's choice of scale bytes for step j of a scale tile: one,
// two or four of its four groups.
template <int FMT>
__device__ __forceinline__ uint32_t step_idesc(uint32_t idesc, int j) {
  const uint32_t id = FMT == ATTN_RES_MXFP8 ? j & 3 : FMT == ATTN_RES_MXFP4 ? (j & 1) * 2 : 0;
  return idesc | id << 4 | id << 29;
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
  unsigned* err;
};

// ---- weight rows on the instruction's M side ----------------------------------------------
//
// A CTA makes 128 output columns (weight rows, the instruction's M) for TN
// tokens (its N).  TN < 128 only with a single token tile: a tile's token
// scales then start at the first of their scale tile's columns.
template <int FMT, int TN>
struct ProductCfg {
  using F = ProductFmt<FMT>;
  static constexpr uint32_t W_BYTES = 128 * 128;
  static constexpr uint32_t A_BYTES = TN * 128;
  static constexpr uint32_t SF_BYTES = F::ATOMS * 512;
  static constexpr uint32_t STAGE = W_BYTES + A_BYTES + 2 * SF_BYTES;
  static constexpr int STAGES = 4;
  static constexpr uint32_t SMEM = STAGES * STAGE + 1024;
  // TMEM columns: the accumulator, then for each stage its scales (so that a
  // stage's scales are replaced only after the products that read them)
  static constexpr int SF_COLS = F::ATOMS * 4;
  static constexpr int COLS_USED = TN + STAGES * 2 * SF_COLS;
  static constexpr int COLS = pow2_at_least(COLS_USED < 32 ? 32 : COLS_USED);
  static_assert(COLS <= 512, "TMEM");
  static constexpr int THREADS = 192;
};

template <int FMT, int TN>
__global__ void __launch_bounds__(192)
    attn_res_mx_product_kernel(const ProductParams p, const __grid_constant__ CUtensorMap map_a,
                               const __grid_constant__ CUtensorMap map_w) {
  using C = ProductCfg<FMT, TN>;
  using F = ProductFmt<FMT>;
  constexpr int S = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) unsigned long long bars[2 * S + 1];
  __shared__ uint32_t tmem_slot;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t full = smem_addr(bars), empty = full + 8 * S, done = empty + 8 * S;
  auto w_at = [&](int s) { return base + s * C::W_BYTES; };
  auto a_at = [&](int s) { return base + S * C::W_BYTES + s * C::A_BYTES; };
  auto wsf_at = [&](int s) { return base + S * (C::W_BYTES + C::A_BYTES) + s * 2 * C::SF_BYTES; };
  auto asf_at = [&](int s) { return wsf_at(s) + C::SF_BYTES; };
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * S + 1; ++i) mbar_init(full + 8 * i, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), C::COLS);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = tmem_slot;
  const int64_t n0 = (int64_t)blockIdx.x * 128, m0 = (int64_t)blockIdx.y * TN;
  const int blocks = (p.row_bytes_used + 127) / 128;
  grid_dep_wait();

  if (warp == 0 && lane == 0) {
    bool failed = false;
    const uint8_t* wsf = p.w_scales + (n0 / 128) * p.group_tiles * 512;
    const uint8_t* asf = p.a_scales + (m0 / 128) * p.group_tiles * 512;
    int issued = 0;
    for (int kb = 0; kb < blocks; ++kb) {
      const int s = kb % S, use = kb / S;
      if (use > 0) wait_or_flag(empty + 8 * s, (use - 1) & 1, failed, p.err, kErrStageTimeout);
      if (failed) break;
      const int64_t left = p.group_tiles - (int64_t)kb * F::ATOMS;
      const uint32_t sf = (uint32_t)(left < F::ATOMS ? left : F::ATOMS) * 512u;
      const uint32_t bar = full + 8 * s;
      mbar_arrive_expect_tx(bar, C::W_BYTES + C::A_BYTES + 2 * sf);
      tma_load_2d(w_at(s), &map_w, kb * 128, (int)n0, bar);
      tma_load_2d(a_at(s), &map_a, kb * 128, (int)m0, bar);
      bulk_load(wsf_at(s), wsf + (int64_t)kb * F::ATOMS * 512, sf, bar);
      bulk_load(asf_at(s), asf + (int64_t)kb * F::ATOMS * 512, sf, bar);
      issued = kb + 1;
    }
    if (failed)  // copies still in flight land before the CTA ends
      for (int kb = issued > S ? issued - S : 0; kb < issued; ++kb)
        (void)mbar_wait_bounded(full + 8 * (kb % S), (kb / S) & 1);
  } else if (warp == 1 && lane == 0) {
    bool failed = false;
    const uint32_t idesc = F::IDESC | (uint32_t)(TN >> 3) << 17;
    for (int kb = 0; kb < blocks; ++kb) {
      const int s = kb % S, use = kb / S;
      wait_or_flag(full + 8 * s, use & 1, failed, p.err, kErrStageTimeout);
      if (failed) break;
      tmem_fence_after();
      const uint32_t sf = tmem + TN + s * 2 * C::SF_COLS;
      const int bytes = p.row_bytes_used - kb * 128;
      const int steps = bytes >= 128 ? 4 : (bytes + 31) / 32;
      const int atoms = (steps + F::STEPS_PER_ATOM - 1) / F::STEPS_PER_ATOM;
      for (int i = 0; i < atoms; ++i) {
        scales_to_tmem(sf + 4 * i, scales_desc(wsf_at(s) + 512 * i));
        scales_to_tmem(sf + C::SF_COLS + 4 * i, scales_desc(asf_at(s) + 512 * i));
      }
      for (int j = 0; j < steps; ++j) {
        const int i = j / F::STEPS_PER_ATOM;
        mma_scaled<FMT>(tmem, operand_desc(w_at(s) + 32 * j), operand_desc(a_at(s) + 32 * j),
                        step_idesc<FMT>(idesc, j), sf + 4 * i, sf + C::SF_COLS + 4 * i,
                        kb > 0 || j > 0);
      }
      mma_commit(empty + 8 * s);
    }
    mma_commit(done);
  } else if (warp >= 2) {
    // warp w reads the TMEM lanes 32 (w % 4) ..: weight rows n0 + those
    bool failed = false;
    wait_or_flag(done, 0, failed, p.err, kErrStageTimeout);
    tmem_fence_after();
    grid_dep_launch_dependents();
    const float scale = tensor_scale_of(p.a_g) * tensor_scale_of(p.w_g);
    const int q = warp % 4;
    const int64_t n = n0 + 32 * q + lane;
    for (int c = 0; c < TN; c += 16) {
      uint32_t r[16];
      tmem_ld16(tmem + ((uint32_t)(32 * q) << 16) + c, r);
      tmem_ld_wait();
      for (int j = 0; j < 16; ++j) {
        const int64_t m = m0 + c + j;
        if (!failed && n < p.n && m < p.m)
          p.out[m * p.out_row + n] =
              (uint16_t)pack_bf16x2(__uint_as_float(r[j]) * scale, 0.f);
      }
    }
    tmem_fence_before();
  }
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    tmem_free(tmem, C::COLS);
  }
}

}  // namespace attn_res_dev
