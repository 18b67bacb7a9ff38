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
// The same with the barrier in any CTA of the pair (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y,
                                                 uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// mbar_wait_bounded and wait_or_flag for a barrier that other CTAs arrive on.
__device__ __forceinline__ void wait_or_flag_cluster(uint32_t bar, uint32_t parity, bool& failed,
                                                     unsigned* err, unsigned bit) {
  if (failed) return;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return;
    if ((it & 1023u) == 0 && global_timer_ns() - t0 > kWaitLimitNs) break;
  }
  failed = true;
  atomicOr(err, bit);
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// tcgen05 for one CTA (G = 1) or a pair (G = 2; issued by the pair's first
// CTA, except alloc and free, which both execute).
template <int G>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  if constexpr (G == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int G>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  if constexpr (G == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Arrive on `bar` (G = 2: the barrier at its place in both CTAs) once every
// MMA and copy that this thread has issued is complete.
template <int G>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  if constexpr (G == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
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
  if (warp == 1) tmem_alloc<1>(smem_addr(&tmem_slot), C::COLS);
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
    const uint32_t idesc = F::idesc(128, TN);
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
        scales_to_tmem<1>(sf + 4 * i, scales_desc(wsf_at(s) + 512 * i));
        scales_to_tmem<1>(sf + C::SF_COLS + 4 * i, scales_desc(asf_at(s) + 512 * i));
      }
      for (int j = 0; j < steps; ++j) {
        const int i = j / F::STEPS_PER_ATOM;
        mma_scaled<FMT, 1>(tmem, operand_desc(w_at(s) + 32 * j), operand_desc(a_at(s) + 32 * j),
                        step_idesc<FMT>(idesc, j), sf + 4 * i, sf + C::SF_COLS + 4 * i,
                        kb > 0 || j > 0);
      }
      mma_commit<1>(empty + 8 * s);
    }
    mma_commit<1>(done);
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
    tmem_free<1>(tmem, C::COLS);
  }
}

// ---- many tokens: CTA pairs, 256 x 256 tiles ------------------------------------------------
//
// A pair of CTAs (cta_group::2) makes 256 tokens x 256 output columns: each
// holds 128 tokens' rows, half of the weight rows (the instruction reads the
// other half from the peer) and the scales of its tokens and of all 256
// weight rows.  Persistent pairs walk the tiles; warp 0 loads, warp 1 of the
// first CTA issues the MMAs of both, warps 4..11 drain the accumulator: to
// bf16 in registers first, which frees it for the next tile, then through
// shared memory to bulk tensor stores.
template <int FMT>
struct WideCfg {
  using F = ProductFmt<FMT>;
  static constexpr int TM = 256, TN = 256;
  static constexpr uint32_t A_BYTES = 128 * 128, W_BYTES = 128 * 128;
  static constexpr uint32_t SF_BYTES = F::ATOMS * 512;  // of 128 rows
  static constexpr uint32_t STAGE = A_BYTES + W_BYTES + 3 * SF_BYTES;
  static constexpr int STAGES = 5;
  static constexpr uint32_t OUT_BYTES = 32 * 128;  // one warp's 32 rows x 64 columns
  static constexpr int EPI_WARPS = 8;
  static constexpr uint32_t SMEM = STAGES * STAGE + EPI_WARPS * OUT_BYTES + 1024;
  static constexpr int SF_COLS = F::ATOMS * 4;  // TMEM columns of 128 rows' scales
  static constexpr int COLS = 512;
  static_assert(TN + STAGES * 3 * SF_COLS <= COLS, "TMEM");
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
};

struct WideMaps {
  CUtensorMap a, w, a_sf, w_sf, out;
};

struct TileWalk {
  int64_t m_tiles, n_tiles;
};
// Tile `i` of the walk: bands of kBand token tiles, column by column within a
// band, so that the pairs at work share weight rows and token rows in L2.
constexpr int64_t kBand = 8;
__device__ __forceinline__ void tile_at(const TileWalk& w, int64_t i, int64_t& mt, int64_t& nt) {
  const int64_t band = i / (kBand * w.n_tiles);
  const int64_t left = w.m_tiles - band * kBand;
  const int64_t rows = left < kBand ? left : kBand;
  const int64_t j = i - band * kBand * w.n_tiles;
  mt = band * kBand + j % rows;
  nt = j / rows;
}

template <int FMT>
__global__ void __launch_bounds__(WideCfg<FMT>::THREADS, 1)
    attn_res_mx_product_wide_kernel(const ProductParams p, const TileWalk walk,
                                    const __grid_constant__ WideMaps maps) {
  using C = WideCfg<FMT>;
  using F = ProductFmt<FMT>;
  constexpr int S = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) unsigned long long bars[2 * S + 2];
  __shared__ uint32_t tmem_slot;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t full = smem_addr(bars), empty = full + 8 * S, acc_full = empty + 8 * S,
                 acc_empty = acc_full + 8;
  auto a_at = [&](int s) { return base + s * C::A_BYTES; };
  auto w_at = [&](int s) { return base + S * C::A_BYTES + s * C::W_BYTES; };
  const uint32_t out_at = base + S * (C::A_BYTES + C::W_BYTES);  // 1024-byte aligned, as the swizzle wants
  auto sf_at = [&](int s) { return out_at + C::EPI_WARPS * C::OUT_BYTES + s * 3 * C::SF_BYTES; };
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * S + 1; ++i) mbar_init(full + 8 * i, 1);
    mbar_init(acc_empty, 2 * C::EPI_WARPS);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc<2>(smem_addr(&tmem_slot), C::COLS);
  tmem_fence_before();
  __syncthreads();
  cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = tmem_slot;
  const int64_t tiles = walk.m_tiles * walk.n_tiles;
  const int64_t first = blockIdx.x / 2, step = gridDim.x / 2;
  const int blocks = (p.row_bytes_used + 127) / 128;
  grid_dep_wait();

  if (warp == 0 && lane == 0) {
    bool failed = false;
    int s = 0;
    uint32_t use = 0, issued = 0;
    const int tiles_k = (int)p.group_tiles;
    for (int64_t i = first; i < tiles && !failed; i += step) {
      int64_t mt, nt;
      tile_at(walk, i, mt, nt);
      const int a_row = (int)(mt * 256 + rank * 128), w_row = (int)(nt * 256 + rank * 128);
      for (int kb = 0; kb < blocks; ++kb) {
        if (use > 0) wait_or_flag(empty + 8 * s, (use - 1) & 1, failed, p.err, kErrStageTimeout);
        if (failed) break;
        const uint32_t bar = full + 8 * s, bar0 = map_rank(bar, 0);
        if (rank == 0) mbar_arrive_expect_tx(bar, 2 * C::STAGE);
        const int sf_row = kb * F::ATOMS;
        tma_load_2d_pair(a_at(s), &maps.a, kb * 128, a_row, bar0);
        tma_load_2d_pair(w_at(s), &maps.w, kb * 128, w_row, bar0);
        tma_load_2d_pair(sf_at(s), &maps.a_sf, 0, a_row / 128 * tiles_k + sf_row, bar0);
        tma_load_2d_pair(sf_at(s) + C::SF_BYTES, &maps.w_sf, 0, (int)nt * 2 * tiles_k + sf_row, bar0);
        tma_load_2d_pair(sf_at(s) + 2 * C::SF_BYTES, &maps.w_sf, 0, ((int)nt * 2 + 1) * tiles_k + sf_row, bar0);
        ++issued;
        if (++s == S) {
          s = 0;
          ++use;
        }
      }
    }
    if (failed && rank == 0)  // copies still in flight (the peer's too) land before the CTAs end
      for (uint32_t b = issued > S ? issued - S : 0; b < issued; ++b)
        (void)mbar_wait_bounded(full + 8 * (b % S), (b / S) & 1);
  } else if (warp == 1 && lane == 0 && rank == 0) {
    bool failed = false;
    int s = 0;
    uint32_t use = 0, tile = 0;
    constexpr uint32_t idesc = F::idesc(256, 256);
    for (int64_t i = first; i < tiles && !failed; i += step, ++tile) {
      if (tile > 0)
        wait_or_flag_cluster(acc_empty, (tile - 1) & 1, failed, p.err, kErrExchangeTimeout);
      for (int kb = 0; kb < blocks && !failed; ++kb) {
        wait_or_flag(full + 8 * s, use & 1, failed, p.err, kErrStageTimeout);
        if (failed) break;
        tmem_fence_after();
        const uint32_t sf = tmem + C::TN + s * 3 * C::SF_COLS;
        const int bytes = p.row_bytes_used - kb * 128;
        const int steps = bytes >= 128 ? 4 : (bytes + 31) / 32;
        const int atoms = (steps + F::STEPS_PER_ATOM - 1) / F::STEPS_PER_ATOM;
        for (int t = 0; t < atoms; ++t) {
          // the token scales, and beside each other those of both halves of the weight rows
          scales_to_tmem<2>(sf + 4 * t, scales_desc(sf_at(s) + 512 * t));
          scales_to_tmem<2>(sf + C::SF_COLS + 8 * t, scales_desc(sf_at(s) + C::SF_BYTES + 512 * t));
          scales_to_tmem<2>(sf + C::SF_COLS + 8 * t + 4, scales_desc(sf_at(s) + 2 * C::SF_BYTES + 512 * t));
        }
        for (int j = 0; j < steps; ++j) {
          const int t = j / F::STEPS_PER_ATOM;
          mma_scaled<FMT, 2>(tmem, operand_desc(a_at(s) + 32 * j), operand_desc(w_at(s) + 32 * j),
                             step_idesc<FMT>(idesc, j), sf + 4 * t, sf + C::SF_COLS + 8 * t,
                             kb > 0 || j > 0);
        }
        mma_commit<2>(empty + 8 * s);
        if (++s == S) {
          s = 0;
          ++use;
        }
      }
      mma_commit<2>(acc_full);
    }
    if (failed) (void)mbar_wait_bounded(acc_full, (tile - 1) & 1);
  } else if (warp >= 4) {
    bool failed = false;
    uint32_t tile = 0;
    const int q = warp % 4, half = (warp - 4) / 4;
    const uint32_t stage = out_at + (uint32_t)(warp - 4) * C::OUT_BYTES;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + 128 * half;
    const float scale = tensor_scale_of(p.a_g) * tensor_scale_of(p.w_g);
    const uint32_t release = map_rank(acc_empty, 0);
    // a bulk tensor store ends on a 16-byte boundary: the columns behind the
    // last one are stored one by one
    const int64_t whole = p.n / 8 * 8;
    for (int64_t i = first; i < tiles && !failed; i += step, ++tile) {
      int64_t mt, nt;
      tile_at(walk, i, mt, nt);
      wait_or_flag(acc_full, tile & 1, failed, p.err, kErrStageTimeout);
      failed = __any_sync(0xffffffffu, failed);
      tmem_fence_after();
      if (i + step >= tiles) grid_dep_launch_dependents();
      uint32_t v[64];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t r[16];
        tmem_ld16(lanes + 16 * c, r);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          v[8 * c + k] = pack_bf16x2(__uint_as_float(r[2 * k]) * scale, __uint_as_float(r[2 * k + 1]) * scale);
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(release);
      const int row = (int)(mt * 256 + rank * 128 + 32 * q);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t col = nt * 256 + 128 * half + 64 * h;
        if (lane == 0) bulk_wait_read();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t at = stage + lane * 128 + ((k ^ (lane & 7)) * 16);
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[32 * h + 4 * k]),
                       "r"(v[32 * h + 4 * k + 1]), "r"(v[32 * h + 4 * k + 2]), "r"(v[32 * h + 4 * k + 3])
                       : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && !failed && row < p.m && col < whole) {
          tma_store_2d(&maps.out, (int)col, row, stage);
          bulk_commit();
        }
        if (whole >= col && whole < col + 64 && whole < p.n && !failed && row + lane < p.m) {
          const uint32_t at = stage + lane * 128 + ((((uint32_t)(whole - col) >> 3) ^ (lane & 7)) * 16);
          for (int k = 0; whole + k < p.n; ++k) {
            uint16_t e;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(e) : "r"(at + 2 * k) : "memory");
            p.out[(row + lane) * p.out_row + whole + k] = e;
          }
        }
      }
    }
    if (lane == 0) bulk_wait();
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
