// attn_res_tcgen05.cuh -- shared by the tensor-core kernels: PTX helpers
// (tensor-map copies, TMEM, tcgen05 barriers, shared-memory descriptors), the
// walk over output tiles and the stores of their rows.
#pragma once

#include <cuda.h>

#include "attn_res_common.cuh"
#include "attn_res_waits.cuh"

namespace attn_res_dev {

// ---- copies, TMEM, barriers, descriptors ------------------------------------------------

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
// An arrival that orders nothing in shared or global memory: it tells that
// this thread's TMEM loads are complete (they are: tcgen05.wait::ld has
// returned, and tcgen05.fence::before_thread_sync keeps them before it).  With
// release semantics it waited about 2000 clocks for the warp's earlier stores.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
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
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
// The loads that gave r are complete (r passes through, so that nothing uses
// it before).
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld64(uint32_t addr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(addr));
}
// The loads that gave r are complete (r passes through, so that nothing uses
// it before).
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[64]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]), "+r"(r[32]), "+r"(r[33]), "+r"(r[34]), "+r"(r[35]), "+r"(r[36]), "+r"(r[37]), "+r"(r[38]), "+r"(r[39]), "+r"(r[40]), "+r"(r[41]), "+r"(r[42]), "+r"(r[43]), "+r"(r[44]), "+r"(r[45]), "+r"(r[46]), "+r"(r[47]), "+r"(r[48]), "+r"(r[49]), "+r"(r[50]), "+r"(r[51]), "+r"(r[52]), "+r"(r[53]), "+r"(r[54]), "+r"(r[55]), "+r"(r[56]), "+r"(r[57]), "+r"(r[58]), "+r"(r[59]), "+r"(r[60]), "+r"(r[61]), "+r"(r[62]), "+r"(r[63])
               :
               : "memory");
}

// Shared-memory descriptors: the low word is the address in 16-byte units (and
// a leading offset that these layouts do not use), the high word a constant
// of the layout, so that steps within a stage are small additions.
// Operands: K-major rows of 128 swizzled bytes, eight rows (1024 bytes) apart.
constexpr uint32_t kOperandHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return (addr >> 4) | 1u << 16; }
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
// One lane of a converged warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// Behind a wait of the issuing warp that has given up at use `use` of stage
// `stage`: copies under way into the stages land before the CTA ends (bounded
// again).  A loading thread that has more to issue meets the same end at the
// stages that are not released, and waits for its own.
template <int S>
__device__ __forceinline__ void drain_stages(uint32_t full, int stage, uint32_t use) {
  uint64_t limit = kWaitLimitNs;
  for (int k = 0; k < S; ++k) {
    if (!phase_wait(full + 8 * stage, use & 1, limit)) limit = 0;
    if (++stage == S) {
      stage = 0;
      ++use;
    }
  }
}

// ---- output tiles ----------------------------------------------------------------------

struct TileWalk {
  int m_tiles, n_tiles;
};
// Tile `i` of the walk: bands of kBand token tiles, column by column within a
// band, so that the pairs at work share weight rows and token rows in L2.
constexpr int kBand = 8;
__device__ __forceinline__ void tile_at(const TileWalk& w, int i, int& mt, int& nt) {
  const int band = i / (kBand * w.n_tiles);
  const int left = w.m_tiles - band * kBand;
  const int rows = left < kBand ? left : kBand;
  const int j = i - band * kBand * w.n_tiles;
  nt = j / rows;
  mt = band * kBand + j - nt * rows;
}

// 64 fp32 columns of a thread's row as bf16 pairs.
__device__ __forceinline__ void pack64(const uint32_t (&r)[64], float scale, uint32_t (&v)[32]) {
#pragma unroll
  for (int k = 0; k < 32; ++k)
    v[k] = pack_bf16x2(__uint_as_float(r[2 * k]) * scale, __uint_as_float(r[2 * k + 1]) * scale);
}
// COUNT of them from FIRST on, `left` of which exist.
template <int FIRST, int COUNT>
__device__ __forceinline__ void store_piece(uint16_t* o, const uint32_t (&v)[32], int left) {
  uint16_t* const at = o + FIRST;
  constexpr int k = FIRST / 2;
  if (left >= FIRST + COUNT) {
    if constexpr (COUNT == 16)
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(v[k]), "r"(v[k + 1]),
                   "r"(v[k + 2]), "r"(v[k + 3]), "r"(v[k + 4]), "r"(v[k + 5]), "r"(v[k + 6]), "r"(v[k + 7])
                   : "memory");
    else
      st_row(at, make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]));
  } else {
#pragma unroll
    for (int e = 0; e < COUNT; ++e)
      if (FIRST + e < left) at[e] = (uint16_t)(v[k + e / 2] >> (16 * (e % 2)));
  }
}

// Stores 64 columns of a lane's row, `left` of which exist, straight from its
// registers: 32 bytes, a whole sector, at a time, after half a sector where the
// row lies between two of them; `wide`: none of the rows does, which a full
// tile then need not look at (2 % of a product's time).  (Half sectors alone: 1361 x 14008 x 864 mxfp8
// 28.4 us instead of 19.9.  Through shared memory and bulk tensor stores the same
// bytes pass shared memory twice, whose bandwidth the operands need: 4096 x
// 16384 x 2048 nvfp4 61 us instead of 56, 8192 x 7168 x 7168 mxfp4 115 either
// way.)
__device__ __forceinline__ void store_row(uint16_t* o, const uint32_t (&v)[32], int left, bool wide) {
  auto sectors = [&](int exist) {
    store_piece<0, 16>(o, v, exist);
    store_piece<16, 16>(o, v, exist);
    store_piece<32, 16>(o, v, exist);
    store_piece<48, 16>(o, v, exist);
  };
  if (wide && left >= 64) {
    sectors(64);
  } else if ((reinterpret_cast<uintptr_t>(o) & 16u) == 0) {
    sectors(left);
  } else {
    store_piece<0, 8>(o, v, left);
    store_piece<8, 16>(o, v, left);
    store_piece<24, 16>(o, v, left);
    store_piece<40, 16>(o, v, left);
    store_piece<56, 8>(o, v, left);
  }
}

}  // namespace attn_res_dev
