// attn_res_f8_rows.cuh -- quantisation into 8 bits with scales for blocks of
// 128, its inverse, and the backward pass of the gated block.
#pragma once

#include "attn_res_f8.cuh"
#include "attn_res_tcgen05.cuh"

namespace attn_res_dev {

constexpr int kF8Threads = 256;
constexpr int kF8Strip = 16;  // rows of a warp's strip, 128 columns wide

// ---- a warp's strip -----------------------------------------------------------------------
//
// A warp takes 16 rows x 128 columns, a lane four neighbouring columns of each
// row: the maximum of a row is one warp-wide integer reduction, that of a
// column stays in its lane, and the 16 codes of a column are one 16-byte piece
// of the transposed matrix.

// Four bf16 of a row from column `col` on, zeros behind the last.
__device__ __forceinline__ uint2 ld_bf16x4(const uint16_t* row, int64_t col, int64_t cols) {
  if (col + 4 <= cols) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(row + col));
    return v;
  }
  uint32_t e[4] = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (col + k < cols) e[k] = row[col + k];
  return make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
}
// Four codes.
__device__ __forceinline__ uint32_t ld_codes4(const uint8_t* row, int64_t col, int64_t cols) {
  if (col + 4 <= cols) return *reinterpret_cast<const uint32_t*>(row + col);
  uint32_t v = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (col + k < cols) v |= (uint32_t)row[col + k] << (8 * k);
  return v;
}
__device__ __forceinline__ void st_codes4(uint8_t* row, int64_t col, int64_t cols, uint32_t v) {
  if (col + 4 <= cols) {
    *reinterpret_cast<uint32_t*>(row + col) = v;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (col + k < cols) row[col + k] = (uint8_t)(v >> (8 * k));
  }
}

// The scales of the strip's rows from each lane's maxima over its columns:
// lane i makes that of row i, every lane gets all through shuffles.
struct StripScales {
  F8Scale mine;
  __device__ __forceinline__ explicit StripScales(const uint32_t (&amax)[kF8Strip]) {
    const int lane = threadIdx.x & 31;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kF8Strip; ++i) {
      const uint32_t r = __reduce_max_sync(0xffffffffu, amax[i]);
      if (lane == i) m = r;
    }
    mine = f8_scale(m);
  }
  __device__ __forceinline__ F8Scale of(int i) const {
    F8Scale s;
    s.by = __shfl_sync(0xffffffffu, mine.by, i);
    s.inverse = __shfl_sync(0xffffffffu, mine.inverse, i);
    return s;
  }
  // the lanes' scales into the matrix (rows row0 + lane of column block b)
  __device__ __forceinline__ void store(const F8View& q, int64_t row0, int64_t b) const {
    const int lane = threadIdx.x & 31;
    if (lane < kF8Strip && row0 + lane < q.rows) q.scales[b * q.scales_row + row0 + lane] = mine.by;
  }
};

// ---- a CTA's tile -------------------------------------------------------------------------
//
// Eight warps' strips make a tile of 128 x 128.  Scales of columns: the maxima
// of the warps' strips meet in shared memory.  The transposed codes pass
// through shared memory: column c's piece of warp w (16 bytes) lies at piece
// w ^ (c / 4 % 8) of the column's 128 bytes, so that neither the writes (lanes
// four columns apart) nor the reads (eight lanes a column) meet in a bank.
struct TileShared {
  uint4 codes[128][8];
  uint32_t amax[8][128];
  F8Scale scale[128];
};

__device__ __forceinline__ uint4& tile_piece(TileShared& t, int col, int piece) {
  return t.codes[col][piece ^ ((col >> 2) & 7)];
}

// Scales of the tile's columns from each lane's maxima over its strip's rows;
// written into the transposed matrix qt (its rows are the columns col0 ..).
// Ends with the CTA's threads synchronised.
__device__ __forceinline__ void tile_column_scales(TileShared& t, const uint32_t (&amax)[4], const F8View& qt,
                                                   int64_t col0, int64_t b) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  *reinterpret_cast<uint4*>(&t.amax[warp][4 * lane]) = make_uint4(amax[0], amax[1], amax[2], amax[3]);
  __syncthreads();
  if (threadIdx.x < 128) {
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, t.amax[w][threadIdx.x]);
    const F8Scale s = f8_scale(m);
    t.scale[threadIdx.x] = s;
    if (col0 + threadIdx.x < qt.rows) qt.scales[b * qt.scales_row + col0 + threadIdx.x] = s.by;
  }
  __syncthreads();
}

// The transposed codes from shared memory to qt: rows col0 .., bytes row0 ..
__device__ __forceinline__ void tile_store_transposed(TileShared& t, const F8View& qt, int64_t col0, int64_t row0) {
  for (int i = threadIdx.x; i < 128 * 8; i += kF8Threads) {
    const int c = i / 8, piece = i % 8;
    const int64_t at = row0 + 16 * piece;
    if (col0 + c >= qt.rows || at >= qt.cols) continue;
    const uint4 v = tile_piece(t, c, piece);
    uint8_t* const o = qt.data + (col0 + c) * qt.row_bytes + at;
    if (at + 16 <= qt.cols) {
      *reinterpret_cast<uint4*>(o) = v;
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (at + k < qt.cols) o[k] = (uint8_t)(vword(v, k / 4) >> (8 * (k % 4)));
    }
  }
}

// ---- quantisation -------------------------------------------------------------------------

struct F8QuantizeParams {
  const uint16_t* x;
  int64_t x_row;
  F8View q, t;  // t: the transposed matrix (the tile kernel)
};

// |x| of four bf16 as fp32 bits.
__device__ __forceinline__ uint32_t bf16x4_amax(uint2 v) {
  const uint32_t m = __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu);
  return max(m << 16, m & 0xffff0000u);
}

// Rows only: a warp a strip.
__global__ void __launch_bounds__(kF8Threads) attn_res_f8_quantize_rows_kernel(const F8QuantizeParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t blocks = f8_blocks(p.q.cols);
  const int64_t job = (int64_t)blockIdx.x * (kF8Threads / 32) + (threadIdx.x >> 5);
  const int64_t row0 = job / blocks * kF8Strip, b = job % blocks;
  grid_dep_wait();
  if (row0 < p.q.rows) {
    const int64_t col = b * kF8Block + 4 * lane;
    const int rows = (int)(p.q.rows - row0 < kF8Strip ? p.q.rows - row0 : kF8Strip);
    uint2 x[kF8Strip];
    uint32_t am[kF8Strip];
#pragma unroll
    for (int i = 0; i < kF8Strip; ++i)
      x[i] = i < rows ? ld_bf16x4(p.x + (row0 + i) * p.x_row, col, p.q.cols) : make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < kF8Strip; ++i) am[i] = bf16x4_amax(x[i]);
    const StripScales s(am);
    s.store(p.q, row0, b);
#pragma unroll
    for (int i = 0; i < kF8Strip; ++i) {
      const F8Scale si = s.of(i);
      if (i < rows)
        st_codes4(p.q.data + (row0 + i) * p.q.row_bytes, col, p.q.cols, f8_codes(bf2_widen(x[i].x), bf2_widen(x[i].y), si));
    }
  }
  grid_dep_launch_dependents();
}

// Tiles: block scales (SQUARE), or row scales with the transposed matrix too;
// TRANSPOSED: the transposed matrix.
template <bool SQUARE, bool TRANSPOSED>
__global__ void __launch_bounds__(kF8Threads) attn_res_f8_quantize_tile_kernel(const F8QuantizeParams p) {
  __shared__ TileShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t blocks = f8_blocks(p.q.cols);
  const int64_t rb = blockIdx.x / blocks, cb = blockIdx.x % blocks;
  const int64_t row0 = rb * kF8Block + warp * kF8Strip, col0 = cb * kF8Block, col = col0 + 4 * lane;
  const int rows = (int)(p.q.rows - row0 < kF8Strip ? p.q.rows - row0 : kF8Strip);  // (may be negative)
  grid_dep_wait();
  uint2 x[kF8Strip];
#pragma unroll
  for (int i = 0; i < kF8Strip; ++i)
    x[i] = i < rows ? ld_bf16x4(p.x + (row0 + i) * p.x_row, col, p.q.cols) : make_uint2(0, 0);
  uint32_t codes[4][4] = {};  // [column][quarter of the strip's rows]
  if constexpr (SQUARE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kF8Strip; ++i) m = max(m, bf16x4_amax(x[i]));
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) sh.amax[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, sh.amax[0][w]);
    const F8Scale s = f8_scale(m);
    if (threadIdx.x == 0) {
      p.q.scales[rb * p.q.scales_row + cb] = s.by;
      if (TRANSPOSED) p.t.scales[cb * p.t.scales_row + rb] = s.by;
    }
#pragma unroll
    for (int i = 0; i < kF8Strip; ++i) {
      const uint32_t c = f8_codes(bf2_widen(x[i].x), bf2_widen(x[i].y), s);
      if (i < rows) st_codes4(p.q.data + (row0 + i) * p.q.row_bytes, col, p.q.cols, c);
#pragma unroll
      for (int j = 0; j < 4; ++j) codes[j][i / 4] |= (c >> (8 * j) & 0xffu) << (8 * (i % 4));
    }
  } else {
    uint32_t am[kF8Strip], cm[4] = {};
#pragma unroll
    for (int i = 0; i < kF8Strip; ++i) {
      am[i] = bf16x4_amax(x[i]);
      cm[0] = max(cm[0], x[i].x << 16 & 0x7fff0000u);
      cm[1] = max(cm[1], x[i].x & 0x7fff0000u);
      cm[2] = max(cm[2], x[i].y << 16 & 0x7fff0000u);
      cm[3] = max(cm[3], x[i].y & 0x7fff0000u);
    }
    const StripScales s(am);
    s.store(p.q, row0, cb);
#pragma unroll
    for (int i = 0; i < kF8Strip; ++i) {
      const F8Scale si = s.of(i);
      if (i < rows)
        st_codes4(p.q.data + (row0 + i) * p.q.row_bytes, col, p.q.cols, f8_codes(bf2_widen(x[i].x), bf2_widen(x[i].y), si));
    }
    tile_column_scales(sh, cm, p.t, col0, rb);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const F8Scale sj = sh.scale[4 * lane + j];
      auto value = [&](int i) {
        const uint32_t w = j < 2 ? x[i].x : x[i].y;
        return j % 2 ? bf_hi(w) : bf_lo(w);
      };
#pragma unroll
      for (int k = 0; k < 4; ++k)
        codes[j][k] = f8_codes(f2_make(value(4 * k), value(4 * k + 1)), f2_make(value(4 * k + 2), value(4 * k + 3)), sj);
    }
  }
  if constexpr (TRANSPOSED) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      tile_piece(sh, 4 * lane + j, warp) = make_uint4(codes[j][0], codes[j][1], codes[j][2], codes[j][3]);
    __syncthreads();
    tile_store_transposed(sh, p.t, col0, rb * kF8Block);
  }
  grid_dep_launch_dependents();
}

// ---- and back -----------------------------------------------------------------------------

struct F8DequantizeParams {
  F8View q;
  uint16_t* x;
  int64_t x_row;
};

template <bool SQUARE>
__global__ void __launch_bounds__(kF8Threads) attn_res_f8_dequantize_kernel(const F8DequantizeParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t blocks = f8_blocks(p.q.cols);
  const int64_t job = (int64_t)blockIdx.x * (kF8Threads / 32) + (threadIdx.x >> 5);
  const int64_t row0 = job / blocks * kF8Strip, b = job % blocks;
  grid_dep_wait();
  if (row0 < p.q.rows) {
    const int64_t col = b * kF8Block + 4 * lane;
    const int rows = (int)(p.q.rows - row0 < kF8Strip ? p.q.rows - row0 : kF8Strip);
    uint32_t c[kF8Strip];
#pragma unroll
    for (int i = 0; i < kF8Strip; ++i)
      c[i] = i < rows ? ld_codes4(p.q.data + (row0 + i) * p.q.row_bytes, col, p.q.cols) : 0u;
    // (a strip lies in one block of rows)
    float s = 0.f;
    if (SQUARE) s = p.q.scales[row0 / kF8Block * p.q.scales_row + b];
    else if (lane < rows) s = p.q.scales[b * p.q.scales_row + row0 + lane];
#pragma unroll
    for (int i = 0; i < kF8Strip; ++i) {
      const float by = SQUARE ? s : __shfl_sync(0xffffffffu, s, i);
      const f32x2 lo = f2_mul(e4m3_pair(c[i]), f2_make(by, by)), hi = f2_mul(e4m3_pair(c[i] >> 16), f2_make(by, by));
      const uint32_t a = pack_bf16x2(f2_lo(lo), f2_hi(lo)), d = pack_bf16x2(f2_lo(hi), f2_hi(hi));
      if (i >= rows) continue;
      uint16_t* const o = p.x + (row0 + i) * p.x_row + col;
      if (col + 4 <= p.q.cols) {
        *reinterpret_cast<uint2*>(o) = make_uint2(a, d);
      } else {
        if (col < p.q.cols) o[0] = (uint16_t)a;
        if (col + 1 < p.q.cols) o[1] = (uint16_t)(a >> 16);
        if (col + 2 < p.q.cols) o[2] = (uint16_t)d;
      }
    }
  }
  grid_dep_launch_dependents();
}

// ---- backward pass of the gated block -----------------------------------------------------
//
// From h's gradient and the codes of both projections: dg = dh u act'(g), du =
// dh act(g), by rows and, for the gradients of the weights, transposed, with
// the transposed h = act(g) u.
//
// Nine bytes an element at the copy rate leave an SM some 45 instructions for
// one, and about as many are needed: a value is made once and stays in
// registers until both its scales are known (512 threads, 8 rows x 4 columns of
// a 128 x 128 tile each, 96 values), and codes are made with the scale's
// inverse.  That leaves room for one CTA an SM, so the CTAs are persistent and
// the next tile's inputs are brought in by TMA meanwhile.
constexpr int kF8BackThreads = 512;
constexpr int kF8BackRows = 8;  // of a warp

struct F8BackwardParams {
  F8View dg, du;           // by rows
  F8View dg_t, du_t, h_t;  // transposed
  int tiles, col_tiles;
  unsigned* err;
};
struct F8BackwardMaps {
  CUtensorMap dh, g, u, g_scales, u_scales;
};
// Shared memory: two stages of inputs, the transposed codes, amaxes and
// inverses of the columns' scales.
struct F8BackStage {
  uint16_t dh[128][128];
  uint8_t g[128][128], u[128][128];
  float g_scales[128], u_scales[128];
};
struct F8BackShared {
  F8BackStage stage[2];
  uint2 codes[3][128][16];  // [dg, du, h][column][8 rows], places mixed
  uint32_t amax[3][128];
  float inverse[3][128];
  unsigned long long full[2];
};

// The codes of four values with a scale's inverse (NaN: none).
__device__ __forceinline__ uint32_t codes_by(f32x2 a, f32x2 b) {
  return e4m3x4(f2_lo(a), f2_hi(a), f2_lo(b), f2_hi(b));
}

template <int ACT, bool TRANSPOSED>
__global__ void __launch_bounds__(kF8BackThreads, 1)
    attn_res_f8_gated_backward_kernel(const __grid_constant__ F8BackwardParams p,
                                      const __grid_constant__ F8BackwardMaps maps) {
  extern __shared__ __align__(128) uint8_t raw[];
  F8BackShared& sh = *reinterpret_cast<F8BackShared*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t full = smem_addr(sh.full);
  const int64_t rows = p.dg.rows, cols = p.dg.cols;
  auto load = [&](int tile, int s) {
    const int row0 = tile / p.col_tiles * 128, col0 = tile % p.col_tiles * 128;
    const uint32_t bar = full + 8 * s;
    F8BackStage& to = sh.stage[s];
    mbar_arrive_expect_tx(bar, sizeof(F8BackStage));
    tma_load_2d(smem_addr(to.dh), &maps.dh, col0, row0, bar);
    tma_load_2d(smem_addr(to.g), &maps.g, col0, row0, bar);
    tma_load_2d(smem_addr(to.u), &maps.u, col0, row0, bar);
    tma_load_2d(smem_addr(to.g_scales), &maps.g_scales, row0, col0 / 128, bar);
    tma_load_2d(smem_addr(to.u_scales), &maps.u_scales, row0, col0 / 128, bar);
  };
  if (threadIdx.x == 0) {
    mbar_init(full, 1);
    mbar_init(full + 8, 1);
    fence_mbar_init();
  }
  if (threadIdx.x < 3 * 128) sh.amax[threadIdx.x / 128][threadIdx.x % 128] = 0;
  grid_dep_wait();
  __syncthreads();
  const int first = blockIdx.x, step = gridDim.x;
  uint32_t issued = 0;  // thread 0's loads
  if (threadIdx.x == 0)
    for (int s = 0; s < 2 && first + s * step < p.tiles; ++s, ++issued) load(first + s * step, s);
  bool failed = false;
  uint32_t it = 0;
  for (int tile = first; tile < p.tiles; tile += step, ++it) {
    const int s = it & 1;
    const int64_t rb = tile / p.col_tiles, cb = tile % p.col_tiles;
    const int64_t row0 = rb * 128 + warp * kF8BackRows, col0 = cb * 128, col = col0 + 4 * lane;
    phase_or_flag(full + 8 * s, (it >> 1) & 1, failed, p.err, kErrStageTimeout);
    const F8BackStage& in = sh.stage[s];
    f32x2 dg[kF8BackRows][2], du[kF8BackRows][2], h[kF8BackRows][2];
    uint32_t am_g = 0, am_u = 0;  // lane i: of row row0 + i
#pragma unroll
    for (int i = 0; i < kF8BackRows; ++i) {
      const int r = warp * kF8BackRows + i;
      // (volatile: a row's inputs only when it is their turn, or registers run out)
      uint2 d;
      uint32_t gc, uc;
      float sg, su;
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(d.x), "=r"(d.y) : "r"(smem_addr(&in.dh[r][4 * lane])) : "memory");
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(gc) : "r"(smem_addr(&in.g[r][4 * lane])) : "memory");
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(uc) : "r"(smem_addr(&in.u[r][4 * lane])) : "memory");
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(sg) : "r"(smem_addr(&in.g_scales[r])) : "memory");
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(su) : "r"(smem_addr(&in.u_scales[r])) : "memory");
      uint32_t a = 0, b = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const f32x2 g = f2_mul(e4m3_pair(gc >> (16 * j)), f2_make(sg, sg));
        const f32x2 u = f2_mul(e4m3_pair(uc >> (16 * j)), f2_make(su, su));
        const f32x2 dh = bf2_widen(j ? d.y : d.x);
        f32x2 act, slope;
        f8_act_both2<ACT>(g, act, slope);
        du[i][j] = f2_mul(dh, act);
        dg[i][j] = f2_mul(f2_mul(dh, u), slope);
        h[i][j] = f2_mul(act, u);
        // (rows and columns behind the last were read as zeros: they count for
        // nothing where the row's scales are numbers, and where one is none the
        // row's values are none either)
        a = max(a, max(magnitude(f2_lo(dg[i][j])), magnitude(f2_hi(dg[i][j]))));
        b = max(b, max(magnitude(f2_lo(du[i][j])), magnitude(f2_hi(du[i][j]))));
      }
      a = __reduce_max_sync(0xffffffffu, a);
      b = __reduce_max_sync(0xffffffffu, b);
      if (lane == i) {
        am_g = a;
        am_u = b;
      }
    }
    if constexpr (TRANSPOSED) {
#pragma unroll
      for (int which = 0; which < 3; ++which)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t lo = 0, hi = 0;
#pragma unroll
          for (int i = 0; i < kF8BackRows; ++i) {
            const f32x2 v = which == 0 ? dg[i][j] : which == 1 ? du[i][j] : h[i][j];
            lo = max(lo, magnitude(f2_lo(v)));
            hi = max(hi, magnitude(f2_hi(v)));
          }
          atomicMax(&sh.amax[which][4 * lane + 2 * j], lo);
          atomicMax(&sh.amax[which][4 * lane + 2 * j + 1], hi);
        }
    }
    __syncthreads();  // the stage has been read, the columns' maxima are there
    if (threadIdx.x == 0 && tile + 2 * step < p.tiles && !failed) {
      load(tile + 2 * step, s);
      ++issued;
    }
    const F8Scale sg = f8_scale(am_g), su = f8_scale(am_u);
    if (TRANSPOSED && threadIdx.x < 3 * 128) {
      const int which = threadIdx.x / 128, c = threadIdx.x % 128;
      const F8Scale sc = f8_scale(sh.amax[which][c]);
      sh.inverse[which][c] = sc.inverse;
      sh.amax[which][c] = 0;
      const F8View& t = which == 0 ? p.dg_t : which == 1 ? p.du_t : p.h_t;
      if (col0 + c < cols && !failed) t.scales[rb * t.scales_row + col0 + c] = sc.by;
    }
    if (lane < kF8BackRows && row0 + lane < rows && !failed) {
      p.dg.scales[cb * p.dg.scales_row + row0 + lane] = sg.by;
      p.du.scales[cb * p.du.scales_row + row0 + lane] = su.by;
    }
#pragma unroll
    for (int i = 0; i < kF8BackRows; ++i) {
      const float ig = __shfl_sync(0xffffffffu, sg.inverse, i), iu = __shfl_sync(0xffffffffu, su.inverse, i);
      const f32x2 by_g = f2_make(ig, ig), by_u = f2_make(iu, iu);
      uint32_t a = codes_by(f2_mul(dg[i][0], by_g), f2_mul(dg[i][1], by_g));
      uint32_t b = codes_by(f2_mul(du[i][0], by_u), f2_mul(du[i][1], by_u));
      if (ig != ig) a = 0;
      if (iu != iu) b = 0;
      if (row0 + i < rows && !failed) {
        st_codes4(p.dg.data + (row0 + i) * p.dg.row_bytes, col, cols, a);
        st_codes4(p.du.data + (row0 + i) * p.du.row_bytes, col, cols, b);
      }
    }
    if constexpr (TRANSPOSED) {
      __syncthreads();  // the inverses are there; the codes of the tile before have left
#pragma unroll
      for (int which = 0; which < 3; ++which) {
        const float4 inv = *reinterpret_cast<const float4*>(&sh.inverse[which][4 * lane]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float i0 = j ? inv.z : inv.x, i1 = j ? inv.w : inv.y;
          const f32x2 by = f2_make(i0, i1);
          f32x2 v[kF8BackRows];
#pragma unroll
          for (int i = 0; i < kF8BackRows; ++i) v[i] = f2_mul(which == 0 ? dg[i][j] : which == 1 ? du[i][j] : h[i][j], by);
          uint2 lo, hi;
          lo.x = e4m3x4(f2_lo(v[0]), f2_lo(v[1]), f2_lo(v[2]), f2_lo(v[3]));
          lo.y = e4m3x4(f2_lo(v[4]), f2_lo(v[5]), f2_lo(v[6]), f2_lo(v[7]));
          hi.x = e4m3x4(f2_hi(v[0]), f2_hi(v[1]), f2_hi(v[2]), f2_hi(v[3]));
          hi.y = e4m3x4(f2_hi(v[4]), f2_hi(v[5]), f2_hi(v[6]), f2_hi(v[7]));
          if (i0 != i0) lo = make_uint2(0, 0);
          if (i1 != i1) hi = make_uint2(0, 0);
          // column c's piece of warp w at w ^ (c / 4 % 16): writes and reads
          // without bank conflicts
          sh.codes[which][4 * lane + 2 * j][warp ^ (lane & 15)] = lo;
          sh.codes[which][4 * lane + 2 * j + 1][warp ^ (lane & 15)] = hi;
        }
      }
      __syncthreads();
      const int64_t at0 = rb * 128;
      for (int i = threadIdx.x; i < 3 * 128 * 8; i += kF8BackThreads) {
        const int which = i / (128 * 8), c = i / 8 % 128, piece = i % 8;
        const int64_t at = at0 + 16 * piece;
        if (col0 + c >= cols || at >= rows || failed) continue;
        const int x = (c >> 2) & 15;
        const uint4 two = *reinterpret_cast<const uint4*>(&sh.codes[which][c][(2 * piece ^ x) & ~1]);
        const uint4 v = x & 1 ? make_uint4(two.z, two.w, two.x, two.y) : two;
        const F8View& t = which == 0 ? p.dg_t : which == 1 ? p.du_t : p.h_t;
        uint8_t* const o = t.data + (col0 + c) * t.row_bytes + at;
        if (at + 16 <= rows) {
          *reinterpret_cast<uint4*>(o) = v;
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (at + k < rows) o[k] = (uint8_t)(vword(v, k / 4) >> (8 * (k % 4)));
        }
      }
    }
  }
  if (failed)  // copies still in flight land before the CTA ends
    for (uint32_t b = issued > 2 ? issued - 2 : 0; b < issued; ++b) (void)phase_wait(full + 8 * (b & 1), (b >> 1) & 1);
  grid_dep_launch_dependents();
}

}  // namespace attn_res_dev
