// attn_res_f8_rows.cuh -- quantisation into 8 bits with scales for blocks of
// 128, its inverse, and the backward pass of the gated block.
#pragma once

#include "attn_res_f8.cuh"

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
// the transposed h = act(g) u.  Each value is needed for two scales and two
// codes: it is made twice, once for the maxima and once for the codes, from
// the inputs in registers.
struct F8BackwardParams {
  const uint16_t* dh;
  int64_t dh_row;
  F8View gate, up;
  F8View dg, du;          // by rows
  F8View dg_t, du_t, h_t;  // transposed; data null: none of the three
};

template <int ACT, bool TRANSPOSED>
__global__ void __launch_bounds__(kF8Threads) attn_res_f8_gated_backward_kernel(const F8BackwardParams p) {
  __shared__ TileShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t blocks = f8_blocks(p.gate.cols), cols = p.gate.cols;
  const int64_t rb = blockIdx.x / blocks, cb = blockIdx.x % blocks;
  const int64_t row0 = rb * kF8Block + warp * kF8Strip, col0 = cb * kF8Block, col = col0 + 4 * lane;
  const int rows = (int)(p.gate.rows - row0 < kF8Strip ? p.gate.rows - row0 : kF8Strip);
  grid_dep_wait();
  uint2 dh[kF8Strip];
  uint32_t g[kF8Strip], u[kF8Strip];
#pragma unroll
  for (int i = 0; i < kF8Strip; ++i) {
    const bool in = i < rows;
    dh[i] = in ? ld_bf16x4(p.dh + (row0 + i) * p.dh_row, col, cols) : make_uint2(0, 0);
    g[i] = in ? ld_codes4(p.gate.data + (row0 + i) * p.gate.row_bytes, col, cols) : 0u;
    u[i] = in ? ld_codes4(p.up.data + (row0 + i) * p.up.row_bytes, col, cols) : 0u;
  }
  float sg = 1.f, su = 1.f;  // of row row0 + lane
  if (lane < rows && lane < kF8Strip) {
    sg = p.gate.scales[cb * p.gate.scales_row + row0 + lane];
    su = p.up.scales[cb * p.up.scales_row + row0 + lane];
  }
  struct Four {
    float dg[4], du[4], h[4];
  };
  auto values = [&](int i) {
    const float by_g = __shfl_sync(0xffffffffu, sg, i), by_u = __shfl_sync(0xffffffffu, su, i);
    Four v;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const f32x2 gv = f2_mul(e4m3_pair(g[i] >> (16 * j)), f2_make(by_g, by_g));
      const f32x2 uv = f2_mul(e4m3_pair(u[i] >> (16 * j)), f2_make(by_u, by_u));
      const uint32_t d = j ? dh[i].y : dh[i].x;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float act, slope;
        f8_act_both<ACT>(k ? f2_hi(gv) : f2_lo(gv), act, slope);
        const float ue = k ? f2_hi(uv) : f2_lo(uv), de = k ? bf_hi(d) : bf_lo(d);
        const int e = 2 * j + k;
        // columns behind the last count for nothing, whatever a row's scale is
        const bool in = col + e < cols;
        v.dg[e] = in ? de * ue * slope : 0.f;
        v.du[e] = in ? de * act : 0.f;
        v.h[e] = in ? act * ue : 0.f;
      }
    }
    return v;
  };
  uint32_t rg[kF8Strip], ru[kF8Strip], cg[4] = {}, cu[4] = {}, ch[4] = {};
#pragma unroll
  for (int i = 0; i < kF8Strip; ++i) {
    const Four v = values(i);
    rg[i] = ru[i] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = magnitude(v.dg[j]), b = magnitude(v.du[j]);
      rg[i] = max(rg[i], a);
      ru[i] = max(ru[i], b);
      cg[j] = max(cg[j], a);
      cu[j] = max(cu[j], b);
      ch[j] = max(ch[j], magnitude(v.h[j]));
    }
  }
  const StripScales srg(rg), sru(ru);
  srg.store(p.dg, row0, cb);
  sru.store(p.du, row0, cb);
#pragma unroll
  for (int i = 0; i < kF8Strip; ++i) {
    const Four v = values(i);
    const F8Scale a = srg.of(i), b = sru.of(i);
    if (i < rows) {
      st_codes4(p.dg.data + (row0 + i) * p.dg.row_bytes, col, cols,
                f8_codes(f2_make(v.dg[0], v.dg[1]), f2_make(v.dg[2], v.dg[3]), a));
      st_codes4(p.du.data + (row0 + i) * p.du.row_bytes, col, cols,
                f8_codes(f2_make(v.du[0], v.du[1]), f2_make(v.du[2], v.du[3]), b));
    }
  }
  if constexpr (TRANSPOSED) {
#pragma unroll
    for (int which = 0; which < 3; ++which) {
      const F8View& t = which == 0 ? p.dg_t : which == 1 ? p.du_t : p.h_t;
      // (its first barrier: the piece before has been read)
      tile_column_scales(sh, which == 0 ? cg : which == 1 ? cu : ch, t, col0, rb);
      F8Scale s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = sh.scale[4 * lane + j];
      uint32_t codes[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v[4][4];  // [row][column]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Four f = values(4 * k + i);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = which == 0 ? f.dg[j] : which == 1 ? f.du[j] : f.h[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) codes[j][k] = f8_codes(f2_make(v[0][j], v[1][j]), f2_make(v[2][j], v[3][j]), s[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        tile_piece(sh, 4 * lane + j, warp) = make_uint4(codes[j][0], codes[j][1], codes[j][2], codes[j][3]);
      __syncthreads();
      tile_store_transposed(sh, t, col0, rb * kF8Block);
    }
  }
  grid_dep_launch_dependents();
}

}  // namespace attn_res_dev
