// attn_res_f8_rows.cuh -- quantisation into 8 bits with scales for blocks of
// 128, its inverse, and the backward pass of the gated block.
#pragma once

#include <type_traits>

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

// Most strips and tiles are whole: their code (WHOLE = 2) asks for no row or
// column (8192 x 7168 with both outputs 68 us when each access did), that of few
// rows of whole columns (1) for rows.  Addresses are a lane's first one and, for
// all lanes alike, rows times a stride.
//
// Four bf16 from `at` on, `left` columns before the row's last; zeros behind it,
// and where `in` is false.
template <int WHOLE>
__device__ __forceinline__ uint2 ld_bf16x4(const uint16_t* at, int64_t left, bool in = true) {
  if (WHOLE == 2 || (in && (WHOLE == 1 || left >= 4))) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(at));
    return v;
  }
  if (WHOLE == 1) return make_uint2(0, 0);
  uint32_t e[4] = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (in && k < left) e[k] = at[k];
  return make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
}
// Four codes.
template <int WHOLE>
__device__ __forceinline__ uint32_t ld_codes4(const uint8_t* at, int64_t left, bool in = true) {
  if (WHOLE == 2 || (in && (WHOLE == 1 || left >= 4))) return *reinterpret_cast<const uint32_t*>(at);
  if (WHOLE == 1) return 0u;
  uint32_t v = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (in && k < left) v |= (uint32_t)at[k] << (8 * k);
  return v;
}
template <int WHOLE>
__device__ __forceinline__ void st_codes4(uint8_t* at, int64_t left, uint32_t v, bool in = true) {
  if (WHOLE == 2 || (in && (WHOLE == 1 || left >= 4))) {
    *reinterpret_cast<uint32_t*>(at) = v;
  } else if (WHOLE == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (in && k < left) at[k] = (uint8_t)(v >> (8 * k));
  }
}
// f(integral constant).
template <class Fn>
__device__ __forceinline__ void with_whole(bool rows, bool cols, Fn f) {
  if (rows && cols) f(std::integral_constant<int, 2>());
  else if (cols) f(std::integral_constant<int, 1>());
  else f(std::integral_constant<int, 0>());
}

// The scales of the strip's rows from each lane's maxima over its columns: lane
// i makes that of row i, all lanes get them through shared memory.
struct StripScales {
  F8Scale mine;
  const F8Scale* all;
  __device__ __forceinline__ StripScales(const uint32_t (&amax)[kF8Strip], F8Scale (&shared)[kF8Strip]) : all(shared) {
    const int lane = threadIdx.x & 31;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kF8Strip; ++i) {
      const uint32_t r = __reduce_max_sync(0xffffffffu, amax[i]);
      if (lane == i) m = r;
    }
    mine = f8_scale(m);
    if (lane < kF8Strip) shared[lane] = mine;
    __syncwarp();
  }
  __device__ __forceinline__ bool held() const {
    return __all_sync(0xffffffffu, f8_quotients_held(mine.by) || (threadIdx.x & 31) >= kF8Strip);
  }
  // of rows i and i + 1 (i even): (by, inverse) twice
  __device__ __forceinline__ float4 two(int i) const { return *reinterpret_cast<const float4*>(&all[i]); }
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
  __align__(16) F8Scale scale[128];
  __align__(16) F8Scale row_scale[8][kF8Strip];
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
template <bool WHOLE>
__device__ __forceinline__ void tile_store_transposed(TileShared& t, const F8View& qt, int64_t col0, int64_t row0) {
  constexpr int STEP = kF8Threads / 8;  // columns
  const int c0 = threadIdx.x / 8, piece = threadIdx.x % 8;
  const int64_t at = row0 + 16 * piece;
  uint8_t* const first = qt.data + (col0 + c0) * qt.row_bytes + at;
#pragma unroll
  for (int k = 0; k < 128 / STEP; ++k) {
    const int c = c0 + STEP * k;
    uint8_t* const o = first + k * STEP * qt.row_bytes;
    if (WHOLE || (col0 + c < qt.rows && at + 16 <= qt.cols)) {
      *reinterpret_cast<uint4*>(o) = tile_piece(t, c, piece);
    } else if (col0 + c < qt.rows) {
      const uint4 v = tile_piece(t, c, piece);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (at + e < qt.cols) o[e] = (uint8_t)(vword(v, e / 4) >> (8 * (e % 4)));
    }
  }
}

// ---- quantisation -------------------------------------------------------------------------

struct F8QuantizeParams {
  const uint16_t* x;
  int64_t x_row;
  F8View q, t;  // t: the transposed matrix (the tile kernel)
};

// The largest of two bf16 magnitudes as fp32 bits, of a pair and of four values.
__device__ __forceinline__ uint32_t pair_amax(uint32_t m) { return max(m << 16, m & 0xffff0000u); }
__device__ __forceinline__ uint2 magnitudes(uint2 v) { return make_uint2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t bf16x4_amax(uint2 v) {
  const uint2 m = magnitudes(v);
  return pair_amax(__vmaxu2(m.x, m.y));
}

// A strip again, from memory, whose quotients want the division itself: rows with
// scales outside 2^-96 .. 2^96 or without one.  (In the strip's own way its code
// would lie between that of every four codes: 8192 x 7168 29.1 us instead of 27.6.)
__device__ __noinline__ void far_strip(const F8QuantizeParams& p, int64_t row0, int64_t b) {
  const int lane = threadIdx.x & 31;
  const int64_t col = b * kF8Block + 4 * lane, left = p.q.cols - col;
#pragma unroll 1
  for (int64_t row = row0; row < row0 + kF8Strip && row < p.q.rows; ++row) {
    const uint2 x = ld_bf16x4<0>(p.x + row * p.x_row + col, left);
    const F8Scale s = f8_scale(__reduce_max_sync(0xffffffffu, bf16x4_amax(x)));
    st_codes4<0>(p.q.data + row * p.q.row_bytes + col, left, f8_codes_far(bf2_widen(x.x), bf2_widen(x.y), s.by));
  }
}

// Rows only: a warp a strip.
__global__ void __launch_bounds__(kF8Threads) attn_res_f8_quantize_rows_kernel(const __grid_constant__ F8QuantizeParams p) {
  __shared__ __align__(16) F8Scale scale[kF8Threads / 32][kF8Strip];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t blocks = f8_blocks(p.q.cols);
  const int64_t job = (int64_t)blockIdx.x * (kF8Threads / 32) + warp;
  const int64_t row0 = job / blocks * kF8Strip, b = job % blocks;
  grid_dep_wait();
  if (row0 < p.q.rows) {
    const int64_t col = b * kF8Block + 4 * lane, left = p.q.cols - col;
    const int rows = (int)(p.q.rows - row0 < kF8Strip ? p.q.rows - row0 : kF8Strip);
    const uint16_t* const from = p.x + row0 * p.x_row + col;
    uint8_t* const to = p.q.data + row0 * p.q.row_bytes + col;
    with_whole(rows == kF8Strip, (b + 1) * kF8Block <= p.q.cols, [&](auto whole) {
      constexpr int W = decltype(whole)::value;
      uint2 x[kF8Strip];
      uint32_t am[kF8Strip];
#pragma unroll
      for (int i = 0; i < kF8Strip; ++i) x[i] = ld_bf16x4<W>(from + i * p.x_row, left, i < rows);
#pragma unroll
      for (int i = 0; i < kF8Strip; ++i) am[i] = bf16x4_amax(x[i]);
      const StripScales s(am, scale[warp]);
      s.store(p.q, row0, b);
      if (s.held()) {
#pragma unroll
        for (int i = 0; i < kF8Strip; i += 2) {
          const float4 si = s.two(i);
          st_codes4<W>(to + i * p.q.row_bytes, left, f8_codes(bf2_widen(x[i].x), bf2_widen(x[i].y), si.x, si.y), i < rows);
          st_codes4<W>(to + (i + 1) * p.q.row_bytes, left,
                       f8_codes(bf2_widen(x[i + 1].x), bf2_widen(x[i + 1].y), si.z, si.w), i + 1 < rows);
        }
      } else {
        far_strip(p, row0, b);
      }
    });
  }
  grid_dep_launch_dependents();
}

// Columns' codes of four rows (their quotients in pairs of columns, negated), the
// first row lowest.
__device__ __forceinline__ uint32_t codes_lo(const f32x2 (&v)[4]) {
  return e4m3x4(f2_lo(v[0]), f2_lo(v[1]), f2_lo(v[2]), f2_lo(v[3])) ^ 0x80808080u;
}
__device__ __forceinline__ uint32_t codes_hi(const f32x2 (&v)[4]) {
  return e4m3x4(f2_hi(v[0]), f2_hi(v[1]), f2_hi(v[2]), f2_hi(v[3])) ^ 0x80808080u;
}

// Tiles: block scales (SQUARE), or row scales with the transposed matrix too;
// TRANSPOSED: the transposed matrix.
template <bool SQUARE, bool TRANSPOSED>
__global__ void __launch_bounds__(kF8Threads, 4) attn_res_f8_quantize_tile_kernel(const __grid_constant__ F8QuantizeParams p) {
  __shared__ TileShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t blocks = f8_blocks(p.q.cols);
  const int64_t rb = blockIdx.x / blocks, cb = blockIdx.x % blocks;
  const int64_t row0 = rb * kF8Block + warp * kF8Strip, col0 = cb * kF8Block, col = col0 + 4 * lane, left = p.q.cols - col;
  const int rows = (int)(p.q.rows - row0 < kF8Strip ? p.q.rows - row0 : kF8Strip);  // (may be negative)
  const uint16_t* const from = p.x + row0 * p.x_row + col;
  uint8_t* const to = p.q.data + row0 * p.q.row_bytes + col;
  grid_dep_wait();
  with_whole((rb + 1) * kF8Block <= p.q.rows, col0 + kF8Block <= p.q.cols, [&](auto whole) {
    constexpr int W = decltype(whole)::value;
    uint2 x[kF8Strip];
#pragma unroll
    for (int i = 0; i < kF8Strip; ++i) x[i] = ld_bf16x4<W>(from + i * p.x_row, left, i < rows);
    if constexpr (SQUARE) {
      uint2 m2 = make_uint2(0, 0);
#pragma unroll
      for (int i = 0; i < kF8Strip; ++i) {
        const uint2 m = magnitudes(x[i]);
        m2 = make_uint2(__vmaxu2(m2.x, m.x), __vmaxu2(m2.y, m.y));
      }
      uint32_t m = __reduce_max_sync(0xffffffffu, pair_amax(__vmaxu2(m2.x, m2.y)));
      if (lane == 0) sh.amax[0][warp] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 8; ++w) m = max(m, sh.amax[0][w]);
      const F8Scale s = f8_scale(m);
      if (threadIdx.x == 0) {
        p.q.scales[rb * p.q.scales_row + cb] = s.by;
        if (TRANSPOSED) p.t.scales[cb * p.t.scales_row + rb] = s.by;
      }
      auto encode = [&](auto far) {
        [[maybe_unused]] uint32_t codes[4][4] = {};  // [column][quarter of the strip's rows]
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t c[4];  // of four rows, turned into those of four columns
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint2 v = x[4 * k + i];
            c[i] = decltype(far)::value ? f8_codes_far(bf2_widen(v.x), bf2_widen(v.y), s.by)
                                        : f8_codes(bf2_widen(v.x), bf2_widen(v.y), s.by, s.inverse);
            st_codes4<W>(to + (4 * k + i) * p.q.row_bytes, left, c[i], 4 * k + i < rows);
          }
          if constexpr (TRANSPOSED) {
            const uint32_t a = __byte_perm(c[0], c[1], 0x5140), b = __byte_perm(c[2], c[3], 0x5140);
            const uint32_t d = __byte_perm(c[0], c[1], 0x7362), e = __byte_perm(c[2], c[3], 0x7362);
            codes[0][k] = __byte_perm(a, b, 0x5410);
            codes[1][k] = __byte_perm(a, b, 0x7632);
            codes[2][k] = __byte_perm(d, e, 0x5410);
            codes[3][k] = __byte_perm(d, e, 0x7632);
          }
        }
        if constexpr (TRANSPOSED)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tile_piece(sh, 4 * lane + j, warp) = make_uint4(codes[j][0], codes[j][1], codes[j][2], codes[j][3]);
      };
      if (f8_quotients_held(s.by)) encode(std::false_type());
      else encode(std::true_type());
    } else {
      uint32_t am[kF8Strip], cm2[2] = {};
#pragma unroll
      for (int i = 0; i < kF8Strip; ++i) {
        const uint2 m = magnitudes(x[i]);
        am[i] = pair_amax(__vmaxu2(m.x, m.y));
        cm2[0] = __vmaxu2(cm2[0], m.x);
        cm2[1] = __vmaxu2(cm2[1], m.y);
      }
      const uint32_t cm[4] = {cm2[0] << 16, cm2[0] & 0xffff0000u, cm2[1] << 16, cm2[1] & 0xffff0000u};
      const StripScales s(am, sh.row_scale[warp]);
      s.store(p.q, row0, cb);
      tile_column_scales(sh, cm, p.t, col0, rb);
      const float4* const scale = reinterpret_cast<const float4*>(&sh.scale[4 * lane]);  // (by, inverse) of two columns each
      const float4 s01 = scale[0], s23 = scale[1];
      const bool held = s.held();
      if (held && __all_sync(0xffffffffu, f8_quotients_held(s01.x) && f8_quotients_held(s01.z) &&
                                              f8_quotients_held(s23.x) && f8_quotients_held(s23.z))) {
        const f32x2 by0 = f2_make(s01.x, s01.z), by1 = f2_make(s23.x, s23.z);
        const f32x2 minus0 = f2_make(-s01.y, -s01.w), minus1 = f2_make(-s23.y, -s23.w);
        uint32_t codes[4][4];  // [column][quarter of the strip's rows]
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f32x2 c0[4], c1[4];  // columns' quotients, negated
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 4 * k + e;
            const f32x2 lo = bf2_widen(x[i].x), hi = bf2_widen(x[i].y);
            const float4 two = s.two(i & ~1);
            st_codes4<W>(to + i * p.q.row_bytes, left,
                         f8_codes(lo, hi, e % 2 ? two.z : two.x, e % 2 ? two.w : two.y), i < rows);
            c0[e] = f8_negated_quotient2(lo, by0, minus0);
            c1[e] = f8_negated_quotient2(hi, by1, minus1);
          }
          codes[0][k] = codes_lo(c0);
          codes[1][k] = codes_hi(c0);
          codes[2][k] = codes_lo(c1);
          codes[3][k] = codes_hi(c1);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          tile_piece(sh, 4 * lane + j, warp) = make_uint4(codes[j][0], codes[j][1], codes[j][2], codes[j][3]);
      } else {
        far_strip(p, row0, cb);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float by = j == 0 ? s01.x : j == 1 ? s01.z : j == 2 ? s23.x : s23.z;
          auto value = [&](int i) {
            const uint32_t w = j < 2 ? x[i].x : x[i].y;
            return j % 2 ? bf_hi(w) : bf_lo(w);
          };
          uint32_t codes[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            codes[k] = f8_codes_far(f2_make(value(4 * k), value(4 * k + 1)), f2_make(value(4 * k + 2), value(4 * k + 3)), by);
          tile_piece(sh, 4 * lane + j, warp) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
        }
      }
    }
    if constexpr (TRANSPOSED) {
      __syncthreads();
      tile_store_transposed<W == 2>(sh, p.t, col0, rb * kF8Block);
    }
  });
  grid_dep_launch_dependents();
}

// ---- and back -----------------------------------------------------------------------------

struct F8DequantizeParams {
  F8View q;
  uint16_t* x;
  int64_t x_row;
};

template <bool SQUARE>
__global__ void __launch_bounds__(kF8Threads) attn_res_f8_dequantize_kernel(const __grid_constant__ F8DequantizeParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t blocks = f8_blocks(p.q.cols);
  const int64_t job = (int64_t)blockIdx.x * (kF8Threads / 32) + (threadIdx.x >> 5);
  const int64_t row0 = job / blocks * kF8Strip, b = job % blocks;
  grid_dep_wait();
  if (row0 < p.q.rows) {
    const int64_t col = b * kF8Block + 4 * lane, left = p.q.cols - col;
    const int rows = (int)(p.q.rows - row0 < kF8Strip ? p.q.rows - row0 : kF8Strip);
    const uint8_t* const from = p.q.data + row0 * p.q.row_bytes + col;
    uint16_t* const to = p.x + row0 * p.x_row + col;
    with_whole(rows == kF8Strip, (b + 1) * kF8Block <= p.q.cols, [&](auto whole) {
      constexpr int W = decltype(whole)::value;
      uint32_t c[kF8Strip];
#pragma unroll
      for (int i = 0; i < kF8Strip; ++i) c[i] = ld_codes4<W>(from + i * p.q.row_bytes, left, i < rows);
      // (a strip lies in one block of rows)
      float s = 0.f;
      if (SQUARE) s = p.q.scales[row0 / kF8Block * p.q.scales_row + b];
      else if (lane < rows) s = p.q.scales[b * p.q.scales_row + row0 + lane];
#pragma unroll
      for (int i = 0; i < kF8Strip; ++i) {
        const float by = SQUARE ? s : __shfl_sync(0xffffffffu, s, i);
        const f32x2 lo = f2_mul(e4m3_pair(c[i]), f2_make(by, by)), hi = f2_mul(e4m3_pair(c[i] >> 16), f2_make(by, by));
        const uint32_t a = pack_bf16x2(f2_lo(lo), f2_hi(lo)), d = pack_bf16x2(f2_lo(hi), f2_hi(hi));
        uint16_t* const o = to + i * p.x_row;
        if (W == 2 || (i < rows && (W == 1 || left >= 4))) {
          *reinterpret_cast<uint2*>(o) = make_uint2(a, d);
        } else if (W == 0 && i < rows) {
          if (left > 0) o[0] = (uint16_t)a;
          if (left > 1) o[1] = (uint16_t)(a >> 16);
          if (left > 2) o[2] = (uint16_t)d;
        }
      }
    });
  }
  grid_dep_launch_dependents();
}

// ---- backward pass of the gated block -----------------------------------------------------
//
// From h's gradient and the codes of both projections: dg = dh u act'(g), du =
// dh act(g), by rows and, for the gradients of the weights, transposed, with
// the transposed h = act(g) u.
//
// Four bytes an element are read and five written: 45.5 us at the copy rate for
// 8192 x 4096, where the kernel takes 87 (GELU 91; the rows alone, six bytes, 49).
// What is left is arithmetic: some 50 instructions an element in 16 warps an SM,
// each a chain of dependent ones.  A value is made once and stays in registers
// until both its scales are known (512 threads, 8 rows x 4 columns of a 128 x 128
// tile each, 96 values), and codes are made with the scale's inverse: such a
// product is off by 2^-23 of itself, less than the values are.  That leaves room
// for one CTA an SM, so the CTAs are persistent and the next tile's inputs are
// brought in by TMA meanwhile.  (With a CTA a tile, quotients and values made
// twice it took 763 us; persistent, 105; whole tiles by themselves, 90.)
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
  float column_inverse[3][128];
  float2 inverse[16][kF8BackRows];  // of a warp's rows, dg's and du's
  unsigned long long full[2];
};

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
      float a = 0.f, b = 0.f;
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
        a = amax3(a, dg[i][j]);
        b = amax3(b, du[i][j]);
      }
      a = warp_amax(a);
      b = warp_amax(b);
      if (lane == i) {
        am_g = __float_as_uint(a);
        am_u = __float_as_uint(b);
      }
    }
    if constexpr (TRANSPOSED) {
#pragma unroll
      for (int which = 0; which < 3; ++which)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float lo = 0.f, hi = 0.f;
#pragma unroll
          for (int i = 0; i < kF8BackRows; i += 2) {
            const f32x2 v = which == 0 ? dg[i][j] : which == 1 ? du[i][j] : h[i][j];
            const f32x2 w = which == 0 ? dg[i + 1][j] : which == 1 ? du[i + 1][j] : h[i + 1][j];
            lo = amax3(lo, f2_lo(v), f2_lo(w));
            hi = amax3(hi, f2_hi(v), f2_hi(w));
          }
          atomicMax(&sh.amax[which][4 * lane + 2 * j], __float_as_uint(lo));
          atomicMax(&sh.amax[which][4 * lane + 2 * j + 1], __float_as_uint(hi));
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
      sh.column_inverse[which][c] = sc.inverse;
      sh.amax[which][c] = 0;
      const F8View& t = which == 0 ? p.dg_t : which == 1 ? p.du_t : p.h_t;
      if (col0 + c < cols && !failed) t.scales[rb * t.scales_row + col0 + c] = sc.by;
    }
    if (lane < kF8BackRows && row0 + lane < rows && !failed) {
      p.dg.scales[cb * p.dg.scales_row + row0 + lane] = sg.by;
      p.du.scales[cb * p.du.scales_row + row0 + lane] = su.by;
    }
    uint8_t* const to_g = p.dg.data + row0 * p.dg.row_bytes + col;
    uint8_t* const to_u = p.du.data + row0 * p.du.row_bytes + col;
    const bool whole = (rb + 1) * 128 <= rows && col0 + 128 <= cols && !failed;
    if (lane < kF8BackRows) sh.inverse[warp][lane] = make_float2(sg.inverse, su.inverse);
    __syncwarp();
    const bool no_number = __any_sync(0xffffffffu, sg.by != sg.by || su.by != su.by);
#pragma unroll
    for (int i = 0; i < kF8BackRows; ++i) {
      const float2 inv = sh.inverse[warp][i];
      const f32x2 by_g = f2_make(inv.x, inv.x), by_u = f2_make(inv.y, inv.y);
      uint32_t a = codes_by(f2_mul(dg[i][0], by_g), f2_mul(dg[i][1], by_g));
      uint32_t b = codes_by(f2_mul(du[i][0], by_u), f2_mul(du[i][1], by_u));
      if (no_number) {
        if (inv.x != inv.x) a = 0;
        if (inv.y != inv.y) b = 0;
      }
      if (whole) {
        *reinterpret_cast<uint32_t*>(to_g + i * p.dg.row_bytes) = a;
        *reinterpret_cast<uint32_t*>(to_u + i * p.du.row_bytes) = b;
      } else if (row0 + i < rows && !failed) {
        st_codes4<0>(to_g + i * p.dg.row_bytes, cols - col, a);
        st_codes4<0>(to_u + i * p.du.row_bytes, cols - col, b);
      }
    }
    if constexpr (TRANSPOSED) {
      __syncthreads();  // the inverses are there; the codes of the tile before have left
#pragma unroll
      for (int which = 0; which < 3; ++which) {
        const float4 inv = *reinterpret_cast<const float4*>(&sh.column_inverse[which][4 * lane]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const f32x2 by = j ? f2_make(inv.z, inv.w) : f2_make(inv.x, inv.y);
          f32x2 v[kF8BackRows];
#pragma unroll
          for (int i = 0; i < kF8BackRows; ++i) v[i] = f2_mul(which == 0 ? dg[i][j] : which == 1 ? du[i][j] : h[i][j], by);
          uint2 lo, hi;
          lo.x = e4m3x4(f2_lo(v[0]), f2_lo(v[1]), f2_lo(v[2]), f2_lo(v[3]));
          lo.y = e4m3x4(f2_lo(v[4]), f2_lo(v[5]), f2_lo(v[6]), f2_lo(v[7]));
          hi.x = e4m3x4(f2_hi(v[0]), f2_hi(v[1]), f2_hi(v[2]), f2_hi(v[3]));
          hi.y = e4m3x4(f2_hi(v[4]), f2_hi(v[5]), f2_hi(v[6]), f2_hi(v[7]));
          const float sum = f2_lo(by) + f2_hi(by);
          if (sum != sum) {  // a column without a scale
            if (f2_lo(by) != f2_lo(by)) lo = make_uint2(0, 0);
            if (f2_hi(by) != f2_hi(by)) hi = make_uint2(0, 0);
          }
          // column c's piece of warp w at w ^ (c / 4 % 16): writes and reads
          // without bank conflicts
          sh.codes[which][4 * lane + 2 * j][warp ^ (lane & 15)] = lo;
          sh.codes[which][4 * lane + 2 * j + 1][warp ^ (lane & 15)] = hi;
        }
      }
      __syncthreads();
      const int c0 = threadIdx.x / 8, piece = threadIdx.x % 8, x = (c0 >> 2) & 15;
      const int64_t at = rb * 128 + 16 * piece;
#pragma unroll
      for (int which = 0; which < 3; ++which) {
        const F8View& t = which == 0 ? p.dg_t : which == 1 ? p.du_t : p.h_t;
        uint8_t* const first = t.data + (col0 + c0) * t.row_bytes + at;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int c = c0 + 64 * k;  // (which leaves x as it is)
          const uint4 two = *reinterpret_cast<const uint4*>(&sh.codes[which][c][(2 * piece ^ x) & ~1]);
          const uint4 v = x & 1 ? make_uint4(two.z, two.w, two.x, two.y) : two;
          uint8_t* const o = first + 64 * k * t.row_bytes;
          if (whole || (col0 + c < cols && at + 16 <= rows && !failed)) {
            *reinterpret_cast<uint4*>(o) = v;
          } else if (col0 + c < cols && !failed) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (at + e < rows) o[e] = (uint8_t)(vword(v, e / 4) >> (8 * (e % 4)));
          }
        }
      }
    }
  }
  if (failed)  // copies still in flight land before the CTA ends
    for (uint32_t b = issued > 2 ? issued - 2 : 0; b < issued; ++b) (void)phase_wait(full + 8 * (b & 1), (b >> 1) & 1);
  grid_dep_launch_dependents();
}

}  // namespace attn_res_dev
