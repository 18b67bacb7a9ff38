// attn_res_f8_product.cu -- launches of the 8-bit products.
#include "attn_res_f8_host.cuh"
#include "attn_res_f8_product.cuh"
#include "attn_res_tensor_host.cuh"

namespace attn_res_host {
namespace {

using namespace attn_res_dev;

// Tensor map of an operand's codes: boxes of 128 bytes x `rows`, swizzled.
cudaError_t codes_map(const attn_res_f8_t& x, uint32_t rows, CUtensorMap* map) {
  return map_2d(CU_TENSOR_MAP_DATA_TYPE_UINT8, x.data, x.cols, x.rows, x.row_bytes, 128, rows,
                CU_TENSOR_MAP_SWIZZLE_128B, map);
}

F8View view(const attn_res_f8_t* q) {
  F8View v = {};
  if (q != nullptr) v = {static_cast<uint8_t*>(q->data), q->scales, q->row_bytes, q->scales_row, q->rows, q->cols};
  return v;
}

F8ProductParams params(const F8Call& c) {
  F8ProductParams p = {};
  p.a[0] = {c.a->scales, c.a->scales_row};
  p.w[0] = {c.w->scales, c.w->scales_row};
  if (c.a2 != nullptr) p.a[1] = {c.a2->scales, c.a2->scales_row};
  if (c.w2 != nullptr) p.w[1] = {c.w2->scales, c.w2->scales_row};
  p.blocks[0] = (int)f8_blocks(c.a->cols);
  p.blocks[1] = c.a2 != nullptr ? (int)f8_blocks(c.a2->cols) : 0;
  p.m = c.a->rows;
  p.n = c.w->rows;
  p.out = c.out;
  p.out_row = c.out_row;
  p.add = c.out_type == ATTN_RES_OUT_F32_ADD;
  p.h = view(c.h);
  p.g = view(c.g);
  p.u = view(c.u);
  p.err = c.err;
  return p;
}

// Every launch is a programmatic one: its start-up overlaps the end of a
// preceding kernel that lets its dependents start, and it waits for that kernel
// before it touches memory.
struct Attributes {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  Attributes(dim3 grid, int threads, uint32_t smem, unsigned cluster, cudaStream_t stream) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
  Attributes(const Attributes&) = delete;
};

template <int OUT, int ACT, bool ROWS_W>
struct Wide {
  using C = F8WideCfg;
  static constexpr auto kern = attn_res_f8_wide_kernel<OUT, ACT, ROWS_W>;

  // Pairs that the device holds at once.
  static cudaError_t resident(const F8Call& c, int* pairs) {
    static std::atomic<uint64_t> enabled{0};
    static std::atomic<int> known[64];
    *pairs = known[c.device].load(std::memory_order_acquire);
    if (*pairs != 0) return cudaSuccess;
    cudaError_t e = allow_smem(kern, C::SMEM, c.device, enabled);
    const Attributes l(dim3(2, 1, 1), C::THREADS, C::SMEM, 2, c.stream);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(pairs, kern, &l.cfg);
    if (e != cudaSuccess) return e;
    if (*pairs < 1) return cudaErrorInvalidConfiguration;
    known[c.device].store(*pairs, std::memory_order_release);
    return cudaSuccess;
  }
  static cudaError_t launch(const F8Call& c) {
    int pairs;
    cudaError_t e = resident(c, &pairs);
    F8ProductMaps maps = {};
    auto operands = [&](int t, const attn_res_f8_t* a, const attn_res_f8_t* w) {
      // (a term of width 0 has no blocks, and maps of nothing are none)
      if (e == cudaSuccess && a != nullptr && a->cols > 0) e = codes_map(*a, 128, &maps.a[t]);
      if (e == cudaSuccess && w != nullptr && w->cols > 0) e = codes_map(*w, 128, &maps.w[t]);
    };
    operands(0, c.a, c.w);
    operands(1, c.a2, c.w2);
    if (e != cudaSuccess) return e;
    const int64_t columns = c.gated ? 128 : C::TN;
    const int64_t m_tiles = (c.a->rows + C::TM - 1) / C::TM, n_tiles = (c.w->rows + columns - 1) / columns;
    const int64_t tiles = m_tiles * n_tiles;
    if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
    const TileWalk walk{(int)m_tiles, (int)n_tiles};
    Attributes l(dim3(2 * (unsigned)(tiles < pairs ? tiles : pairs), 1, 1), C::THREADS, C::SMEM, 2, c.stream);
    return cudaLaunchKernelEx(&l.cfg, kern, params(c), walk, maps);
  }
};

}  // namespace

cudaError_t launch_f8_product(const F8Call& c) {
  if (c.gated) {
    const bool silu = c.activation == ATTN_RES_SILU;
    if (c.out == nullptr)
      return silu ? Wide<kF8GatedCodes, ATTN_RES_SILU, false>::launch(c) : Wide<kF8GatedCodes, ATTN_RES_GELU, false>::launch(c);
    return silu ? Wide<kF8GatedBf16, ATTN_RES_SILU, false>::launch(c) : Wide<kF8GatedBf16, ATTN_RES_GELU, false>::launch(c);
  }
  const bool rows = c.w->block == ATTN_RES_F8_ROWS;
  if (c.out_type == ATTN_RES_OUT_BF16)
    return rows ? Wide<kF8OutBf16, 0, true>::launch(c) : Wide<kF8OutBf16, 0, false>::launch(c);
  return rows ? Wide<kF8OutF32, 0, true>::launch(c) : Wide<kF8OutF32, 0, false>::launch(c);
}

}  // namespace attn_res_host
