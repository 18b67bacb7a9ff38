// f8_binding.cpp -- Python binding of the 8-bit entry points (attn_res_f8_* of
// include/attn_res.h): argument marshalling only, compiled as the microscaled
// entry points' is.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "binding.h"

namespace {

using namespace attn_res_binding;

int64_t blocks(int64_t n) { return (n + 127) / 128; }

void check_block(int block) {
  if (block != ATTN_RES_F8_ROWS && block != ATTN_RES_F8_SQUARE) refuse("block must be 1 or 128");
}
std::array<int64_t, 2> scales_shape(int64_t rows, int64_t cols, int block) {
  if (block == ATTN_RES_F8_ROWS) return {blocks(cols), rows};
  return {blocks(rows), blocks(cols)};
}

// As with the microscaled matrices, addresses, strides and sizes are taken, and
// the parts checked, at each call.
struct F8Tensor {
  at::Tensor data, scales;
  int block;

  int64_t rows() const { return data.sizes().at(0); }
  int64_t cols() const { return data.sizes().at(1); }
  at::Device device() const { return data.device(); }

  void check() const {
    const at::IntArrayRef size = data.sizes();
    if (data.scalar_type() != at::kFloat8_e4m3fn || size.size() != 2 || !data.is_cuda() ||
        (data.strides()[1] != 1 && size[1] > 1))
      refuse("data must be a CUDA float8_e4m3fn matrix with unit inner stride");
    const auto shape = scales_shape(size[0], size[1], block);
    if (scales.scalar_type() != at::kFloat || scales.device() != data.device() ||
        scales.sizes() != at::IntArrayRef(shape) || (scales.strides()[1] != 1 && shape[1] > 1))
      refuse("scales must be a float32 matrix of scales_shape(rows, cols, block) with unit inner stride beside data");
  }

  attn_res_f8_t matrix() const {
    check();
    attn_res_f8_t c = {};
    c.block = block;
    c.rows = rows();
    c.cols = cols();
    c.data = address("data", data);
    c.row_bytes = row_stride(data, 16);
    c.scales = static_cast<float*>(address("scales", scales));
    c.scales_row = row_stride(scales, 4);
    return c;
  }
};

F8Tensor make(const at::Tensor& data, const at::Tensor& scales, int block) {
  check_block(block);
  F8Tensor t{data, scales, block};
  t.check();
  return t;
}

// Rows of codes a multiple of 16 bytes apart, rows of scales of 16 bytes too (the
// last row without its padding, which nothing touches).
at::Tensor padded(int64_t rows, int64_t cols, int64_t to, at::ScalarType type, at::Device device) {
  const int64_t size[2] = {rows, cols}, stride[2] = {(cols + to - 1) / to * to, 1};
  return at::detail::empty_strided_cuda(size, stride, type, device);
}
F8Tensor allocate(int64_t rows, int64_t cols, int block, at::Device device) {
  const auto s = scales_shape(rows, cols, block);
  return {padded(rows, cols, 16, at::kFloat8_e4m3fn, device), padded(s[0], s[1], 4, at::kFloat, device), block};
}

// A result: `out`, checked, or a new one where it is None or True.
struct Result {
  py::object object;
  attn_res_f8_t c;
  Result(const char* name, const py::object& out, int64_t rows, int64_t cols, int block, at::Device device) {
    if (out.is_none() || out.ptr() == Py_True) {
      object = py::cast(allocate(rows, cols, block, device));
    } else {
      if (!py::isinstance<F8Tensor>(out)) refuse(std::string(name) + " must be an F8Tensor");
      const F8Tensor& o = out.cast<const F8Tensor&>();
      if (o.block != block || o.device() != device || o.data.dim() != 2 || o.rows() != rows || o.cols() != cols)
        refuse(std::string(name) + " must be an F8Tensor of [" + std::to_string(rows) + ", " + std::to_string(cols) +
               "] with block " + std::to_string(block) + " on the inputs' device");
      object = out;
    }
    c = object.cast<const F8Tensor&>().matrix();
  }
};

void same_device(at::Device device, const F8Tensor& t) {
  if (t.device() != device) refuse("all tensors of a call must be on one device");
}
bool wanted(const py::object& o) { return !o.is_none() && o.ptr() != Py_False; }

// n outputs, given as a sequence or (None, True) to be made.
std::vector<py::object> outputs(const char* name, const py::object& given, size_t n) {
  std::vector<py::object> v(n, py::none());
  if (given.is_none() || given.ptr() == Py_True) return v;
  if (!py::isinstance<py::sequence>(given) || py::len(given) != n)
    refuse(std::string(name) + " must be " + std::to_string(n) + " F8Tensors");
  for (size_t i = 0; i < n; ++i) v[i] = given.cast<py::sequence>()[i];
  return v;
}

uint32_t flags_of(bool pdl, int kernel, int split) {
  if (kernel < 0 || kernel > 15 || split < 0 || split > 255) refuse("no such kernel or split");
  return attn_res_binding::flags_of(pdl) | ATTN_RES_FLAG_KERNEL(kernel) | ATTN_RES_FLAG_SPLIT(split);
}

int activation_code(const std::string& a) {
  if (a == "silu") return ATTN_RES_SILU;
  if (a == "gelu") return ATTN_RES_GELU;
  refuse("activation must be silu or gelu");
}

at::ScalarType dtype_of(const py::object& o) {
  if (!THPDtype_Check(o.ptr())) refuse("dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o.ptr())->scalar_type;
}

py::object quantize(const at::Tensor& x, int block, const py::object& out, const py::object& transposed, bool pdl,
                    const py::object& stream) {
  check_rows("x", x);
  check_block(block);
  const int64_t rows = x.size(0), cols = x.size(1);
  const On on(x.device(), stream);
  const Result q("out", out, rows, cols, block, x.device());
  if (!wanted(transposed)) {
    check(attn_res_f8_quantize(bf16("x", x), row_stride(x, 8), &q.c, nullptr, attn_res_binding::flags_of(pdl), on.handle));
    return q.object;
  }
  const Result t("transposed", transposed, cols, rows, block, x.device());
  check(attn_res_f8_quantize(bf16("x", x), row_stride(x, 8), &q.c, &t.c, attn_res_binding::flags_of(pdl), on.handle));
  return py::make_tuple(q.object, t.object);
}

at::Tensor dequantize(const F8Tensor& q, const OptTensor& out, bool pdl, const py::object& stream) {
  const attn_res_f8_t c = q.matrix();
  const On on(q.device(), stream);
  if (out) check_rows("out", *out, c.rows, c.cols, q.device());
  const at::Tensor x = out ? *out : padded(c.rows, c.cols, 8, at::kBFloat16, q.device());
  check(attn_res_f8_dequantize(&c, bf16("out", x), row_stride(x, 8), attn_res_binding::flags_of(pdl), on.handle));
  return x;
}

at::Tensor matmul(const F8Tensor& a, const F8Tensor& w, const OptTensor& out, const py::object& dtype, bool add,
                  const std::optional<std::tuple<F8Tensor, F8Tensor>>& plus, bool pdl, int kernel, int split,
                  const py::object& stream) {
  const at::Device device = a.device();
  same_device(device, w);
  const attn_res_f8_t ca = a.matrix(), cw = w.matrix();
  if (ca.block != ATTN_RES_F8_ROWS) refuse("a must have a scale for each row (block 1)");
  if (ca.cols != cw.cols) refuse("a and w must have one width");
  attn_res_f8_t ca2 = {}, cw2 = {};
  if (plus) {
    same_device(device, std::get<0>(*plus));
    same_device(device, std::get<1>(*plus));
    ca2 = std::get<0>(*plus).matrix();
    cw2 = std::get<1>(*plus).matrix();
    if (ca2.block != ca.block || cw2.block != cw.block || ca2.rows != ca.rows || cw2.rows != cw.rows ||
        ca2.cols != cw2.cols)
      refuse("plus must have the rows and blocks of a and w, and one width");
  }
  const at::ScalarType type = out && dtype.is_none() ? out->scalar_type()
                              : dtype.is_none()      ? at::kBFloat16
                                                     : dtype_of(dtype);
  if (type != at::kBFloat16 && type != at::kFloat) refuse("the result is bfloat16 or float32");
  if (add && (!out || type != at::kFloat)) refuse("add needs a float32 out");
  const int64_t m = ca.rows, n = cw.rows, to = type == at::kFloat ? 4 : 8;
  const On on(device, stream);
  at::Tensor y;
  if (out) {
    y = *out;
    if (!y.is_cuda() || y.device() != device || y.scalar_type() != type || y.dim() != 2 || y.size(0) != m ||
        y.size(1) != n || (y.stride(1) != 1 && n > 1))
      refuse(std::string("out must be a ") + c10::toString(type) + " [" + std::to_string(m) + ", " + std::to_string(n) +
             "] matrix with unit inner stride beside a");
  } else {
    // rows start on 16-byte boundaries, whatever n; where they are padded
    // anyway, on 32-byte ones (whole sectors are then stored)
    y = padded(m, n, n % to == 0 ? to : 2 * to, type, device);
  }
  check(attn_res_f8_matmul(&ca, &cw, plus ? &ca2 : nullptr, plus ? &cw2 : nullptr, address("out", y), row_stride(y, to),
                           type == at::kBFloat16 ? ATTN_RES_OUT_BF16 : add ? ATTN_RES_OUT_F32_ADD : ATTN_RES_OUT_F32,
                           flags_of(pdl, kernel, split), on.handle));
  return y;
}

py::object gated(const F8Tensor& x, const F8Tensor& gate, const F8Tensor& up, const std::string& activation,
                 const py::object& out, const py::object& dtype, const py::object& save, bool pdl,
                 int kernel, int split, const py::object& stream) {
  const at::Device device = x.device();
  same_device(device, gate);
  same_device(device, up);
  const int act = activation_code(activation);
  const attn_res_f8_t cx = x.matrix(), cg = gate.matrix(), cu = up.matrix();
  if (cx.block != ATTN_RES_F8_ROWS || cg.block != ATTN_RES_F8_SQUARE || cu.block != ATTN_RES_F8_SQUARE)
    refuse("x must have a scale for each row (block 1), gate and up for each block of 128 x 128");
  if (cx.cols != cg.cols || cg.rows != cu.rows || cg.cols != cu.cols)
    refuse("gate and up must have one shape, and x their width");
  const int64_t T = cx.rows, F = cg.rows;
  const bool given = !out.is_none();
  bool codes = given ? py::isinstance<F8Tensor>(out) : true;
  if (!dtype.is_none()) {
    const at::ScalarType type = dtype_of(dtype);
    if (type != at::kFloat8_e4m3fn && type != at::kBFloat16) refuse("the result is float8_e4m3fn or bfloat16");
    if (given && codes != (type == at::kFloat8_e4m3fn)) refuse("out has another dtype");
    codes = type == at::kFloat8_e4m3fn;
  }
  const On on(device, stream);
  std::optional<Result> h;
  at::Tensor rows;
  py::object result;
  if (codes) {
    h.emplace("out", out, T, F, ATTN_RES_F8_ROWS, device);
    result = h->object;
  } else {
    if (given) {
      if (!THPVariable_Check(out.ptr())) refuse("out must be an F8Tensor or a tensor");
      rows = out.cast<at::Tensor>();
      check_rows("out", rows, T, F, device);
    } else {
      rows = padded(T, F, F % 8 == 0 ? 8 : 16, at::kBFloat16, device);
    }
    result = py::cast(rows);
  }
  std::optional<Result> g, u;
  if (wanted(save)) {
    const auto into = outputs("save", save, 2);
    g.emplace("save", into[0], T, F, ATTN_RES_F8_ROWS, device);
    u.emplace("save", into[1], T, F, ATTN_RES_F8_ROWS, device);
  }
  check(attn_res_f8_gated(&cx, &cg, &cu, act, codes ? &h->c : nullptr, codes ? nullptr : bf16("out", rows),
                          codes ? 0 : row_stride(rows, 8), g ? &g->c : nullptr, u ? &u->c : nullptr,
                          flags_of(pdl, kernel, split), on.handle));
  if (!g) return result;
  return py::make_tuple(result, g->object, u->object);
}

py::object gated_backward(const at::Tensor& dh, const F8Tensor& gate, const F8Tensor& up, const std::string& activation,
                          const py::object& out, bool transposed, bool pdl, const py::object& stream) {
  const at::Device device = gate.device();
  same_device(device, up);
  const int act = activation_code(activation);
  const attn_res_f8_t cg = gate.matrix(), cu = up.matrix();
  if (cg.block != ATTN_RES_F8_ROWS || cu.block != ATTN_RES_F8_ROWS || cg.rows != cu.rows || cg.cols != cu.cols)
    refuse("gate and up must have one shape and a scale for each row (block 1)");
  const int64_t T = cg.rows, F = cg.cols;
  check_rows("dh", dh, T, F, device);
  const On on(device, stream);
  const auto into = outputs("out", out, transposed ? 5 : 2);
  std::vector<Result> r;
  r.reserve(into.size());
  for (size_t i = 0; i < into.size(); ++i)
    r.emplace_back("out", into[i], i < 2 ? T : F, i < 2 ? F : T, ATTN_RES_F8_ROWS, device);
  check(attn_res_f8_gated_backward(bf16("dh", dh), row_stride(dh, 8), &cg, &cu, act, &r[0].c, &r[1].c,
                                   transposed ? &r[2].c : nullptr, transposed ? &r[3].c : nullptr,
                                   transposed ? &r[4].c : nullptr, attn_res_binding::flags_of(pdl), on.handle));
  py::tuple t(r.size());
  for (size_t i = 0; i < r.size(); ++i) t[i] = r[i].object;
  return t;
}

}  // namespace

PYBIND11_MODULE(_f8, m) {
  using namespace py::literals;
  py::class_<F8Tensor>(m, "F8Tensor", R"(A matrix [rows, cols] of e4m3 codes with fp32 scales for blocks of 128.

data: [rows, cols] float8_e4m3fn, unit inner stride, rows a multiple of 16 bytes
apart; scales: float32 of ``scales_shape(rows, cols, block)``, unit inner stride,
for block 1 (a scale for each row and 128 columns) rows a multiple of 4 floats
apart.  block 128: a scale for each 128 x 128.  Every call takes and checks both
tensors as they then are.)")
      .def(py::init(&make), "data"_a, "scales"_a, "block"_a = ATTN_RES_F8_ROWS)
      .def_static(
          "empty",
          [](int64_t rows, int64_t cols, int block, const py::object& device) {
            check_block(block);
            if (rows < 0 || cols < 0) refuse("rows and cols must be >= 0");
            at::Device d = py::module_::import("torch").attr("device")(device).cast<at::Device>();
            if (!d.is_cuda()) refuse("the device must be a CUDA device");
            if (!d.has_index()) d = at::Device(at::kCUDA, c10::cuda::current_device());
            return allocate(rows, cols, block, d);
          },
          "rows"_a, "cols"_a, "block"_a = ATTN_RES_F8_ROWS, "device"_a = "cuda",
          "Uninitialised codes and scales for [rows, cols].")
      .def_property_readonly("data", [](const F8Tensor& t) { return t.data; })
      .def_property_readonly("scales", [](const F8Tensor& t) { return t.scales; })
      .def_property_readonly("block", [](const F8Tensor& t) { return t.block; })
      .def_property_readonly("shape", [](const F8Tensor& t) { return std::make_tuple(t.rows(), t.cols()); })
      .def_property_readonly("device", [](const F8Tensor& t) { return t.device(); });
  m.def("quantize", &quantize, "x"_a, "block"_a = ATTN_RES_F8_ROWS, "out"_a = py::none(), py::kw_only(),
        "transposed"_a = py::none(), "pdl"_a = false, "stream"_a = py::none(),
        R"(bf16 rows [rows, cols] to 8 bits, with scales for each row and 128 columns
(block 1) or for each 128 x 128 (attn_res_f8_quantize).  Returns ``out`` (made if
not given); with ``transposed`` (True, or an F8Tensor to fill) also the transposed
matrix, quantised by itself: (q, qt).)");
  m.def("dequantize", &dequantize, "q"_a, "out"_a = py::none(), py::kw_only(), "pdl"_a = false,
        "stream"_a = py::none(), "The bf16 values that ``q`` stands for (attn_res_f8_dequantize).");
  m.def("matmul", &matmul, "a"_a, "w"_a, "out"_a = py::none(), py::kw_only(), "dtype"_a = py::none(), "add"_a = false,
        "plus"_a = py::none(), "pdl"_a = false, "kernel"_a = 0, "split"_a = 0, "stream"_a = py::none(),
        R"(``a`` [m, k] (block 1) times the transpose of ``w`` [n, k] (either block), plus
the product of the pair ``plus`` if given: [m, n] in ``dtype``, bfloat16 (the
default) or float32, fp32 sums (attn_res_f8_matmul).  ``add`` adds to the float32
``out``.  ``kernel`` (KERNEL_NARROW, KERNEL_WIDE) and ``split`` override the
automatic choice.)");
  m.def("gated", &gated, "x"_a, "gate"_a, "up"_a, "activation"_a = "silu", "out"_a = py::none(), py::kw_only(),
        "dtype"_a = py::none(), "save"_a = false, "pdl"_a = false, "kernel"_a = 0, "split"_a = 0,
        "stream"_a = py::none(),
        R"(act(x gate^T) * (x up^T) for x [T, H] (block 1), gate and up [F, H] (block 128):
[T, F] as an F8Tensor, or with ``dtype`` (or ``out``) bfloat16 as a tensor
(attn_res_f8_gated).  ``save`` (True, or two F8Tensors to fill) keeps both
projections in 8 bits for gated_backward: (h, g, u).  ``activation``: "silu", or
"gelu" (tanh form).)");
  m.def("gated_backward", &gated_backward, "dh"_a, "gate"_a, "up"_a, "activation"_a = "silu", "out"_a = py::none(),
        py::kw_only(), "transposed"_a = true, "pdl"_a = false, "stream"_a = py::none(),
        R"(From the gradient dh [T, F] (bf16) of gated's result and its saved projections
the projections' gradients in 8 bits: (dg, du), and with ``transposed`` (dg, du,
dg^T, du^T, h^T), for the gradients of the weights (attn_res_f8_gated_backward).
``out``: as many F8Tensors to fill.)");
}
