// mx_binding.cpp -- Python binding of the microscaled entry points
// (attn_res_mx_* of include/attn_res.h): argument marshalling only, as the
// ctypes binding's, compiled because a decode step's calls take the GPU two to
// six microseconds each and interpreted marshalling with two allocations took
// fourteen.  PyTorch provides the device memory, the streams and the tensors.
#include <ATen/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <pybind11/stl.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>
#include <tuple>

#include "attn_res.h"

namespace py = pybind11;

namespace {

using OptTensor = std::optional<at::Tensor>;

[[noreturn]] void refuse(const std::string& why) { throw py::value_error(why); }

int format_code(const std::string& f) {
  if (f == "mxfp8") return ATTN_RES_MXFP8;
  if (f == "mxfp4") return ATTN_RES_MXFP4;
  if (f == "nvfp4") return ATTN_RES_NVFP4;
  refuse("format must be one of mxfp8, mxfp4, nvfp4");
}
const char* format_name(int f) {
  return f == ATTN_RES_MXFP8 ? "mxfp8" : f == ATTN_RES_MXFP4 ? "mxfp4" : "nvfp4";
}
at::ScalarType data_type(int f) { return f == ATTN_RES_MXFP8 ? at::kFloat8_e4m3fn : at::kByte; }
at::ScalarType scales_type(int f) { return f == ATTN_RES_NVFP4 ? at::kFloat8_e4m3fn : at::kFloat8_e8m0fnu; }
std::array<int64_t, 5> scales_shape(int f, int64_t rows, int64_t cols) {
  return {(rows + 127) / 128, (cols / (f == ATTN_RES_NVFP4 ? 16 : 32) + 3) / 4, 32, 4, 4};
}

at::Tensor new_tensor(at::IntArrayRef shape, at::ScalarType type, at::Device device) {
  return at::detail::empty_cuda(shape, type, device, std::nullopt);
}

// The stride of a single row says nothing (it may be anything): such a matrix
// gets the least that the entry points take.
int64_t row_stride(const at::Tensor& t, int64_t to) {
  return t.size(0) > 1 ? t.stride(0) : (t.size(1) + to - 1) / to * to;
}

// The address of a tensor's first element.  A storage can shrink under its
// tensors (untyped_storage().resize_()): elements outside it have no address.
void* address(const char* name, const at::Tensor& t) {
  const c10::TensorImpl* const impl = t.unsafeGetTensorImpl();
  const int64_t n = impl->numel();
  if (n > 0) {
    int64_t last = impl->storage_offset();
    if (impl->is_contiguous()) {
      last += n - 1;
    } else {
      const at::IntArrayRef size = impl->sizes(), stride = impl->strides();
      for (size_t d = 0; d < size.size(); ++d) last += (size[d] - 1) * stride[d];
    }
    if ((static_cast<size_t>(last) + 1) * impl->itemsize() > impl->unsafe_storage().nbytes())
      refuse(std::string(name) + "'s storage does not hold its elements");
  }
  return t.data_ptr();
}

void check_global_scale(int f, const OptTensor& g, at::Device device) {
  if (g && (f != ATTN_RES_NVFP4 || g->scalar_type() != at::kFloat || g->numel() != 1 || g->device() != device))
    refuse("global_scale must be one float32 beside the data (nvfp4 only)");
}

// The tensors are the caller's too, who may give them other storage, sizes or
// types between two calls: addresses, strides and sizes are taken, and the
// parts checked, at each call.
struct MxTensor {
  at::Tensor data, scales;
  OptTensor global_scale;
  int format;

  int64_t rows() const { return data.sizes().at(0); }
  int64_t cols() const { return data.sizes().at(1) * (format == ATTN_RES_MXFP8 ? 1 : 2); }
  at::Device device() const { return data.device(); }

  void check() const {
    const at::IntArrayRef size = data.sizes();
    if (data.scalar_type() != data_type(format) || size.size() != 2 || !data.is_cuda() ||
        (data.strides()[1] != 1 && size[1] > 1))
      refuse(std::string("data must be a CUDA ") + c10::toString(data_type(format)) +
             " matrix with unit inner stride");
    const auto shape = scales_shape(format, rows(), cols());
    if (scales.scalar_type() != scales_type(format) || scales.device() != data.device() ||
        scales.sizes() != at::IntArrayRef(shape) || !scales.is_contiguous())
      refuse(std::string("scales must be a contiguous ") + c10::toString(scales_type(format)) +
             " tensor of scales_shape(format, rows, cols) beside data");
    check_global_scale(format, global_scale, data.device());
  }

  attn_res_mx_t matrix() const {
    check();
    attn_res_mx_t c = {};
    c.format = format;
    c.rows = rows();
    c.cols = cols();
    c.data = address("data", data);
    c.row_bytes = row_stride(data, 16);
    c.scales = static_cast<uint8_t*>(address("scales", scales));
    c.tensor_scale = global_scale ? static_cast<const float*>(address("global_scale", *global_scale)) : nullptr;
    return c;
  }
};

MxTensor make(const at::Tensor& data, const at::Tensor& scales, const std::string& format, const OptTensor& g) {
  MxTensor t{data, scales, g, format_code(format)};
  t.check();
  return t;
}

void check_shape(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0 || cols % 32) refuse("rows must be >= 0 and the width a positive multiple of 32");
}

MxTensor allocate(int64_t rows, int64_t cols, int f, const OptTensor& g, at::Device device) {
  check_shape(rows, cols);
  check_global_scale(f, g, device);
  return {new_tensor({rows, f == ATTN_RES_MXFP8 ? cols : cols / 2}, data_type(f), device),
          new_tensor(scales_shape(f, rows, cols), scales_type(f), device), g, f};
}

void check_rows(const char* name, const at::Tensor& t) {
  if (t.scalar_type() != at::kBFloat16 || !t.is_cuda()) refuse(std::string(name) + " must be a CUDA bfloat16 tensor");
  if (t.dim() != 2 || (t.stride(1) != 1 && t.size(1) > 1))
    refuse(std::string(name) + " must be a 2-D matrix with unit inner stride");
}
void check_rows(const char* name, const at::Tensor& t, int64_t rows, int64_t cols, at::Device device) {
  check_rows(name, t);
  if (t.size(0) != rows || t.size(1) != cols)
    refuse(std::string(name) + " must be a [" + std::to_string(rows) + ", " + std::to_string(cols) + "] matrix");
  if (t.device() != device) refuse("all tensors of a call must be on one device");
}
attn_res_bf16_t* bf16(const char* name, const at::Tensor& t) {
  return static_cast<attn_res_bf16_t*>(address(name, t));
}

// The device and stream of a call: current while outputs are allocated and the
// kernel is launched.
struct On {
  c10::cuda::OptionalCUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard stream;
  void* handle;
  On(at::Device d, const py::object& s) {
    if (s.is_none()) {
      device.set_device(d);
      handle = c10::cuda::getCurrentCUDAStream(d.index()).stream();
    } else {
      if (!py::hasattr(s, "stream_id") || !py::hasattr(s, "device_index") || !py::hasattr(s, "device_type"))
        refuse("stream must be a torch.cuda.Stream");
      const auto given = c10::cuda::CUDAStream::unpack3(
          s.attr("stream_id").cast<int64_t>(), static_cast<c10::DeviceIndex>(s.attr("device_index").cast<int64_t>()),
          static_cast<c10::DeviceType>(s.attr("device_type").cast<int64_t>()));
      if (given.device() != d) refuse("stream must belong to the tensors' device");
      stream.reset_stream(given);
      handle = given.stream();
    }
  }
};

void check(attn_res_status_t st) {
  if (st == ATTN_RES_OK) return;
  const py::object type = py::module_::import("attention_residual_fusion_gb300").attr("AttnResError");
  const py::object error = type(static_cast<int>(st), attn_res_status_string(st));
  PyErr_SetObject(type.ptr(), error.ptr());
  throw py::error_already_set();
}
uint32_t flags_of(bool pdl) { return pdl ? ATTN_RES_FLAG_PDL : 0u; }

// The result of a quantising call: `out`, checked, or a new one.
py::object result(const py::object& out, int64_t rows, int64_t cols, const std::string& format, const OptTensor& g,
                  at::Device device, attn_res_mx_t* c) {
  const int f = format_code(format);
  if (out.is_none()) {
    py::object made = py::cast(allocate(rows, cols, f, g, device));
    *c = made.cast<const MxTensor&>().matrix();
    return made;
  }
  if (!py::isinstance<MxTensor>(out)) refuse("out must be an MxTensor");
  const MxTensor& o = out.cast<const MxTensor&>();
  if (o.format != f || (g && !(o.global_scale && g->is_same(*o.global_scale))))
    refuse("out has another format or global_scale");
  *c = o.matrix();
  if (c->rows != rows || c->cols != cols || o.device() != device)
    refuse("out must be an MxTensor of the rows' shape, on their device");
  return out;
}

py::object quantize(const at::Tensor& x, const std::string& format, const OptTensor& global_scale,
                    const py::object& out, bool pdl, const py::object& stream) {
  check_rows("x", x);
  const On on(x.device(), stream);
  attn_res_mx_t c;
  py::object q = result(out, x.size(0), x.size(1), format, global_scale, x.device(), &c);
  check(attn_res_mx_quantize(bf16("x", x), row_stride(x, 8), &c, flags_of(pdl), on.handle));
  return q;
}

at::Tensor dequantize(const MxTensor& q, const OptTensor& out, bool pdl, const py::object& stream) {
  const attn_res_mx_t c = q.matrix();
  const On on(q.device(), stream);
  if (out) check_rows("out", *out, c.rows, c.cols, q.device());
  at::Tensor x = out ? *out : new_tensor({c.rows, c.cols}, at::kBFloat16, q.device());
  check(attn_res_mx_dequantize(&c, bf16("out", x), row_stride(x, 8), flags_of(pdl), on.handle));
  return x;
}

py::object add_rms_norm(const at::Tensor& prefix, const OptTensor& delta, const at::Tensor& weight, double eps,
                        const std::string& format, const OptTensor& global_scale, const py::object& out,
                        const OptTensor& norm_out, bool pdl, const py::object& stream) {
  check_rows("prefix", prefix);
  const at::Device device = prefix.device();
  const int64_t rows = prefix.size(0), cols = prefix.size(1);
  if (delta) check_rows("delta", *delta, rows, cols, device);
  if (norm_out) check_rows("norm_out", *norm_out, rows, cols, device);
  if (weight.scalar_type() != at::kBFloat16 || weight.device() != device || weight.dim() != 1 ||
      weight.size(0) != cols || !weight.is_contiguous())
    refuse("weight must be a contiguous bfloat16 [H] tensor beside prefix");
  const On on(device, stream);
  attn_res_mx_t c;
  py::object q = result(out, rows, cols, format, global_scale, device, &c);
  check(attn_res_mx_norm(bf16("prefix", prefix), row_stride(prefix, 8), delta ? bf16("delta", *delta) : nullptr,
                         delta ? row_stride(*delta, 8) : 0, bf16("weight", weight), static_cast<float>(eps),
                         norm_out ? bf16("norm_out", *norm_out) : nullptr, norm_out ? row_stride(*norm_out, 8) : 0,
                         &c, flags_of(pdl), on.handle));
  return q;
}

at::Tensor matmul(const MxTensor& a, const MxTensor& w, const OptTensor& out, bool pdl, int kernel, int split,
                  const py::object& stream) {
  const attn_res_mx_t ca = a.matrix(), cw = w.matrix();
  const at::Device device = a.device();
  const int64_t m = ca.rows, n = cw.rows;
  if (ca.format != cw.format || ca.cols != cw.cols) refuse("a and w must have one format and one width");
  if (w.device() != device) refuse("all tensors of a call must be on one device");
  const On on(device, stream);
  at::Tensor y;
  int64_t row;
  if (out) {
    check_rows("out", *out, m, n, device);
    y = *out;
    row = row_stride(y, 8);
  } else {
    // rows start on 16-byte boundaries, whatever n; where they are padded
    // anyway, on 32-byte ones (the wide forms then store whole sectors)
    row = n % 8 == 0 ? n : (n + 15) / 16 * 16;
    y = new_tensor({m, row}, at::kBFloat16, device);
    if (row != n) y = y.narrow(1, 0, n);
  }
  if (kernel < 0 || kernel > 15 || split < 0 || split > 255) refuse("no such kernel or split");
  check(attn_res_mx_matmul(&ca, &cw, bf16("out", y), row,
                           flags_of(pdl) | ATTN_RES_FLAG_KERNEL(kernel) | ATTN_RES_FLAG_SPLIT(split), on.handle));
  return y;
}

}  // namespace

PYBIND11_MODULE(_mx, m) {
  using namespace py::literals;
  py::class_<MxTensor>(m, "MxTensor", R"(A matrix [rows, cols] in a microscaled format.

data: [rows, cols] float8_e4m3fn ("mxfp8") or [rows, cols // 2] uint8 (two
e2m1 codes a byte, the even column low), unit inner stride; scales:
``scales_shape(format, rows, cols)``, contiguous, float8_e8m0fnu or (nvfp4)
float8_e4m3fn; global_scale: one fp32 on the device, nvfp4 only, or None.
Every call takes and checks the three tensors as they then are, so they may be
given other storage in between; one whose storage is gone is refused.)")
      .def(py::init(&make), "data"_a, "scales"_a, "format"_a, "global_scale"_a = py::none())
      .def_static(
          "empty",
          [](int64_t rows, int64_t cols, const std::string& format, const OptTensor& g, const py::object& device) {
            const int f = format_code(format);
            check_shape(rows, cols);
            at::Device d = py::module_::import("torch").attr("device")(device).cast<at::Device>();
            if (!d.is_cuda()) refuse("the device must be a CUDA device");
            if (!d.has_index()) d = at::Device(at::kCUDA, c10::cuda::current_device());
            return allocate(rows, cols, f, g, d);
          },
          "rows"_a, "cols"_a, "format"_a, "global_scale"_a = py::none(), "device"_a = "cuda",
          "Uninitialised codes and scales for [rows, cols] (cols a multiple of 32).")
      .def_property_readonly("data", [](const MxTensor& t) { return t.data; })
      .def_property_readonly("scales", [](const MxTensor& t) { return t.scales; })
      .def_property_readonly("global_scale", [](const MxTensor& t) { return t.global_scale; })
      .def_property_readonly("format", [](const MxTensor& t) { return format_name(t.format); })
      .def_property_readonly("shape", [](const MxTensor& t) { return std::make_tuple(t.rows(), t.cols()); })
      .def_property_readonly("device", [](const MxTensor& t) { return t.device(); });
  m.def("quantize", &quantize, "x"_a, "format"_a = "mxfp4", "global_scale"_a = py::none(), "out"_a = py::none(),
        py::kw_only(), "pdl"_a = false, "stream"_a = py::none(),
        R"(bf16 rows [rows, cols] to ``format`` (attn_res_mx_quantize).  cols is a
multiple of 32; ``global_scale`` (nvfp4) is the tensor's scale, 1 if None.
Returns ``out`` (allocated if not given; its own global_scale then holds).)");
  m.def("dequantize", &dequantize, "q"_a, "out"_a = py::none(), py::kw_only(), "pdl"_a = false,
        "stream"_a = py::none(),
        "The bf16 values [rows, cols] that ``q`` stands for (attn_res_mx_dequantize).");
  m.def("add_rms_norm", &add_rms_norm, "prefix"_a, "delta"_a.none(true), "weight"_a, "eps"_a = 1e-6,
        "format"_a = "mxfp8", "global_scale"_a = py::none(), "out"_a = py::none(), "norm_out"_a = py::none(),
        py::kw_only(), "pdl"_a = false, "stream"_a = py::none(),
        R"(Residual addition and RMSNorm of token rows, quantised (attn_res_mx_norm).

c = bf16(prefix + delta) (prefix if ``delta`` is None; prefix [T, H] is
updated in place otherwise), y = c * weight / sqrt(mean(c^2) + eps); the
result is y in ``format``, from fp32.  ``norm_out`` [T, H] receives y in
bf16 as well, if given.  H is a multiple of 32, at most 65536.)");
  m.def("matmul", &matmul, "a"_a, "w"_a, "out"_a = py::none(), py::kw_only(), "pdl"_a = false, "kernel"_a = 0,
        "split"_a = 0, "stream"_a = py::none(),
        R"(``a`` [m, k] times the transpose of ``w`` [n, k], of one format: bf16
[m, n], fp32 sums (attn_res_mx_matmul).  ``kernel`` (KERNEL_NARROW,
KERNEL_WIDE, KERNEL_WIDER) and ``split`` override the automatic choice.)");
}
