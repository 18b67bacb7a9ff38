// binding.h -- shared by the compiled Python bindings: checks of tensors, their
// addresses, the device and stream of a call, errors.
#pragma once

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

namespace attn_res_binding {

using OptTensor = std::optional<at::Tensor>;

[[noreturn]] inline void refuse(const std::string& why) { throw py::value_error(why); }

inline at::Tensor new_tensor(at::IntArrayRef shape, at::ScalarType type, at::Device device) {
  return at::detail::empty_cuda(shape, type, device, std::nullopt);
}

// The stride of a single row says nothing (it may be anything): such a matrix
// gets the least that the entry points take.
inline int64_t row_stride(const at::Tensor& t, int64_t to) {
  return t.size(0) > 1 ? t.stride(0) : (t.size(1) + to - 1) / to * to;
}

// The address of a tensor's first element.  A storage can shrink under its
// tensors (untyped_storage().resize_()): elements outside it have no address.
inline void* address(const char* name, const at::Tensor& t) {
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

inline void check_rows(const char* name, const at::Tensor& t) {
  if (t.scalar_type() != at::kBFloat16 || !t.is_cuda()) refuse(std::string(name) + " must be a CUDA bfloat16 tensor");
  if (t.dim() != 2 || (t.stride(1) != 1 && t.size(1) > 1))
    refuse(std::string(name) + " must be a 2-D matrix with unit inner stride");
}
inline void check_rows(const char* name, const at::Tensor& t, int64_t rows, int64_t cols, at::Device device) {
  check_rows(name, t);
  if (t.size(0) != rows || t.size(1) != cols)
    refuse(std::string(name) + " must be a [" + std::to_string(rows) + ", " + std::to_string(cols) + "] matrix");
  if (t.device() != device) refuse("all tensors of a call must be on one device");
}
inline attn_res_bf16_t* bf16(const char* name, const at::Tensor& t) {
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

inline void check(attn_res_status_t st) {
  if (st == ATTN_RES_OK) return;
  const py::object type = py::module_::import("attention_residual_fusion_gb300").attr("AttnResError");
  const py::object error = type(static_cast<int>(st), attn_res_status_string(st));
  PyErr_SetObject(type.ptr(), error.ptr());
  throw py::error_already_set();
}
inline uint32_t flags_of(bool pdl) { return pdl ? ATTN_RES_FLAG_PDL : 0u; }

}  // namespace attn_res_binding
