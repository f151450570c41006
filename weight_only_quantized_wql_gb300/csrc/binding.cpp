// binding.cpp -- the Python calls of the operators around the head: argument
// checks, outputs from torch's allocator, torch's current stream, one call of
// the C ABI.  No computation.  Through ctypes and Python a call cost the host
// 10 to 14 us, through this 5.5 to 8.5 us (a 1 x 1024 row's norm 12 and 8.2, whose
// kernel takes 2): the smallest calls are bound by the host.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <optional>
#include <string>
#include <tuple>

#include "wql.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using MaybeTensor = std::optional<Tensor>;

[[noreturn]] void refuse(const std::string& why) { throw py::value_error(why); }

void check_status(const char* fn, wql_status status) {
  if (status == WQL_OK) return;
  const py::object e =
      py::module_::import("weight_only_quantized_wql_gb300").attr("WQLError")(fn, (int)status);
  PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e.ptr())), e.ptr());
  throw py::error_already_set();
}

void check_cuda(const Tensor& t, const char* name) {
  if (!t.is_cuda())
    refuse(std::string(name) + " must be a CUDA tensor (the library has no CPU path)");
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
}

// A contiguous tensor of `numel` elements of a type, on x's device.
void check_like(const Tensor& t, const char* name, const Tensor& x, at::ScalarType type,
                int64_t numel) {
  check_cuda(t, name);
  if (t.scalar_type() != type || t.numel() != numel || t.get_device() != x.get_device())
    refuse(std::string(name) + " must be a " + c10::toString(type) + " tensor of " +
           std::to_string(numel) + " elements on cuda:" + std::to_string(x.get_device()));
}

const void* pointer(const MaybeTensor& t) { return t ? t->const_data_ptr() : nullptr; }

// wql_dtype; anything else is refused by the library
int32_t dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return WQL_F32;
    case at::kHalf: return WQL_F16;
    case at::kBFloat16: return WQL_BF16;
    default: return -1;
  }
}

cudaStream_t stream_of(const Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
}

// Rows and columns, leading dimensions flattened.
std::pair<int64_t, int64_t> rows_of(const Tensor& x, const char* name) {
  check_cuda(x, name);
  if (x.dim() < 1) refuse(std::string(name) + " must have at least one dimension");
  const int64_t k = x.size(-1);
  return {k ? x.numel() / k : 0, k};
}

struct Codes {
  Tensor codes, scales;
};
Codes empty_codes(int64_t rows, int64_t k, int64_t fmt, const Tensor& x) {
  if (fmt != WQL_MX_FP4 && fmt != WQL_MX_FP8) refuse("fmt must be MX_FP4 or MX_FP8");
  const auto bytes = x.options().dtype(at::kByte);
  return {at::empty({rows, fmt == WQL_MX_FP4 ? k / 2 : k}, bytes),
          at::empty({(rows + 127) / 128, (k + 127) / 128, 512}, bytes)};
}

// (codes, scales, format, rows, columns) of an MXMatrix
using Matrix = std::tuple<Tensor, Tensor, int64_t, int64_t, int64_t>;

wql_mx checked(const Matrix& m, const char* name) {
  const auto& [codes, scales, fmt, rows, k] = m;
  const std::string n(name);
  check_cuda(codes, (n + ".codes").c_str());
  check_cuda(scales, (n + ".scales").c_str());
  if (codes.scalar_type() != at::kByte || scales.scalar_type() != at::kByte)
    refuse(n + ".codes and .scales must be uint8");
  if (codes.numel() != rows * (fmt == WQL_MX_FP4 ? k / 2 : k))
    refuse(n + ".codes does not hold " + std::to_string(rows) + " x " + std::to_string(k) +
           " codes");
  if (scales.numel() != (rows + 127) / 128 * ((k + 127) / 128) * 512)
    refuse(n + ".scales does not hold the scale tiles of " + std::to_string(rows) + " x " +
           std::to_string(k));
  if (codes.get_device() != scales.get_device())
    refuse(n + "'s codes and scales must lie on one device");
  return wql_mx{(int32_t)fmt, 0, rows, k, codes.const_data_ptr(), scales.const_data_ptr()};
}

std::tuple<Tensor, Tensor, int64_t, int64_t> mx_quantize(const Tensor& x, int64_t fmt) {
  const auto [rows, k] = rows_of(x, "x");
  const c10::cuda::CUDAGuard on(x.device());
  Codes c = empty_codes(rows, k, fmt, x);
  check_status("wql_mx_quantize",
               wql_mx_quantize(x.const_data_ptr(), dtype_code(x.scalar_type()), rows, k,
                               (int32_t)fmt, c.codes.data_ptr(), c.scales.data_ptr(),
                               stream_of(x)));
  return {c.codes, c.scales, rows, k};
}

Tensor mx_dequantize(const Matrix& a, at::ScalarType out_dtype) {
  const wql_mx m = checked(a, "a");
  const Tensor& codes = std::get<0>(a);
  const c10::cuda::CUDAGuard on(codes.device());
  Tensor out = at::empty({m.rows, m.k}, codes.options().dtype(out_dtype));
  check_status("wql_mx_dequantize",
               wql_mx_dequantize(&m, dtype_code(out_dtype), out.data_ptr(), stream_of(codes)));
  return out;
}

Tensor mx_logits(const Matrix& x, const Matrix& w, at::ScalarType out_dtype,
                 const MaybeTensor& bias, const MaybeTensor& out, const MaybeTensor& workspace) {
  const wql_mx mx = checked(x, "x"), mw = checked(w, "w");
  const Tensor& codes = std::get<0>(x);
  if (codes.get_device() != std::get<0>(w).get_device()) refuse("x and w must lie on one device");
  if (workspace) {
    check_cuda(*workspace, "workspace");
    if (workspace->scalar_type() != at::kByte ||
        workspace->get_device() != codes.get_device())
      refuse("workspace must hold bytes on cuda:" + std::to_string(codes.get_device()));
  }
  const c10::cuda::CUDAGuard on(codes.device());
  Tensor y;
  if (out) {
    check_like(*out, "out", codes, out_dtype, mx.rows * mw.rows);
    y = *out;
  } else {
    y = at::empty({mx.rows, mw.rows}, codes.options().dtype(out_dtype));
  }
  if (bias) check_like(*bias, "bias", codes, out_dtype, mw.rows);
  check_status("wql_mx_logits",
               wql_mx_logits(&mx, &mw, pointer(bias), dtype_code(out_dtype), y.data_ptr(),
                             workspace ? workspace->data_ptr() : nullptr,
                             workspace ? (size_t)workspace->numel() : 0, stream_of(codes)));
  return y;
}

// (y or codes, residual_out, row scales, scale tiles)
std::tuple<Tensor, MaybeTensor, MaybeTensor, MaybeTensor> add_rmsnorm(
    const Tensor& x, const Tensor& gamma, const MaybeTensor& residual, double eps, int64_t fmt,
    const MaybeTensor& residual_out) {
  const auto [m, k] = rows_of(x, "x");
  const at::ScalarType type = x.scalar_type();
  check_like(gamma, "gamma", x, type, k);
  if (residual) check_like(*residual, "residual", x, type, m * k);
  if (residual_out) check_like(*residual_out, "residual_out", x, type, m * k);
  const c10::cuda::CUDAGuard on(x.device());
  MaybeTensor h = residual_out;
  if (residual && !h) h = at::empty_like(*residual);
  Tensor y;
  MaybeTensor scales, tiles;
  switch (fmt) {
    case WQL_NORM_SAME: y = at::empty_like(x); break;
    case WQL_NORM_E4M3:
      y = at::empty(x.sizes(), x.options().dtype(at::kFloat8_e4m3fn));
      scales = at::empty(x.sizes().slice(0, x.dim() - 1), x.options().dtype(at::kFloat));
      break;
    case WQL_NORM_MX_FP8:
    case WQL_NORM_MX_FP4: {
      Codes c = empty_codes(m, k, fmt == WQL_NORM_MX_FP8 ? WQL_MX_FP8 : WQL_MX_FP4, x);
      y = c.codes;
      tiles = c.scales;
      break;
    }
    default: refuse("fmt must be one of NORM_SAME, NORM_E4M3, NORM_MX_FP8, NORM_MX_FP4");
  }
  void* out_scales = scales ? scales->data_ptr() : tiles ? tiles->data_ptr() : nullptr;
  check_status("wql_add_rmsnorm",
               wql_add_rmsnorm(x.const_data_ptr(), pointer(residual), gamma.const_data_ptr(),
                               dtype_code(type), m, k, (float)eps, (int32_t)fmt, y.data_ptr(),
                               out_scales, h ? h->data_ptr() : nullptr, stream_of(x)));
  return {y, h, scales, tiles};
}

std::tuple<Tensor, Tensor> sample(const Tensor& logits, const Tensor& u,
                                  const MaybeTensor& temperature, const MaybeTensor& top_k,
                                  const MaybeTensor& top_p, const MaybeTensor& min_p) {
  const auto [m, n] = rows_of(logits, "logits");
  check_like(u, "u", logits, at::kFloat, m);
  if (temperature) check_like(*temperature, "temperature", logits, at::kFloat, m);
  if (top_k) check_like(*top_k, "top_k", logits, at::kInt, m);
  if (top_p) check_like(*top_p, "top_p", logits, at::kFloat, m);
  if (min_p) check_like(*min_p, "min_p", logits, at::kFloat, m);
  const c10::cuda::CUDAGuard on(logits.device());
  const auto shape = logits.sizes().slice(0, logits.dim() - 1);
  Tensor ids = at::empty(shape, logits.options().dtype(at::kInt));
  Tensor logp = at::empty(shape, logits.options().dtype(at::kFloat));
  check_status(
      "wql_sample",
      wql_sample(logits.const_data_ptr(), dtype_code(logits.scalar_type()), m, n,
                 static_cast<const float*>(u.const_data_ptr()),
                 static_cast<const float*>(pointer(temperature)),
                 static_cast<const int32_t*>(pointer(top_k)),
                 static_cast<const float*>(pointer(top_p)),
                 static_cast<const float*>(pointer(min_p)), static_cast<int32_t*>(ids.data_ptr()),
                 static_cast<float*>(logp.data_ptr()), stream_of(logits)));
  return {ids, logp};
}

}  // namespace

PYBIND11_MODULE(_wql_torch, m) {
  m.def("mx_quantize", &mx_quantize);
  m.def("mx_dequantize", &mx_dequantize);
  m.def("mx_logits", &mx_logits);
  m.def("add_rmsnorm", &add_rmsnorm);
  m.def("sample", &sample);
}
