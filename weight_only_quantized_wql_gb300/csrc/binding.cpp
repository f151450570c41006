// binding.cpp -- the Python calls of the operators around the head: argument
// checks, outputs from torch's allocator, torch's current stream, one call of
// the C ABI.  No computation.  Through ctypes and Python a call cost the host
// 10 to 14 us, through this 5.5 to 8.5 us (a 1 x 1024 row's norm 12 and 8.2, whose
// kernel takes 2): the smallest calls are bound by the host.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <optional>
#include <string>
#include <tuple>
#include <vector>

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

// A new tensor on the device of another one, without the dispatcher's part (half
// a microsecond each).
Tensor empty_on(const Tensor& like, at::IntArrayRef sizes, at::ScalarType type) {
  return at::detail::empty_cuda(sizes, type, like.device(), std::nullopt);
}

// A call's workspace: the one given, or memory of torch's allocator, which
// orders its reuse on the current stream and takes a captured call's from its
// graph's own pool.
struct Scratch {
  c10::DataPtr own;
  void* data;
  size_t bytes;
  Scratch(const MaybeTensor& given, size_t need, const Tensor& like) {
    if (given) {
      check_cuda(*given, "workspace");
      if (given->scalar_type() != at::kByte || given->get_device() != like.get_device())
        refuse("workspace must hold bytes on cuda:" + std::to_string(like.get_device()));
      data = given->data_ptr();
      bytes = (size_t)given->numel();
    } else {
      if (need) own = c10::cuda::CUDACachingAllocator::get()->allocate(need);
      data = own.get();
      bytes = need;
    }
  }
};

Tensor lora_add(const Tensor& y, const Tensor& x, const Tensor& a, const Tensor& b,
                const MaybeTensor& scale, const Tensor& ids, const MaybeTensor& out,
                const MaybeTensor& workspace) {
  const auto [m, k] = rows_of(x, "x");
  const at::ScalarType type = x.scalar_type();
  check_cuda(a, "a");
  check_cuda(b, "b");
  if (a.dim() != 3 || b.dim() != 3 || a.size(0) != b.size(0) || a.size(1) != b.size(2))
    refuse("the adapters' a must be [count, rank, k] and b [count, n, rank]");
  if (a.size(2) != k) refuse("x and the adapters' a must have the same last dimension");
  if (a.scalar_type() != type || b.scalar_type() != type || a.get_device() != x.get_device() ||
      b.get_device() != x.get_device())
    refuse("the adapters must have x's type and lie on its device");
  const int64_t count = a.size(0), rank = a.size(1), n = b.size(1);
  if (scale) check_like(*scale, "scale", x, at::kFloat, count);
  check_like(ids, "ids", x, at::kInt, m);
  check_like(y, "y", x, type, m * n);
  if (y.dim() < 1 || y.size(-1) != n) refuse("y's last dimension must be the adapters' n");
  if (out) check_like(*out, "out", x, type, m * n);
  const c10::cuda::CUDAGuard on(x.device());
  Tensor to = out ? *out : empty_on(y, y.sizes(), type);
  const Scratch ws(workspace, wql_lora_workspace_size(m, (int32_t)rank), x);
  const wql_lora w{dtype_code(type), (int32_t)rank, count, n, k, a.const_data_ptr(),
                   b.const_data_ptr(), static_cast<const float*>(pointer(scale))};
  check_status("wql_lora_add",
               wql_lora_add(&w, x.const_data_ptr(), m, static_cast<const int32_t*>(ids.const_data_ptr()),
                            y.const_data_ptr(), to.data_ptr(), ws.data, ws.bytes, stream_of(x)));
  return to;
}

// (tokens, parents, scores, ended)
std::tuple<Tensor, Tensor, Tensor, MaybeTensor> beam_select(const Tensor& logits,
                                                            const Tensor& scores,
                                                            std::optional<int64_t> eos,
                                                            int64_t order,
                                                            const MaybeTensor& workspace) {
  const auto [rows, n] = rows_of(logits, "logits");
  if (scores.dim() != 2) refuse("scores must be [batch, beams]");
  check_like(scores, "scores", logits, at::kFloat, rows);
  const int64_t batch = scores.size(0), beams = scores.size(1);
  if (eos && (*eos < 0 || *eos >= n)) refuse("eos must be a token of the vocabulary, or None");
  if (order != WQL_BEAM_RANKED && order != WQL_BEAM_ANCHORED)
    refuse("order must be BEAM_RANKED or BEAM_ANCHORED");
  const c10::cuda::CUDAGuard on(logits.device());
  Tensor tokens = empty_on(logits, {batch, beams}, at::kInt);
  Tensor parents = empty_on(logits, {batch, beams}, at::kInt);
  Tensor best = empty_on(logits, {batch, beams}, at::kFloat);
  MaybeTensor ended;
  if (eos) ended = empty_on(logits, {batch, beams}, at::kFloat);
  const Scratch ws(workspace, wql_beam_workspace_size(batch, beams, n), logits);
  check_status(
      "wql_beam_select",
      wql_beam_select(logits.const_data_ptr(), dtype_code(logits.scalar_type()), batch, beams, n,
                      static_cast<const float*>(scores.const_data_ptr()),
                      eos ? (int32_t)*eos : -1, (int32_t)order,
                      static_cast<int32_t*>(tokens.data_ptr()),
                      static_cast<int32_t*>(parents.data_ptr()),
                      static_cast<float*>(best.data_ptr()),
                      ended ? static_cast<float*>(ended->data_ptr()) : nullptr, ws.data, ws.bytes,
                      stream_of(logits)));
  return {tokens, parents, best, ended};
}

// The dimensions [from, to) of a tensor as one, given what lies behind them.
struct Folded {
  int64_t count = 1, stride = 0;         // bytes
};
bool fold(const Tensor& t, int64_t from, int64_t to, Folded* f) {
  const int64_t size = t.element_size();
  for (int64_t d = to - 1; d >= from; --d) {
    if (t.size(d) == 1) continue;
    const int64_t stride = t.stride(d) * size;
    if (f->count == 1) f->stride = stride;
    else if (stride != f->stride * f->count) return false;
    f->count *= t.size(d);
  }
  return true;
}

wql_state state_of(Tensor& t, int64_t rows, const std::optional<int64_t>& position_dim) {
  if (!t.is_cuda()) refuse("states must be CUDA tensors (the library has no CPU path)");
  if (t.dim() < 1 || t.size(0) < rows)
    refuse("a state's first dimension must hold batch * beams = " + std::to_string(rows) + " rows");
  const int64_t size = t.element_size(), dims = t.dim();
  wql_state s{};
  s.data = t.data_ptr();
  s.row_stride = t.stride(0) * size;
  s.outer = s.positions = 1;
  if (t.numel() == 0) {
    s.positions = 0;
    return s;
  }
  // what is contiguous at the end
  int64_t inner = dims;
  const int64_t stop = position_dim ? *position_dim + 1 : 1;
  s.position_bytes = size;
  while (inner > stop && (t.size(inner - 1) == 1 || t.stride(inner - 1) * size == s.position_bytes)) {
    --inner;
    s.position_bytes *= t.size(inner);
  }
  Folded positions, outer;
  if (position_dim) {
    if (inner != stop) refuse("the dimensions behind position_dim must be contiguous");
    fold(t, *position_dim, stop, &positions);
    if (!fold(t, 1, *position_dim, &outer))
      refuse("the dimensions between the rows and position_dim must have a common stride");
  } else {
    // up to two levels of gaps
    int64_t d = inner;
    while (d > 1) {
      Folded next = positions;
      if (!fold(t, d - 1, d, &next)) break;
      positions = next;
      --d;
    }
    if (!fold(t, 1, d, &outer)) refuse("a state's strides must fall into at most two levels of gaps");
  }
  s.positions = positions.count;
  s.position_stride = positions.count > 1 ? positions.stride : s.position_bytes;
  s.outer = outer.count;
  s.outer_stride = outer.stride;
  return s;
}

void beam_reorder(std::vector<Tensor>& states, const Tensor& parents, const MaybeTensor& lengths,
                  const std::optional<int64_t>& position_dim) {
  if (states.empty()) return;
  if (parents.dim() != 2) refuse("parents must be [batch, beams]");
  const int64_t batch = parents.size(0), beams = parents.size(1);
  const Tensor& first = states[0];
  if (!first.is_cuda()) refuse("states must be CUDA tensors (the library has no CPU path)");
  check_like(parents, "parents", first, at::kInt, batch * beams);
  if (lengths) {
    if (!position_dim) refuse("lengths need position_dim");
    check_like(*lengths, "lengths", first, at::kInt, batch);
  }
  std::vector<wql_state> list;
  list.reserve(states.size());
  for (Tensor& t : states) {
    if (t.get_device() != first.get_device()) refuse("states must lie on one device");
    if (position_dim && (*position_dim < 1 || *position_dim >= t.dim()))
      refuse("position_dim must be a dimension of every state behind the rows");
    list.push_back(state_of(t, batch * beams, position_dim));
  }
  const c10::cuda::CUDAGuard on(first.device());
  check_status("wql_beam_reorder",
               wql_beam_reorder(list.data(), (int64_t)list.size(),
                                static_cast<const int32_t*>(parents.const_data_ptr()), batch, beams,
                                static_cast<const int32_t*>(pointer(lengths)), stream_of(first)));
}

}  // namespace

PYBIND11_MODULE(_wql_torch, m) {
  m.def("mx_quantize", &mx_quantize);
  m.def("mx_dequantize", &mx_dequantize);
  m.def("mx_logits", &mx_logits);
  m.def("add_rmsnorm", &add_rmsnorm);
  m.def("sample", &sample);
  m.def("lora_add", &lora_add);
  m.def("beam_select", &beam_select);
  m.def("beam_reorder", &beam_reorder);
}
