// The torch conveniences' calls of the dense C ABI (include/nvfp4dense.h) from
// C++: checks, output and workspace allocation and the call itself in one step.
// Through ctypes the same steps take 9 to 18 us of host time, more than the
// kernels of few tokens take on the GPU.
//
// Every function returns None where an argument is not as the call needs it, autograd
// follows an operator without a backward pass, memory is short or the call is refused; nothing has been enqueued then, and the caller repeats
// the steps one by one in Python, where the error is raised.  Work goes to
// torch's current stream of x's device; memory comes from torch's allocator on
// that stream.  The interpreter lock is released meanwhile: allocation may wait for
// the GPU, and a launch for room in a full queue.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <optional>
#include <tuple>
#include <type_traits>

#include "../../../include/nvfp4dense.h"

namespace {

using at::Tensor;

int dtype_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return NVFP4DENSE_BF16;
    case at::kHalf: return NVFP4DENSE_F16;
    case at::kFloat: return NVFP4DENSE_F32;
    default: return -1;
  }
}

// A [rows, features] device tensor with contiguous features and rows that do
// not overlap; its row stride in elements.
bool rows_ok(const Tensor& t, int64_t& ld) {
  if (!t.is_cuda() || t.dim() != 2) return false;
  const int64_t n = t.size(0), f = t.size(1);
  if (f > 1 && t.stride(1) != 1) return false;
  ld = n <= 1 ? f : t.stride(0);
  return ld >= f;
}

// Whether autograd would follow what is computed from t: in a graph, or by a tangent.
bool recorded(const Tensor& t) {
  if (t.requires_grad() && c10::GradMode::is_enabled()) return true;
  return t._fw_grad(0).defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode();
}

bool matrix_ok(const Tensor& t, int64_t r, int64_t c, const Tensor& like) {
  return t.is_cuda() && t.dim() == 2 && t.size(0) == r && t.size(1) == c && t.is_contiguous() &&
         t.scalar_type() == like.scalar_type() && t.get_device() == like.get_device();
}

using Gradients = std::tuple<std::optional<Tensor>, std::optional<Tensor>, std::optional<Tensor>, std::optional<Tensor>>;

// An uninitialised tensor on like's device (at::empty without its dispatch).
Tensor empty(at::IntArrayRef size, at::ScalarType type, const Tensor& like) {
  return at::detail::empty_cuda(size, type, like.device(), std::nullopt);
}
Tensor bytes(size_t n, const Tensor& like) { return empty({(int64_t)std::max<size_t>(n, 256)}, at::kByte, like); }

void* current_stream(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }

std::optional<std::tuple<Tensor, Tensor>> quantize(const Tensor& x) {
  int64_t ld;
  const int dt = dtype_of(x);
  if (dt < 0 || !rows_ok(x, ld)) return std::nullopt;
  const c10::cuda::CUDAGuard guard(x.device());
  const int64_t R = x.size(0), K = x.size(1), nb = (K + 31) / 32;
  Tensor codes = empty({R, 16 * nb}, at::kByte, x), scales = empty({R, nb}, at::kByte, x);
  if (mxfp4_quantize(x.data_ptr(), dt, R, K, ld, codes.data_ptr<uint8_t>(), scales.data_ptr<uint8_t>(),
                     current_stream(x)) != NVFP4_OK)
    return std::nullopt;
  return std::make_tuple(std::move(codes), std::move(scales));
}

// K < 0: whole blocks
std::optional<Tensor> dequantize(const Tensor& codes, const Tensor& scales, int64_t K, bool bf16) {
  if (!codes.is_cuda() || !scales.is_cuda() || scales.dim() != 2 || codes.scalar_type() != at::kByte) return std::nullopt;
  const int64_t R = scales.size(0), nb = scales.size(1);
  if (!matrix_ok(codes, R, 16 * nb, codes) || !matrix_ok(scales, R, nb, codes)) return std::nullopt;
  if (K < 0) K = 32 * nb;
  if ((K + 31) / 32 != nb) return std::nullopt;
  const c10::cuda::CUDAGuard guard(codes.device());
  Tensor out = empty({R, K}, bf16 ? at::kBFloat16 : at::kFloat, codes);
  if (mxfp4_dequantize(codes.data_ptr<uint8_t>(), scales.data_ptr<uint8_t>(), R, K, out.data_ptr(), dtype_of(out),
                       current_stream(codes)) != NVFP4_OK)
    return std::nullopt;
  return out;
}

// codes [N, 16 B], scales [N, B] of a weight
std::optional<Tensor> linear(const Tensor& x, const Tensor& codes, const Tensor& scales, int act, bool a4) {
  int64_t ld;
  const int dt = dtype_of(x);
  if (dt < 0 || recorded(x) || !rows_ok(x, ld) || scales.dim() != 2 || codes.scalar_type() != at::kByte) return std::nullopt;
  const int64_t N = scales.size(0), nb = scales.size(1);
  if (!matrix_ok(codes, N, 16 * nb, codes) || !matrix_ok(scales, N, nb, codes)) return std::nullopt;
  if (x.size(1) != 32 * nb || x.get_device() != codes.get_device()) return std::nullopt;
  if (x.size(0) > INT32_MAX || N > INT32_MAX || 32 * nb > INT32_MAX) return std::nullopt;
  const mxfp4_weight weight{codes.data_ptr<uint8_t>(), scales.data_ptr<uint8_t>(), (int32_t)N, (int32_t)(32 * nb)};
  const mxfp4_weight* const w = &weight;
  const c10::cuda::CUDAGuard guard(x.device());
  const int32_t T = (int32_t)x.size(0);
  const size_t need = a4 ? mxfp4_linear_a4_workspace_bytes(T, w, act) : mxfp4_linear_workspace_bytes(T, w, act);
  if (need == 0) return std::nullopt;  // refused
  Tensor y = empty({T, act ? w->N / 2 : w->N}, x.scalar_type(), x), ws;
  if (need > 256) ws = bytes(need, x);
  void* const wp = ws.defined() ? ws.data_ptr() : nullptr;
  const auto call = a4 ? mxfp4_linear_a4 : mxfp4_linear;
  if (call(x.data_ptr(), dt, ld, T, w, act, y.data_ptr(), wp, need, current_stream(x)) != NVFP4_OK) return std::nullopt;
  return y;
}

bool ffn_weights(const Tensor& x, const Tensor& gate, const Tensor& up, const Tensor& down, int act, int64_t& ld,
                 gated_ffn_weights& f) {
  const int dt = dtype_of(x);
  if ((dt != NVFP4DENSE_BF16 && dt != NVFP4DENSE_F16) || !rows_ok(x, ld) || gate.dim() != 2) return false;
  const int64_t I = gate.size(0), H = gate.size(1);
  if (x.size(0) > INT32_MAX || I > INT32_MAX || H > INT32_MAX || x.size(1) != H) return false;
  if (!matrix_ok(gate, I, H, x) || !matrix_ok(up, I, H, x) || !matrix_ok(down, H, I, x)) return false;
  f = gated_ffn_weights{gate.data_ptr(), up.data_ptr(), down.data_ptr(), (int32_t)H, (int32_t)I, act, dt};
  return true;
}

// (y, what is kept: empty without `save`)
std::optional<std::tuple<Tensor, Tensor>> ffn_forward_both(const Tensor& x, const Tensor& gate, const Tensor& up,
                                                           const Tensor& down, int act, bool save) {
  int64_t ld;
  gated_ffn_weights f;
  if (!ffn_weights(x, gate, up, down, act, ld, f)) return std::nullopt;
  if (!save && (recorded(x) || recorded(gate) || recorded(up) || recorded(down))) return std::nullopt;
  const c10::cuda::CUDAGuard guard(x.device());
  const int32_t T = (int32_t)x.size(0);
  const size_t need = save ? gated_ffn_saved_bytes(T, &f) : gated_ffn_forward_workspace_bytes(T, &f);
  if (need == 0) return std::nullopt;
  Tensor y = empty({T, f.H}, x.scalar_type(), x), ws = bytes(need, x);
  if (gated_ffn_forward(x.data_ptr(), ld, T, &f, y.data_ptr(), save ? ws.data_ptr() : nullptr,
                        save ? nullptr : ws.data_ptr(), save ? 0 : ws.numel(), current_stream(x)) != NVFP4_OK)
    return std::nullopt;
  return std::make_tuple(std::move(y), save ? std::move(ws) : Tensor());
}

std::optional<Gradients> ffn_backward(const Tensor& dy, const Tensor& x, const Tensor& gate, const Tensor& up, const Tensor& down,
                        const Tensor& saved, int act, bool need_dx, bool need_dgate, bool need_dup, bool need_ddown) {
  int64_t ld, lddy;
  gated_ffn_weights f;
  if (!ffn_weights(x, gate, up, down, act, ld, f) || !rows_ok(dy, lddy)) return std::nullopt;
  const int32_t T = (int32_t)x.size(0);
  if (dy.size(0) != T || dy.size(1) != f.H || dy.scalar_type() != x.scalar_type() || dy.get_device() != x.get_device())
    return std::nullopt;
  const size_t kept = gated_ffn_saved_bytes(T, &f), need = gated_ffn_backward_workspace_bytes(T, &f);
  if (need == 0 || !saved.is_cuda() || saved.scalar_type() != at::kByte || saved.get_device() != x.get_device() ||
      saved.dim() != 1 || !saved.is_contiguous() || saved.numel() != (int64_t)std::max<size_t>(kept, 256))
    return std::nullopt;
  const c10::cuda::CUDAGuard guard(x.device());
  const Tensor ws = bytes(need, x);
  const Tensor* like[] = {&x, &gate, &up, &down};
  const bool needs[] = {need_dx, need_dgate, need_dup, need_ddown};
  std::optional<Tensor> out[4];
  void* p[4] = {};
  for (int i = 0; i < 4; ++i)
    if (needs[i]) {
      out[i] = empty(like[i]->sizes(), x.scalar_type(), x);
      p[i] = out[i]->data_ptr();
    }
  if (gated_ffn_backward(dy.data_ptr(), lddy, x.data_ptr(), ld, saved.data_ptr(), T, &f, p[0], p[1], p[2], p[3],
                         ws.data_ptr(), ws.numel(), current_stream(x)) != NVFP4_OK)
    return std::nullopt;
  return Gradients(out[0], out[1], out[2], out[3]);
}

// An allocation that fails is the Python steps' to report, with torch's own error.
template <typename R, typename... A>
std::optional<R> attempt(std::optional<R> (*f)(A...), std::type_identity_t<A>... a) {
  const py::gil_scoped_release release;
  try {
    return f(a...);
  } catch (const c10::Error&) {
    return std::nullopt;
  }
}
template <typename R, typename... A>
auto guarded(std::optional<R> (*f)(A...)) {
  return [f](A... a) { return attempt(f, a...); };
}

// y, or (y, saved)
py::object ffn_forward(const Tensor& x, const Tensor& gate, const Tensor& up, const Tensor& down, int act, bool save) {
  auto out = attempt(&ffn_forward_both, x, gate, up, down, act, save);
  if (!out) return py::none();
  if (save) return py::cast(std::move(*out));
  return py::cast(std::move(std::get<0>(*out)));
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  m.def("quantize", guarded(&quantize));
  m.def("dequantize", guarded(&dequantize));
  m.def("linear", guarded(&linear));
  m.def("ffn_forward", &ffn_forward);
  m.def("ffn_backward", guarded(&ffn_backward));
}
