// The Python binding of the indexer's operators: checks and marshals torch tensors, in C++ because a call from
// Python through ctypes took three to five times as long as the small kernels themselves (a decode step's
// operators: 16 to 25 us of host time each). All work runs in the C entry points of indexer_ops.h; nothing falls
// back to torch. Errors: TypeError and ValueError for arguments, the package's TopkError for a status.

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/graph_task.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>
#include <unordered_set>
#include <utility>
#include <vector>

#include "indexer_ops.h"

namespace {

namespace py = pybind11;
using at::ScalarType;
using at::Tensor;
using Stream = std::optional<int64_t>;  // a cudaStream_t; none: torch's current stream

struct StatusError : std::runtime_error {
  using std::runtime_error::runtime_error;
};

template <typename... Args>
std::string text(const Args&... args) {
  std::ostringstream s;
  (s << ... << args);
  return s.str();
}

void require(bool ok, const char* message) {
  if (!ok) throw py::value_error(message);
}

void check_status(int status, const char* what) {
  if (status == TOPK_OK) return;
  std::string m = text(what, ": ", topk_status_string(status));
  if (status == TOPK_ERR_CUDA) m += text(" (cudaError ", topk_last_cuda_error(), ")");
  throw StatusError(m);
}

// A tensor of one type on a CUDA device, and on x's where x is given.
void check_tensor(const Tensor& t, const char* name, ScalarType type, const Tensor* x = nullptr) {
  if (t.scalar_type() != type) throw py::type_error(text(name, " must be ", type, ", got ", t.scalar_type()));
  if (!t.is_cuda()) throw py::value_error(text(name, " must be on a CUDA device (the library has no CPU path)"));
  if (x != nullptr && t.device() != x->device())
    throw py::value_error(text(name, " is on ", t.device(), ", expected ", x->device()));
}

int dtype_of(const Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case ScalarType::BFloat16: return INDEXER_BF16;
    case ScalarType::Half: return INDEXER_FP16;
    case ScalarType::Float: return INDEXER_FP32;
    default: throw py::type_error(text(name, " must be BFloat16, Half or Float, got ", t.scalar_type()));
  }
}

void check_contiguous(const Tensor& t, const char* name, ScalarType type, at::IntArrayRef shape, const Tensor& x) {
  check_tensor(t, name, type, &x);
  if (t.sizes() != shape || !t.is_contiguous())
    throw py::value_error(text(name, " must be contiguous, of shape ", shape, ", got ", t.sizes()));
}

// A contiguous vector of n values.
void check_vector(const Tensor& t, const char* name, ScalarType type, int64_t n, const Tensor& x) {
  check_tensor(t, name, type, &x);
  if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    throw py::value_error(text(name, " must be a contiguous vector of length ", n));
}

// No operator has a forward-mode derivative: a tangent is refused, not dropped. Nor, `backward` says, has this
// one a backward: an input that asks for a gradient is refused, not detached. Most tensors carry nothing that
// could say either, and are done with after one look: the others' questions would cost each call 0.1 to 0.3 us.
void check_autograd(std::initializer_list<const Tensor*> tensors, bool backward) {
  for (const Tensor* t : tensors) {
    if (t == nullptr || t->unsafeGetTensorImpl()->autograd_meta() == nullptr) continue;
    if (c10::AutogradState::get_tls_state().get_fw_grad_mode() && t->_fw_grad(/*level=*/0).defined())
      throw py::value_error("no forward-mode derivative: a tensor of the call carries a tangent");
    if (!backward && t->requires_grad() && at::GradMode::is_enabled())
      throw py::value_error("no gradient: a tensor of the call requires one (detach it, or call under torch.no_grad())");
  }
}

const Tensor* given(const std::optional<Tensor>& t) { return t ? &*t : nullptr; }

// [tokens, dim] or [tokens, heads, dim] with unit column stride.
struct Rows {
  int dtype;
  int64_t tokens, heads, dim, ts, hs;
};

Rows rows_of(const Tensor& x, const char* name) {
  Rows r;
  r.dtype = dtype_of(x, name);
  if (!x.is_cuda()) throw py::value_error(text(name, " must be on a CUDA device (the library has no CPU path)"));
  if ((x.dim() != 2 && x.dim() != 3) || (x.size(-1) > 1 && x.stride(-1) != 1))
    throw py::value_error(text(name, " must be [tokens, dim] or [tokens, heads, dim] with unit inner stride"));
  const bool heads = x.dim() == 3;
  r.tokens = x.size(0);
  r.heads = heads ? x.size(1) : 1;
  r.dim = x.size(-1);
  r.ts = x.stride(0);
  r.hs = heads ? x.stride(1) : 0;
  require(r.tokens <= INT32_MAX && r.heads <= INT32_MAX && r.dim <= 65536,
          "at most 2**31 - 1 tokens and heads, and rows of 65536 columns");
  return r;
}

cudaStream_t stream_of(const Stream& stream, const Tensor& x) {
  return stream ? reinterpret_cast<cudaStream_t>(*stream) : c10::cuda::getCurrentCUDAStream(x.device().index()).stream();
}

// An output. Of a call on a stream of the caller's it comes from that stream's memory: a block of the current
// stream's may still be in use by work queued there, which `stream` is not behind. The current stream, where
// the caller goes on, counts as a user of it: work queued there holds the block when the caller lets go of it.
Tensor fresh(at::IntArrayRef shape, ScalarType type, const Tensor& x, const Stream& stream) {
  // straight from the caching allocator: at::empty's way through the dispatcher takes longer than the checks
  if (!stream) return at::detail::empty_cuda(shape, type, x.device(), std::nullopt);
  const c10::DeviceIndex device = x.device().index();
  const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(device);
  const c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal(stream_of(stream, x), device));
  Tensor t = at::detail::empty_cuda(shape, type, x.device(), std::nullopt);
  t.record_stream(current);
  return t;
}

// A tensor of the caller's that a call has written: autograd is told, for the sake of operations that saved it.
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// A node of a gradient graph from before that was made on the default stream would take a captured backward there, which no
// capture can hold, and torch ends the process over it. So a differentiable call under capture is refused if one of its
// leaves has such a node already; and a captured backward, whatever the call's inputs were made from, if one of the nodes
// that it goes on to is one.
constexpr const char* kHeldGraph = "capture: a tensor of the call still belongs to a gradient graph of the default stream (let go of its results first)";

bool on_default_stream(torch::autograd::Node& node) {
  const auto stream = node.stream();
  return stream && stream->id() == c10::cuda::getDefaultCUDAStream(stream->device_index()).unwrap().id();
}

bool capturing(const Tensor& t) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  return cudaStreamIsCapturing(stream_of(Stream(), t), &status) == cudaSuccess && status != cudaStreamCaptureStatusNone;
}

void check_capture(std::initializer_list<const Tensor*> tensors) {
  bool known = false;
  for (const Tensor* t : tensors) {
    if (t == nullptr || !t->requires_grad() || !t->is_leaf()) continue;
    if (!known && !capturing(*t)) return;
    known = true;
    const auto node = torch::autograd::impl::try_get_grad_accumulator(*t);
    if (node != nullptr && on_default_stream(*node)) throw py::value_error(kHeldGraph);
  }
}

// In a backward, before it launches anything.
void check_captured_backward(const Tensor& grad) {
  if (!capturing(grad)) return;
  const auto here = torch::autograd::get_current_node();
  const auto* wanted = torch::autograd::get_current_graph_task_exec_info();  // empty: all nodes run
  if (here == nullptr) return;
  std::vector<torch::autograd::Node*> open = {here.get()};
  std::unordered_set<torch::autograd::Node*> seen = {here.get()};
  while (!open.empty()) {
    torch::autograd::Node* const node = open.back();
    open.pop_back();
    for (const auto& edge : node->next_edges()) {
      torch::autograd::Node* const next = edge.function.get();
      if (next == nullptr || !seen.insert(next).second) continue;
      if (wanted != nullptr && !wanted->empty()) {
        const auto found = wanted->find(next);
        if (found == wanted->end() || !found->second.should_execute()) continue;
      }
      if (on_default_stream(*next)) throw py::value_error(kHeldGraph);
      open.push_back(next);
    }
  }
}

// ---------------------------------------------------------------- rotary positions

// axes: undefined where there is one position a token.
void run_rotary(const Tensor& x, const Rows& r, const Tensor& positions, const Tensor& freqs, const Tensor& axes, int layout,
                int64_t start, double scale, bool transpose, const Tensor& out, const Stream& stream) {
  const c10::cuda::CUDAGuard guard(x.device());
  if (axes.defined()) {
    check_status(indexer_rotary_axes(x.data_ptr(), r.ts, r.hs, positions.data_ptr<int32_t>(), positions.stride(0),
                                     static_cast<int32_t>(positions.size(0)), axes.data_ptr<int32_t>(),
                                     freqs.data_ptr<double>(), r.dtype, r.tokens, static_cast<int32_t>(r.heads),
                                     static_cast<int32_t>(r.dim), static_cast<int32_t>(2 * freqs.size(0)),
                                     static_cast<int32_t>(start), layout, static_cast<float>(scale), transpose ? 1 : 0,
                                     out.data_ptr(), out.stride(0), out.dim() == 3 ? out.stride(1) : 0,
                                     stream_of(stream, x)),
                 "indexer_rotary_axes");
    return;
  }
  check_status(indexer_rotary(x.data_ptr(), r.ts, r.hs, positions.data_ptr<int32_t>(), freqs.data_ptr<double>(), r.dtype,
                              r.tokens, static_cast<int32_t>(r.heads), static_cast<int32_t>(r.dim),
                              static_cast<int32_t>(2 * freqs.size(0)), static_cast<int32_t>(start), layout,
                              static_cast<float>(scale), transpose ? 1 : 0, out.data_ptr(), out.stride(0),
                              out.dim() == 3 ? out.stride(1) : 0, stream_of(stream, x)),
               "indexer_rotary");
}

// The rotation is linear in x: its gradient is the transposed rotation, by this same function.
struct Rotary : torch::autograd::Function<Rotary> {
  static Tensor forward(torch::autograd::AutogradContext* ctx, const Tensor& x, const Tensor& positions,
                        const Tensor& freqs, const std::optional<Tensor>& axes_given, int64_t layout, int64_t start,
                        double scale, bool transpose) {
    const Tensor axes = axes_given ? *axes_given : Tensor();
    ctx->save_for_backward({positions, freqs, axes});
    ctx->saved_data["layout"] = layout;
    ctx->saved_data["start"] = start;
    ctx->saved_data["scale"] = scale;
    ctx->saved_data["transpose"] = transpose;
    Tensor out = fresh(x.sizes(), x.scalar_type(), x, Stream());
    run_rotary(x, rows_of(x, "x"), positions, freqs, axes, static_cast<int>(layout), start, scale, transpose, out, Stream());
    return out;
  }

  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads) {
    Tensor grad = grads[0];
    if (grad.defined()) {
      check_captured_backward(grad);
      if (grad.size(-1) > 1 && grad.stride(-1) != 1) grad = grad.contiguous();
      const auto saved = ctx->get_saved_variables();
      const std::optional<Tensor> axes = saved[2].defined() ? std::optional<Tensor>(saved[2]) : std::nullopt;
      grad = Rotary::apply(grad, saved[0], saved[1], axes, ctx->saved_data["layout"].toInt(),
                           ctx->saved_data["start"].toInt(), ctx->saved_data["scale"].toDouble(),
                           !ctx->saved_data["transpose"].toBool());
    }
    return {grad, Tensor(), Tensor(), Tensor(), Tensor(), Tensor(), Tensor(), Tensor()};
  }
};

// The span of memory of a tensor, in bytes.
std::pair<uintptr_t, uintptr_t> span_of(const Tensor& t) {
  int64_t last = 0;
  for (int64_t i = 0; i < t.dim(); ++i) last += (t.size(i) - 1) * t.stride(i);
  const uintptr_t at = reinterpret_cast<uintptr_t>(t.data_ptr());
  return {at, at + static_cast<uintptr_t>((last + 1) * t.element_size())};
}

Tensor rotary(const Tensor& x, const Tensor& positions, const Tensor& freqs, int layout, int64_t start, double scale,
              bool transpose, const std::optional<Tensor>& axes_given, const std::optional<Tensor>& out, const Stream& stream) {
  const Rows r = rows_of(x, "x");
  const Tensor axes = axes_given ? *axes_given : Tensor();
  if (axes.defined()) {
    check_tensor(positions, "positions", ScalarType::Int, &x);
    if (positions.dim() != 2 || positions.size(0) < 1 || positions.size(0) > INT32_MAX || positions.size(1) != r.tokens ||
        (r.tokens > 1 && positions.stride(1) != 1))
      throw py::value_error(text("positions must be [axes, ", r.tokens, "] with unit inner stride"));
  } else {
    check_vector(positions, "positions", ScalarType::Int, r.tokens, x);
  }
  check_tensor(freqs, "freqs", ScalarType::Double, &x);
  require(freqs.dim() == 1 && freqs.size(0) >= 1 && (freqs.size(0) == 1 || freqs.stride(0) == 1),
          "freqs must be a contiguous fp64 vector of at least one frequency");
  if (start < 0 || start > r.dim || 2 * freqs.size(0) > r.dim - start)
    throw py::value_error(text("columns [", start, ", ", start + 2 * freqs.size(0), ") do not lie within the row of ", r.dim));
  if (axes.defined()) check_vector(axes, "axes", ScalarType::Int, freqs.size(0), x);
  check_autograd({&x, given(out)}, true);
  const bool recording = at::GradMode::is_enabled();
  if (recording && x.requires_grad()) {
    require(!out && !stream, "a differentiable call takes neither out nor stream");
    check_capture({&x});
    return Rotary::apply(x, positions, freqs, axes_given, static_cast<int64_t>(layout), start, scale, transpose);
  }
  Tensor y;
  if (out) {
    y = *out;
    check_tensor(y, "out", x.scalar_type(), &x);
    require(y.sizes() == x.sizes() && (r.dim <= 1 || y.stride(-1) == 1), "out must have x's shape and unit inner stride");
    require(!(recording && y.requires_grad()), "out must not require a gradient");
    if (x.numel() > 0 && !(y.data_ptr() == x.data_ptr() && y.strides() == x.strides())) {
      const auto a = span_of(x), b = span_of(y);
      require(a.first >= b.second || b.first >= a.second, "out must be x itself or not overlap it");
    }
  } else {
    y = fresh(x.sizes(), x.scalar_type(), x, stream);
  }
  run_rotary(x, r, positions, freqs, axes, layout, start, scale, transpose, y, stream);
  if (out) written(y);
  return y;
}

// ---------------------------------------------------------------- layer norm

Tensor run_norm(const Tensor& x, const Tensor& weight, const Tensor& bias, double eps, Tensor out, float* stats,
                const Stream& stream) {
  const Rows r = rows_of(x, "x");
  const c10::cuda::CUDAGuard guard(x.device());
  check_status(indexer_layer_norm(x.data_ptr(), r.ts, r.hs, r.dtype, r.tokens, static_cast<int32_t>(r.heads),
                                  static_cast<int32_t>(r.dim), weight.data_ptr(), bias.defined() ? bias.data_ptr() : nullptr,
                                  dtype_of(weight, "weight"), static_cast<float>(eps), out.data_ptr(), stats,
                                  stream_of(stream, x)),
               "indexer_layer_norm");
  return out;
}

struct LayerNorm : torch::autograd::Function<LayerNorm> {
  static Tensor forward(torch::autograd::AutogradContext* ctx, const Tensor& x, const Tensor& weight,
                        const std::optional<Tensor>& bias_given, double eps) {
    const Tensor bias = bias_given ? *bias_given : Tensor();
    ctx->saved_data["bias"] = bias.defined();
    Tensor stats = fresh({x.numel() / x.size(-1), 2}, ScalarType::Float, x, Stream());
    ctx->save_for_backward({x, weight, stats});
    return run_norm(x, weight, bias, eps, fresh(x.sizes(), x.scalar_type(), x, Stream()), stats.data_ptr<float>(), Stream());
  }

  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads) {
    if (!grads[0].defined()) return {Tensor(), Tensor(), Tensor(), Tensor()};
    require(!at::GradMode::is_enabled(), "indexer_layer_norm has no second derivative: call backward without create_graph");
    check_captured_backward(grads[0]);
    const auto saved = ctx->get_saved_variables();
    const Tensor &x = saved[0], &weight = saved[1], &stats = saved[2];
    Tensor grad = grads[0];
    if (grad.size(-1) > 1 && grad.stride(-1) != 1) grad = grad.contiguous();
    const Rows r = rows_of(x, "x"), g = rows_of(grad, "grad");
    const auto wanted = [&](size_t i, at::IntArrayRef shape, ScalarType type) {
      return ctx->needs_input_grad(i) ? fresh(shape, type, x, Stream()) : Tensor();
    };
    Tensor dx = wanted(0, x.sizes(), x.scalar_type());
    Tensor dw = wanted(1, weight.sizes(), weight.scalar_type()), db;
    if (ctx->saved_data["bias"].toBool()) db = wanted(2, weight.sizes(), weight.scalar_type());
    const c10::cuda::CUDAGuard guard(x.device());
    const int32_t heads = static_cast<int32_t>(r.heads), dim = static_cast<int32_t>(r.dim);
    size_t bytes = 0;
    Tensor workspace;
    if (dw.defined() || db.defined()) {
      bytes = indexer_layer_norm_grad_workspace_bytes(r.tokens, heads, dim);
      workspace = fresh({static_cast<int64_t>(bytes)}, ScalarType::Byte, x, Stream());
    }
    const auto at = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    check_status(indexer_layer_norm_grad(x.data_ptr(), r.ts, r.hs, grad.data_ptr(), g.ts, g.hs, r.dtype, r.tokens, heads, dim,
                                         weight.data_ptr(), dtype_of(weight, "weight"), stats.data_ptr<float>(), at(dx),
                                         at(dw), at(db), at(workspace), bytes, stream_of(Stream(), x)),
                 "indexer_layer_norm_grad");
    return {dx, dw, db, Tensor()};
  }
};

Tensor layer_norm(const Tensor& x, const Tensor& weight, const std::optional<Tensor>& bias_given, double eps,
                  const std::optional<Tensor>& out, const Stream& stream) {
  const Rows r = rows_of(x, "x");
  const Tensor bias = bias_given ? *bias_given : Tensor();
  require(r.dim >= 1, "rows must have at least one column");
  require(eps >= 0.0 && eps <= 3.0e38, "eps must be a finite number, at least 0");
  if (weight.scalar_type() != x.scalar_type() && weight.scalar_type() != ScalarType::Float)
    throw py::type_error(text("weight must be ", x.scalar_type(), " or Float, got ", weight.scalar_type()));
  check_vector(weight, "weight", weight.scalar_type(), r.dim, x);
  if (bias.defined()) check_vector(bias, "bias", weight.scalar_type(), r.dim, x);
  check_autograd({&x, &weight, bias.defined() ? &bias : nullptr, given(out)}, true);
  const bool recording = at::GradMode::is_enabled();
  if (recording && (x.requires_grad() || weight.requires_grad() || (bias.defined() && bias.requires_grad()))) {
    require(!out && !stream, "a differentiable call takes neither out nor stream");
    check_capture({&x, &weight, bias.defined() ? &bias : nullptr});
    return LayerNorm::apply(x, weight, bias_given, eps);
  }
  if (!out) return run_norm(x, weight, bias, eps, fresh(x.sizes(), x.scalar_type(), x, stream), nullptr, stream);
  check_contiguous(*out, "out", x.scalar_type(), x.sizes(), x);
  require(!(recording && out->requires_grad()), "out must not require a gradient");
  if (x.numel() > 0) {
    const auto a = span_of(x), b = span_of(*out);
    require(a.first >= b.second || b.first >= a.second, "out must not overlap x");
  }
  run_norm(x, weight, bias, eps, *out, nullptr, stream);
  written(*out);
  return *out;
}

// ---------------------------------------------------------------- 8-bit rows and cache

int64_t blocks_of(int64_t dim) { return (dim + INDEXER_BLOCK - 1) / INDEXER_BLOCK; }

std::pair<Tensor, Tensor> quantise(const Tensor& x, int format, const std::optional<Tensor>& weights,
                                   const std::optional<Tensor>& codes, const std::optional<Tensor>& scales,
                                   const Stream& stream) {
  const Rows r = rows_of(x, "x");
  require(r.dim >= 1, "rows must have at least one column");
  check_autograd({&x, given(weights), given(codes), given(scales)}, false);
  const int64_t nb = blocks_of(r.dim);
  c10::SmallVector<int64_t, 4> shape(x.sizes().begin(), x.sizes().end() - 1);
  if (weights) {
    if (nb != 1)
      throw py::value_error(text("weights need rows of one block (at most ", INDEXER_BLOCK, " columns), got ", r.dim));
    check_contiguous(*weights, "weights", ScalarType::Float, shape, x);
  } else {
    shape.push_back(nb);
  }
  if (codes) check_contiguous(*codes, "codes", ScalarType::Float8_e4m3fn, x.sizes(), x);
  if (scales) check_contiguous(*scales, "scales", ScalarType::Float, shape, x);
  Tensor c = codes ? *codes : fresh(x.sizes(), ScalarType::Float8_e4m3fn, x, stream);
  Tensor s = scales ? *scales : fresh(shape, ScalarType::Float, x, stream);
  const c10::cuda::CUDAGuard guard(x.device());
  check_status(indexer_quantise(x.data_ptr(), r.ts, r.hs, r.dtype, r.tokens, static_cast<int32_t>(r.heads),
                                static_cast<int32_t>(r.dim), format, weights ? weights->data_ptr<float>() : nullptr,
                                static_cast<uint8_t*>(c.data_ptr()), s.data_ptr<float>(), stream_of(stream, x)),
               "indexer_quantise");
  if (codes) written(c);
  if (scales) written(s);
  return {c, s};
}

// Rows apart from each other: pages outside rows, or rows outside pages.
void check_apart(const Tensor& t, const char* name, int64_t width) {
  int a = t.stride(0) < t.stride(1) ? 0 : 1;
  for (int i = 0; i < 2; ++i, a = 1 - a) {
    if (t.size(a) <= 1) continue;
    if (t.stride(a) < width) throw py::value_error(text(name, ": rows must not overlap"));
    width += (t.size(a) - 1) * t.stride(a);
  }
}

indexer_cache_t cache_of(const Tensor& codes, const Tensor& scales, const Tensor* x) {
  check_tensor(codes, "codes", ScalarType::Float8_e4m3fn, x);
  check_tensor(scales, "scales", ScalarType::Float, &codes);
  require(codes.dim() == 3 && codes.size(2) >= 1 && codes.size(2) <= 65536 && (codes.size(2) == 1 || codes.stride(2) == 1),
          "codes must be [pages, page_size, dim] with unit inner stride");
  const int64_t pages = codes.size(0), size = codes.size(1), dim = codes.size(2), nb = blocks_of(dim);
  if (scales.dim() != 3 || scales.size(0) != pages || scales.size(1) != size || scales.size(2) != nb ||
      (nb > 1 && scales.stride(2) != 1))
    throw py::value_error(text("scales must be [", pages, ", ", size, ", ", nb, "] (one for each ", INDEXER_BLOCK,
                               " columns) with unit inner stride"));
  require(size >= 1, "a page must hold at least one row");
  require(size <= INT32_MAX && pages <= INT32_MAX / size, "a cache holds at most 2**31 - 1 rows");
  check_apart(codes, "codes", dim);
  check_apart(scales, "scales", nb);
  indexer_cache_t c = {};
  c.codes = static_cast<uint8_t*>(codes.data_ptr());
  c.scales = scales.data_ptr<float>();
  c.num_pages = pages;
  c.code_page_stride = codes.stride(0);
  c.code_token_stride = codes.stride(1);
  c.scale_page_stride = scales.stride(0);
  c.scale_token_stride = scales.stride(1);
  c.page_size = static_cast<int32_t>(size);
  c.dim = static_cast<int32_t>(dim);
  return c;
}

void cache_write(const Tensor& x, const Tensor& slots, const Tensor& codes, const Tensor& scales, int format,
                 const Stream& stream) {
  const Rows r = rows_of(x, "x");
  require(x.dim() == 2, "x must be [tokens, dim]");
  const indexer_cache_t cache = cache_of(codes, scales, &x);
  if (r.dim != cache.dim) throw py::value_error(text("x has rows of ", r.dim, " columns, the cache ", cache.dim));
  check_vector(slots, "slots", ScalarType::Int, r.tokens, x);
  check_autograd({&x, &codes, &scales}, false);
  const c10::cuda::CUDAGuard guard(x.device());
  check_status(indexer_cache_write(x.data_ptr(), r.ts, r.dtype, r.tokens, slots.data_ptr<int32_t>(), format, &cache,
                                   stream_of(stream, x)),
               "indexer_cache_write");
  written(codes);
  written(scales);
}

Tensor cache_read(const Tensor& codes, const Tensor& scales, const Tensor& slots, int dtype, const std::optional<Tensor>& out,
                  const Stream& stream) {
  constexpr ScalarType kTypes[] = {ScalarType::BFloat16, ScalarType::Half, ScalarType::Float};
  const indexer_cache_t cache = cache_of(codes, scales, nullptr);
  check_tensor(slots, "slots", ScalarType::Int, &codes);
  require(slots.is_contiguous(), "slots must be contiguous");
  check_autograd({&codes, &scales, given(out)}, false);
  c10::SmallVector<int64_t, 4> shape(slots.sizes().begin(), slots.sizes().end());
  shape.push_back(cache.dim);
  if (out) check_contiguous(*out, "out", kTypes[dtype], shape, codes);
  Tensor y = out ? *out : fresh(shape, kTypes[dtype], codes, stream);
  const c10::cuda::CUDAGuard guard(codes.device());
  check_status(indexer_cache_read(&cache, slots.data_ptr<int32_t>(), slots.numel(), dtype, y.data_ptr(),
                                  stream_of(stream, codes)),
               "indexer_cache_read");
  if (out) written(y);
  return y;
}

// ---------------------------------------------------------------- scores

Tensor scores(const Tensor& q, const Tensor& weights, const Tensor& codes, const Tensor& scales, const Tensor& page_table,
              const Tensor& seq_lens, int64_t row_len, const std::optional<Tensor>& out, const Stream& stream) {
  check_tensor(q, "q", ScalarType::Float8_e4m3fn);
  require(q.dim() == 4 && q.size(3) == INDEXER_SCORE_DIM && q.is_contiguous(),
          "q must be a contiguous [batch, queries, heads, 128] tensor");
  const int64_t batch = q.size(0), queries = q.size(1), heads = q.size(2);
  if (heads < 1 || heads > INDEXER_MAX_HEADS)
    throw py::value_error(text("heads must be in [1, ", INDEXER_MAX_HEADS, "], got ", heads));
  require(batch <= INT32_MAX && queries <= INT32_MAX && (batch == 0 || queries <= INT32_MAX / batch),
          "at most 2**31 - 1 queries");
  check_contiguous(weights, "weights", ScalarType::Float, {batch, queries, heads}, q);
  const indexer_cache_t cache = cache_of(codes, scales, &q);
  if (cache.dim != INDEXER_SCORE_DIM)
    throw py::value_error(text("the cache's rows must have ", INDEXER_SCORE_DIM, " columns, got ", cache.dim));
  require(((reinterpret_cast<uintptr_t>(q.data_ptr()) | reinterpret_cast<uintptr_t>(cache.codes) |
            static_cast<uintptr_t>(cache.num_pages > 1 ? cache.code_page_stride : 0) |
            static_cast<uintptr_t>(cache.page_size > 1 ? cache.code_token_stride : 0)) & 15u) == 0,
          "q and every row of codes must start on 16 bytes");
  if (row_len < 1 || row_len > INT32_MAX) throw py::value_error(text("row_len must be in [1, 2**31 - 1], got ", row_len));
  check_tensor(page_table, "page_table", ScalarType::Int, &q);
  require(page_table.dim() == 2 && page_table.size(0) == batch && (page_table.size(1) <= 1 || page_table.stride(1) == 1),
          "page_table must be [batch, pages] int32 with unit inner stride");
  require(page_table.size(1) >= (row_len + cache.page_size - 1) / cache.page_size, "page_table has too few pages for the rows");
  const int64_t pt_stride = batch > 1 ? page_table.stride(0) : page_table.size(1);
  require(pt_stride >= page_table.size(1), "page_table rows must not overlap (use .contiguous() on expanded tables)");
  check_contiguous(seq_lens, "seq_lens", ScalarType::Int, {batch, queries}, q);
  const int64_t shape[2] = {batch * queries, row_len};
  if (out) check_contiguous(*out, "out", ScalarType::Float, shape, q);
  check_autograd({&q, &weights, &codes, &scales, given(out)}, false);
  Tensor y = out ? *out : fresh(shape, ScalarType::Float, q, stream);
  const c10::cuda::CUDAGuard guard(q.device());
  check_status(indexer_scores(static_cast<const uint8_t*>(q.data_ptr()), weights.data_ptr<float>(), &cache,
                              page_table.data_ptr<int32_t>(), pt_stride, seq_lens.data_ptr<int32_t>(),
                              static_cast<int32_t>(batch), static_cast<int32_t>(queries), static_cast<int32_t>(heads), row_len,
                              y.data_ptr<float>(), stream_of(stream, q)),
               "indexer_scores");
  if (out) written(y);
  return y;
}

// ---------------------------------------------------------------- caches of heads, with scales of blocks of tokens

// Rows of `width` along the first three axes apart from each other, whatever their order.
void check_apart3(const Tensor& t, const char* name, int64_t width) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return t.stride(a) < t.stride(b); });
  for (const int a : order) {
    if (t.size(a) <= 1) continue;
    if (t.stride(a) < width) throw py::value_error(text(name, ": rows must not overlap"));
    width += (t.size(a) - 1) * t.stride(a);
  }
}

indexer_block_cache_t block_cache_of(const Tensor& codes, const Tensor& scales, const Tensor& x, const char* codes_name,
                                     const char* scales_name) {
  check_tensor(codes, codes_name, ScalarType::Float8_e4m3fn, &x);
  check_tensor(scales, scales_name, ScalarType::Float, &x);
  if (codes.dim() != 4 || codes.size(1) < 1 || codes.size(2) < 1 || codes.size(3) < 16 || codes.size(3) % 16 != 0 ||
      codes.size(3) > INDEXER_MAX_HEAD_DIM || codes.stride(3) != 1)
    throw py::value_error(text(codes_name, " must be [pages, page_size, heads, dim] with unit inner stride, dim a multiple of 16, at most ",
                               INDEXER_MAX_HEAD_DIM));
  const int64_t pages = codes.size(0), size = codes.size(1), heads = codes.size(2), dim = codes.size(3);
  if (scales.dim() != 3 || scales.size(0) != pages || scales.size(1) < 1 || size % scales.size(1) != 0 || scales.size(2) != heads)
    throw py::value_error(text(scales_name, " must be [", pages, ", blocks, ", heads, "] with blocks a divisor of the page size ", size));
  require(size <= INT32_MAX && pages <= INT32_MAX / size && heads <= INT32_MAX, "a cache holds at most 2**31 - 1 rows");
  for (int a = 0; a < 3; ++a)
    if (codes.size(a) > 1 && codes.stride(a) % 16 != 0) throw py::value_error(text(codes_name, ": every row must start on 16 bytes"));
  if ((reinterpret_cast<uintptr_t>(codes.data_ptr()) & 15u) != 0)
    throw py::value_error(text(codes_name, ": every row must start on 16 bytes"));
  check_apart3(codes, codes_name, dim);
  check_apart3(scales, scales_name, 1);
  indexer_block_cache_t c = {};
  c.codes = static_cast<uint8_t*>(codes.data_ptr());
  c.scales = scales.data_ptr<float>();
  c.num_pages = pages;
  c.code_page_stride = codes.stride(0), c.code_token_stride = codes.stride(1), c.code_head_stride = codes.stride(2);
  c.scale_page_stride = scales.stride(0), c.scale_block_stride = scales.stride(1), c.scale_head_stride = scales.stride(2);
  c.page_size = static_cast<int32_t>(size);
  c.block = static_cast<int32_t>(size / scales.size(1));
  c.heads = static_cast<int32_t>(heads);
  c.dim = static_cast<int32_t>(dim);
  return c;
}

// A row's stride of an int32 [rows, width] tensor with unit inner stride.
int64_t index_stride_of(const Tensor& t, const char* name, int64_t rows, const Tensor& x) {
  check_tensor(t, name, ScalarType::Int, &x);
  if (t.dim() != 2 || t.size(0) != rows || (t.size(1) > 1 && t.stride(1) != 1))
    throw py::value_error(text(name, " must be [", rows, ", width] int32 with unit inner stride"));
  if (rows <= 1) return t.size(1);
  if (t.stride(0) < t.size(1)) throw py::value_error(text(name, " rows must not overlap (use .contiguous() on expanded tables)"));
  return t.stride(0);
}

void cache_append(const Tensor& x, const Tensor& starts, const Tensor& seq_lens, const Tensor& page_table, const Tensor& codes,
                  const Tensor& scales, const Stream& stream) {
  const Rows r = rows_of(x, "x");
  require(x.dim() == 3, "x must be [tokens, heads, dim]");
  const indexer_block_cache_t cache = block_cache_of(codes, scales, x, "codes", "scales");
  if (r.heads != cache.heads || r.dim != cache.dim)
    throw py::value_error(text("x has ", r.heads, " heads of ", r.dim, " columns, the cache ", cache.heads, " of ", cache.dim));
  check_tensor(seq_lens, "seq_lens", ScalarType::Int, &x);
  require(seq_lens.dim() == 1, "seq_lens must be a contiguous vector");
  const int64_t batch = seq_lens.size(0);
  require(r.tokens <= (INT64_C(1) << 30) && batch <= (1 << 28) && r.tokens / cache.block + 2 * batch <= INT32_MAX / cache.heads,
          "too many rows or sequences for one call");
  check_vector(seq_lens, "seq_lens", ScalarType::Int, batch, x);
  check_vector(starts, "starts", ScalarType::Int, batch + 1, x);
  const int64_t pt_stride = index_stride_of(page_table, "page_table", batch, x);
  check_autograd({&x, &codes, &scales}, false);
  const c10::cuda::CUDAGuard guard(x.device());
  check_status(indexer_cache_append(x.data_ptr(), r.ts, r.hs, r.dtype, r.tokens, starts.data_ptr<int32_t>(),
                                    seq_lens.data_ptr<int32_t>(), page_table.data_ptr<int32_t>(), pt_stride,
                                    page_table.size(1), static_cast<int32_t>(batch), &cache, stream_of(stream, x)),
               "indexer_cache_append");
  written(codes);
  written(scales);
}

// The output, and log(sum of weights) where it is asked for.
std::pair<Tensor, std::optional<Tensor>> attention(const Tensor& q, const Tensor& k_codes, const Tensor& k_scales,
                                                   const Tensor& v_codes, const Tensor& v_scales,
                                                   const std::optional<Tensor>& page_table, const std::optional<Tensor>& seq_lens,
                                                   const std::optional<Tensor>& slots, std::optional<double> softmax_scale,
                                                   bool return_lse, const std::optional<Tensor>& out, const Stream& stream) {
  if (q.scalar_type() != ScalarType::BFloat16 && q.scalar_type() != ScalarType::Half)
    throw py::type_error(text("q must be BFloat16 or Half, got ", q.scalar_type()));
  require(q.is_cuda(), "q must be on a CUDA device (the library has no CPU path)");
  require(q.dim() == 4 && q.is_contiguous(), "q must be a contiguous [batch, queries, heads, dim] tensor");
  const indexer_block_cache_t keys = block_cache_of(k_codes, k_scales, q, "k_codes", "k_scales");
  const indexer_block_cache_t values = block_cache_of(v_codes, v_scales, q, "v_codes", "v_scales");
  require(k_codes.sizes() == v_codes.sizes(), "k_codes and v_codes must be of one shape");
  const int64_t batch = q.size(0), queries = q.size(1), heads = q.size(2);
  if (q.size(3) != keys.dim || heads < 1 || heads % keys.heads != 0)
    throw py::value_error(text("q has ", heads, " heads of ", q.size(3), " columns, the cache ", keys.heads, " of ", keys.dim,
                               ": the columns must be as many, the heads a multiple"));
  require(batch <= INT32_MAX && (batch == 0 || queries <= INT32_MAX / batch) && heads <= INT32_MAX &&
              queries <= (1 << 30) / (heads / keys.heads),
          "too many queries for one call");
  require((reinterpret_cast<uintptr_t>(q.data_ptr()) & 15u) == 0, "q must start on 16 bytes");
  if (slots.has_value() == page_table.has_value() || slots.has_value() == seq_lens.has_value())
    throw py::value_error("give slots, or page_table and seq_lens");
  const Tensor& index = slots ? *slots : *page_table;
  const int64_t stride = slots ? index_stride_of(index, "slots", batch * queries, q) : index_stride_of(index, "page_table", batch, q);
  require(index.size(1) <= INT32_MAX - 65536, "at most 2**31 - 65537 slots or pages a row");
  if (seq_lens) check_contiguous(*seq_lens, "seq_lens", ScalarType::Int, {batch, queries}, q);
  const double scale = softmax_scale ? *softmax_scale : 1.0 / std::sqrt(static_cast<double>(keys.dim));
  require(scale > -1.0e38 && scale < 1.0e38, "softmax_scale must be a finite number");
  if (out) {
    check_contiguous(*out, "out", q.scalar_type(), q.sizes(), q);
    require((reinterpret_cast<uintptr_t>(out->data_ptr()) & 15u) == 0, "out must start on 16 bytes");
    if (q.numel() > 0) {
      const auto a = span_of(q), b = span_of(*out);
      require(a.first >= b.second || b.first >= a.second, "out must not overlap q");
    }
  }
  check_autograd({&q, &k_codes, &k_scales, &v_codes, &v_scales, given(out)}, false);
  Tensor y = out ? *out : fresh(q.sizes(), q.scalar_type(), q, stream);
  std::optional<Tensor> lse;
  if (return_lse) lse = fresh({batch, queries, heads}, ScalarType::Float, q, stream);
  if (batch == 0 || queries == 0) return {y, lse};
  const c10::cuda::CUDAGuard guard(q.device());
  const size_t bytes = indexer_attention_workspace_bytes(static_cast<int32_t>(queries), static_cast<int32_t>(heads), keys.heads,
                                                         keys.dim, slots ? 1 : 0);
  const Tensor workspace = fresh({static_cast<int64_t>(bytes)}, ScalarType::Byte, q, stream);
  check_status(indexer_attention(q.data_ptr(), dtype_of(q, "q"), &keys, &values, index.data_ptr<int32_t>(), stride, index.size(1),
                                 seq_lens ? seq_lens->data_ptr<int32_t>() : nullptr, static_cast<int32_t>(batch),
                                 static_cast<int32_t>(queries), static_cast<int32_t>(heads), static_cast<float>(scale),
                                 y.data_ptr(), lse ? lse->data_ptr<float>() : nullptr, workspace.data_ptr(), bytes,
                                 stream_of(stream, q)),
               "indexer_attention");
  if (out) written(y);
  return {y, lse};
}

}  // namespace

PYBIND11_MODULE(indexer_binding, m) {
  static PyObject* topk_error = PyExc_RuntimeError;
  m.def("set_error", [](py::object type) { topk_error = type.release().ptr(); });
  py::register_exception_translator([](std::exception_ptr p) {
    try {
      if (p) std::rethrow_exception(p);
    } catch (const StatusError& e) {
      PyErr_SetString(topk_error, e.what());
    }
  });
  m.def("rotary", &rotary);
  m.def("layer_norm", &layer_norm);
  m.def("quantise", &quantise);
  m.def("cache_write", &cache_write);
  m.def("cache_read", &cache_read);
  m.def("scores", &scores);
  m.def("cache_append", &cache_append);
  m.def("attention", &attention);
}
