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
#include <torch/csrc/utils/pybind.h>

#include <initializer_list>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>
#include <utility>

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

// ---------------------------------------------------------------- rotary positions

void run_rotary(const Tensor& x, const Rows& r, const Tensor& positions, const Tensor& freqs, int layout, int64_t start,
                double scale, bool transpose, const Tensor& out, const Stream& stream) {
  const c10::cuda::CUDAGuard guard(x.device());
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
                        const Tensor& freqs, int64_t layout, int64_t start, double scale, bool transpose) {
    ctx->save_for_backward({positions, freqs});
    ctx->saved_data["layout"] = layout;
    ctx->saved_data["start"] = start;
    ctx->saved_data["scale"] = scale;
    ctx->saved_data["transpose"] = transpose;
    Tensor out = fresh(x.sizes(), x.scalar_type(), x, Stream());
    run_rotary(x, rows_of(x, "x"), positions, freqs, static_cast<int>(layout), start, scale, transpose, out, Stream());
    return out;
  }

  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads) {
    Tensor grad = grads[0];
    if (grad.defined()) {
      if (grad.size(-1) > 1 && grad.stride(-1) != 1) grad = grad.contiguous();
      const auto saved = ctx->get_saved_variables();
      grad = Rotary::apply(grad, saved[0], saved[1], ctx->saved_data["layout"].toInt(), ctx->saved_data["start"].toInt(),
                           ctx->saved_data["scale"].toDouble(), !ctx->saved_data["transpose"].toBool());
    }
    return {grad, Tensor(), Tensor(), Tensor(), Tensor(), Tensor(), Tensor()};
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
              bool transpose, const std::optional<Tensor>& out, const Stream& stream) {
  const Rows r = rows_of(x, "x");
  check_vector(positions, "positions", ScalarType::Int, r.tokens, x);
  check_tensor(freqs, "freqs", ScalarType::Double, &x);
  require(freqs.dim() == 1 && freqs.size(0) >= 1 && (freqs.size(0) == 1 || freqs.stride(0) == 1),
          "freqs must be a contiguous fp64 vector of at least one frequency");
  if (start < 0 || start > r.dim || 2 * freqs.size(0) > r.dim - start)
    throw py::value_error(text("columns [", start, ", ", start + 2 * freqs.size(0), ") do not lie within the row of ", r.dim));
  check_autograd({&x, given(out)}, true);
  const bool recording = at::GradMode::is_enabled();
  if (recording && x.requires_grad()) {
    require(!out && !stream, "a differentiable call takes neither out nor stream");
    return Rotary::apply(x, positions, freqs, static_cast<int64_t>(layout), start, scale, transpose);
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
  run_rotary(x, r, positions, freqs, layout, start, scale, transpose, y, stream);
  if (out) written(y);
  return y;
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
  m.def("quantise", &quantise);
  m.def("cache_write", &cache_write);
  m.def("cache_read", &cache_read);
  m.def("scores", &scores);
}
