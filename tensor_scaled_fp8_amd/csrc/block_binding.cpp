// The block-scaled operators' autograd nodes and their calls of few
// microseconds (store, restore, serve): argument layout, memory and one
// C-ABI call each. A backward runs on autograd's device thread; as Python
// there it took 40 us a call more than an empty one where that thread ran on
// another part of the chip than the caller's, since every object it touches
// then moves between their caches.
#include <c10/hip/HIPStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/extension.h>

#include <optional>

#include "fp8lin.h"
#include "serve_binding.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::tensor_list;

// The entry points, of the library that the package has loaded (FP8LIN_LIB may
// name another than the one beside this file: linked with that, one process
// would compute with two).
#define FP8LIN_ENTRIES(X) \
  X(fp8_block_dequantize) X(fp8_block_linear_bwd) X(fp8_block_linear_bytes) X(fp8_block_linear_cached_bytes) \
  X(fp8_block_linear_few) X(fp8_block_linear_fwd) X(fp8_block_linear_fwd_cached) X(fp8_block_linear_fwd_few) \
  X(fp8_block_mlp_bwd) X(fp8_block_mlp_bytes) X(fp8_block_mlp_fwd) X(fp8_block_quantize) X(fp8_status_str) \
  X(fp8_swiglu_bwd) X(fp8_swiglu_fwd) X(fp8_swiglu_kept_bytes)
struct Api {
#define X(name) decltype(&::name) name;
  FP8LIN_ENTRIES(X)
#undef X
  void open(void* library) {
#define X(entry)                                            \
  entry = (decltype(entry))dlsym(library, #entry);          \
  if (!entry) throw py::import_error("libfp8lin lacks " #entry);
    FP8LIN_ENTRIES(X)
#undef X
  }
};
Api api;

void check(fp8_status s, const char* what) {
  if (s != FP8_OK) throw std::runtime_error(std::string(what) + ": " + api.fp8_status_str(s) + " (status " + std::to_string((int)s) + ")");
}
hipStream_t stream_of(const Tensor& t) { return c10::hip::getCurrentHIPStream(t.get_device()).stream(); }

// t [..., n] bf16 as a matrix with contiguous rows, a view where it can be
struct Rows {
  Tensor t;
  int64_t ld, rows, cols;
  explicit Rows(const Tensor& x) : t(x) {
    if (t.dim() != 2) {
      const auto s = t.sizes();
      int64_t n = 1;
      for (size_t i = 0; i + 1 < s.size(); ++i) n *= s[i];
      t = t.reshape({n, s.back()});
    }
    rows = t.size(0);
    cols = t.size(1);
    if (t.stride(1) != 1 && cols > 1) t = t.contiguous();
    ld = t.stride(0);
  }
  const void* p() const { return t.data_ptr(); }
};
Rows grad_rows(const Tensor& dy) { return Rows(dy.scalar_type() == at::kBFloat16 ? dy : dy.to(at::kBFloat16)); }

Tensor space(size_t n, const Tensor& like) { return at::empty({(int64_t)n}, like.options().dtype(at::kByte)); }
Tensor make(at::IntArrayRef shape, const Tensor& like) { return at::empty(shape, like.options().dtype(at::kBFloat16)); }
void* ptr(const Tensor& t) { return t.defined() && t.numel() ? t.data_ptr() : nullptr; }

// A graph of the gradients themselves (create_graph, which is when a backward
// runs with gradients enabled) is refused when it is used: the kernels'
// results would be taken for constants. Whether the incoming gradient wants
// one does not matter (a sum's is an expanded constant): the results depend on
// the forward's operands too, and some of those do, or there would be no node.
tensor_list once(tensor_list out) {
  if (!at::GradMode::is_enabled()) return out;
  for (Tensor& t : out)
    if (t.defined()) t = t.detach().set_requires_grad(true);
  auto err = std::make_shared<torch::autograd::DelayedError>(
      "trying to differentiate twice a function that was marked with @once_differentiable", (int64_t)out.size());
  return (*err)(std::move(out));
}

int flag(const Tensor& t, int f) { return t.requires_grad() ? f : 0; }

struct Linear : torch::autograd::Function<Linear> {
  static Tensor forward(AutogradContext* ctx, const Tensor& X, const Tensor& W) {
    const int flags = flag(X, FP8_BLOCK_NEED_DX) | flag(W, FP8_BLOCK_NEED_DW);
    const Rows x(X), w(W);
    const int64_t M = x.rows, K = x.cols, N = w.cols;
    size_t nk, nf, nb;
    check(api.fp8_block_linear_bytes(M, K, N, flags, &nk, &nf, &nb), "fp8_block_linear_bytes");
    const Tensor kept = space(nk, X), scratch = space(nf, X);
    auto shape = X.sizes().vec();
    shape.back() = N;
    Tensor Y = make(shape, X);
    check(api.fp8_block_linear_fwd(x.p(), x.ld, w.p(), w.ld, M, K, N, flags, ptr(kept), nk, ptr(scratch), nf, Y.data_ptr(),
                               stream_of(X)),
          "fp8_block_linear_fwd");
    ctx->save_for_backward({kept});
    ctx->saved_data["flags"] = (int64_t)flags;
    ctx->saved_data["X"] = X.sizes().vec();
    ctx->saved_data["N"] = N;
    return Y;
  }
  static tensor_list backward(AutogradContext* ctx, const tensor_list& grads) {
    const Tensor kept = ctx->get_saved_variables()[0];
    const int flags = (int)ctx->saved_data["flags"].toInt();
    const auto shape = ctx->saved_data["X"].toIntVector();
    const Rows dy = grad_rows(grads[0]);
    const int64_t M = dy.rows, K = shape.back(), N = ctx->saved_data["N"].toInt();
    size_t nk, nf, nb;
    check(api.fp8_block_linear_bytes(M, K, N, flags, &nk, &nf, &nb), "fp8_block_linear_bytes");
    const Tensor scratch = space(nb, dy.t);
    Tensor dX, dW;
    if (flags & FP8_BLOCK_NEED_DX) dX = make(shape, dy.t);
    if (flags & FP8_BLOCK_NEED_DW) dW = make({K, N}, dy.t);
    check(api.fp8_block_linear_bwd(dy.p(), dy.ld, M, K, N, flags, ptr(kept), nk, ptr(scratch), nb, ptr(dX), ptr(dW),
                               stream_of(dy.t)),
          "fp8_block_linear_bwd");
    return once({dX, dW});
  }
};

struct Swiglu : torch::autograd::Function<Swiglu> {
  static Tensor forward(AutogradContext* ctx, const Tensor& gate, const Tensor& up) {
    const Rows g(gate), u(up);
    const size_t n = api.fp8_swiglu_kept_bytes(g.rows, g.cols);
    const Tensor kept = space(n, gate);
    Tensor h = make(gate.sizes(), gate);
    check(api.fp8_swiglu_fwd(g.p(), g.ld, u.p(), u.ld, g.rows, g.cols, h.data_ptr(), ptr(kept), n, stream_of(gate)),
          "fp8_swiglu_fwd");
    ctx->save_for_backward({kept});
    ctx->saved_data["need"] = (int64_t)(flag(gate, 1) | flag(up, 2));
    return h;
  }
  static tensor_list backward(AutogradContext* ctx, const tensor_list& grads) {
    const Tensor kept = ctx->get_saved_variables()[0];
    const int need = (int)ctx->saved_data["need"].toInt();
    const Rows d = grad_rows(grads[0]);
    Tensor dg, du;
    if (need & 1) dg = make(grads[0].sizes(), d.t);
    if (need & 2) du = make(grads[0].sizes(), d.t);
    check(api.fp8_swiglu_bwd(d.p(), d.ld, d.rows, d.cols, ptr(kept), (size_t)kept.numel(), ptr(dg), ptr(du), stream_of(d.t)),
          "fp8_swiglu_bwd");
    return once({dg, du});
  }
};

struct Mlp : torch::autograd::Function<Mlp> {
  static Tensor forward(AutogradContext* ctx, const Tensor& X, const Tensor& Wgu, const Tensor& Wd) {
    const int flags = flag(X, FP8_BLOCK_NEED_DX) | flag(Wgu, FP8_BLOCK_NEED_DW) | flag(Wd, FP8_BLOCK_NEED_DW2);
    const Rows x(X), g(Wgu), d(Wd);
    const int64_t M = x.rows, K = x.cols, F = d.rows;
    size_t nk, nf, nb;
    check(api.fp8_block_mlp_bytes(M, K, F, flags, &nk, &nf, &nb), "fp8_block_mlp_bytes");
    const Tensor kept = space(nk, X), scratch = space(nf, X);
    Tensor Y = make(X.sizes(), X);
    check(api.fp8_block_mlp_fwd(x.p(), x.ld, g.p(), g.ld, d.p(), d.ld, M, K, F, flags, ptr(kept), nk, ptr(scratch), nf,
                            Y.data_ptr(), stream_of(X)),
          "fp8_block_mlp_fwd");
    ctx->save_for_backward({kept});
    ctx->saved_data["flags"] = (int64_t)flags;
    ctx->saved_data["F"] = F;
    return Y;
  }
  static tensor_list backward(AutogradContext* ctx, const tensor_list& grads) {
    const Tensor kept = ctx->get_saved_variables()[0];
    const int flags = (int)ctx->saved_data["flags"].toInt();
    const Rows dy = grad_rows(grads[0]);
    const int64_t M = dy.rows, K = dy.cols, F = ctx->saved_data["F"].toInt();
    size_t nk, nf, nb;
    check(api.fp8_block_mlp_bytes(M, K, F, flags, &nk, &nf, &nb), "fp8_block_mlp_bytes");
    const Tensor scratch = space(nb, dy.t);
    Tensor dX, dWgu, dWd;
    if (flags & FP8_BLOCK_NEED_DX) dX = make(grads[0].sizes(), dy.t);
    if (flags & FP8_BLOCK_NEED_DW) dWgu = make({K, 2 * F}, dy.t);
    if (flags & FP8_BLOCK_NEED_DW2) dWd = make({F, K}, dy.t);
    check(api.fp8_block_mlp_bwd(dy.p(), dy.ld, M, K, F, flags, ptr(kept), nk, ptr(scratch), nb, ptr(dX), ptr(dWgu), ptr(dWd),
                            stream_of(dy.t)),
          "fp8_block_mlp_bwd");
    return once({dX, dWgu, dWd});
  }
};

// A stored matrix in one allocation: codes, then scales.
int64_t round_blk(int64_t n) { return (n + 127) / 128 * 128; }
struct Stored {
  Tensor data;
  uint8_t *codes, *scales;
  static int64_t bytes(int64_t rows, int64_t cols) {
    return rows * round_blk(cols) + round_blk(rows) * (round_blk(cols) / 128);
  }
  // the kernels read all of it: what is not that long is refused
  Stored(const Tensor& d, int64_t rows, int64_t cols) : data(d) {
    const int64_t n = rows < 0 || cols < 0 ? -1 : bytes(rows, cols);
    if (data.numel() != n || data.scalar_type() != at::kByte || !data.is_contiguous())
      throw py::value_error("a stored [" + std::to_string(rows) + ", " + std::to_string(cols) + "] must be " +
                            std::to_string(n) + " contiguous bytes (uint8)");
    codes = (uint8_t*)data.data_ptr();
    scales = codes + rows * round_blk(cols);
  }
  Stored(int64_t rows, int64_t cols, const Tensor& like) : Stored(space(bytes(rows, cols), like), rows, cols) {}
};

using Maybe = std::optional<Tensor>;

std::pair<Maybe, Maybe> quantize(const Tensor& x, int64_t fmt, bool rowwise, bool transposed) {
  const int64_t rows = x.size(0), cols = x.size(1);
  std::optional<Stored> q, t;
  if (rowwise) q.emplace(rows, cols, x);
  if (transposed) t.emplace(cols, rows, x);
  check(api.fp8_block_quantize(x.data_ptr(), rows, cols, x.stride(0), (fp8_fmt)fmt, q ? q->codes : nullptr,
                           q ? q->scales : nullptr, t ? t->codes : nullptr, t ? t->scales : nullptr, stream_of(x)),
        "fp8_block_quantize");
  return {q ? Maybe(q->data) : Maybe(), t ? Maybe(t->data) : Maybe()};
}

Tensor dequantize(const Tensor& data, int64_t rows, int64_t cols, int64_t fmt, const Maybe& out) {
  const Stored q(data, rows, cols);
  const Tensor o = out ? *out : make({rows, cols}, data);
  check(api.fp8_block_dequantize(q.codes, q.scales, rows, cols, (fp8_fmt)fmt, o.data_ptr(), o.stride(0), stream_of(o)),
        "fp8_block_dequantize");
  return o;
}

// Y [M, N] = X W for a stored weight (transposed form, [N, K])
Tensor serve(const Tensor& X, const Tensor& weight, int64_t N, const Maybe& out) {
  const int64_t M = X.size(0), K = X.size(1);
  const Stored w(weight, N, K);
  const Tensor Y = out ? *out : make({M, N}, X);
  if (api.fp8_block_linear_few(M, K, N)) {
    check(api.fp8_block_linear_fwd_few(X.data_ptr(), X.stride(0), M, K, N, w.codes, w.scales, Y.data_ptr(), stream_of(X)),
          "fp8_block_linear_fwd_few");
    return Y;
  }
  const size_t n = api.fp8_block_linear_cached_bytes(M, K, N);
  const Tensor scratch = space(n, X);
  check(api.fp8_block_linear_fwd_cached(X.data_ptr(), X.stride(0), M, K, N, w.codes, w.scales, ptr(scratch), n, Y.data_ptr(),
                                    stream_of(X)),
        "fp8_block_linear_fwd_cached");
  return Y;
}

}  // namespace

PYBIND11_MODULE(_block_binding, m) {
  void* library = (void*)py::module_::import("tensor_scaled_fp8_amd._lib").attr("load")().attr("_handle").cast<uintptr_t>();
  api.open(library);
  m.def("quantize", &quantize);
  m.def("dequantize", &dequantize);
  m.def("serve", &serve);
  m.def("linear", [](const Tensor& X, const Tensor& W) { return Linear::apply(X, W); });
  m.def("swiglu", [](const Tensor& gate, const Tensor& up) { return Swiglu::apply(gate, up); });
  m.def("mlp", [](const Tensor& X, const Tensor& Wgu, const Tensor& Wd) { return Mlp::apply(X, Wgu, Wd); });
  bind_serve(m, library);
}
