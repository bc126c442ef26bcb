// Compiled binding of the serving operators: argument checks, memory and one
// C-ABI call each. In C++ since a decode step makes several such calls of a
// few microseconds.
#include "serve_binding.h"

#include <c10/hip/HIPStream.h>
#include <dlfcn.h>

#include <cmath>
#include <optional>

#include "fp8lin_serve.h"
#include "serve_overlap.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;

#define SERVE_ENTRIES(X)                                                                                          \
  X(fp8_status_str) X(fp8_cache_codes_bytes) X(fp8_cache_scales_bytes) X(fp8_cache_append) X(fp8_cache_read)      \
  X(fp8_cache_attention_workspace_bytes) X(fp8_cache_attention) X(fp4_codes_bytes) X(fp4_scales_bytes)            \
  X(fp4_quantize) X(fp4_dequantize) X(fp4_linear_bytes) X(fp4_linear_fwd_cached)
struct Api {
#define X(name) decltype(&::name) name;
  SERVE_ENTRIES(X)
#undef X
  void open(void* library) {
#define X(entry)                                   \
  entry = (decltype(entry))dlsym(library, #entry); \
  if (!entry) throw py::import_error("libfp8lin lacks " #entry);
    SERVE_ENTRIES(X)
#undef X
  }
};
Api api;

void check(fp8_status s, const char* what) {
  if (s != FP8_OK)
    throw std::runtime_error(std::string(what) + ": " + api.fp8_status_str(s) + " (status " + std::to_string((int)s) + ")");
}
hipStream_t stream_of(const Tensor& t) { return c10::hip::getCurrentHIPStream(t.get_device()).stream(); }
void* ptr(const Tensor& t) { return t.numel() ? t.data_ptr() : nullptr; }

std::string shape_of(const Tensor& t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "]";
}
[[noreturn]] void refuse(const std::string& why) { throw py::value_error(why); }
void want(bool ok, const char* name, const char* what) {
  if (!ok) refuse(std::string(name) + " must be " + what);
}
// These operators serve: a gradient or a tangent would be lost in them.
void no_grad(const Tensor& t, const char* name) {
  if ((at::GradMode::is_enabled() && t.requires_grad()) || t._fw_grad(0).defined()) {
    PyErr_SetString(PyExc_NotImplementedError,
                    (std::string(name) + " wants a gradient: the serving operators have none (use torch.no_grad())").c_str());
    throw py::error_already_set();
  }
}
// A tensor that a call wrote: a backward that saved it finds out by its version
void wrote(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void on(const Tensor& t, const Tensor& like, const char* name) {
  if (t.device() != like.device()) refuse(std::string(name) + " must be on " + like.device().str() + ", got " + t.device().str());
}
void on_device(const Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a device tensor (no CPU path exists)");
}
void bf16(const Tensor& t, const char* name) {
  want(t.scalar_type() == at::kBFloat16, name, "bfloat16");
}
void ints(const Tensor& t, const char* name) {
  want(t.scalar_type() == at::kInt, name, "int32");
}

// A cache's data: codes of the keys, of the values, then the scales
fp8_cache cache_of(const Tensor& data, int64_t pages, int64_t page_tokens, int64_t heads, int64_t head_dim) {
  const size_t codes = api.fp8_cache_codes_bytes(pages, (int)page_tokens, (int)heads, (int)head_dim);
  const size_t scales = api.fp8_cache_scales_bytes(pages, (int)page_tokens, (int)heads, (int)head_dim);
  if (data.scalar_type() != at::kByte || !data.is_contiguous() || (size_t)data.numel() != 2 * codes + scales)
    refuse("the cache's data must be " + std::to_string(2 * codes + scales) + " contiguous bytes (uint8)");
  uint8_t* p = (uint8_t*)ptr(data);
  return {p, p + codes, p + 2 * codes, pages, (int32_t)page_tokens, (int32_t)heads, (int32_t)head_dim};
}

fp8_cache_batch batch_of(const Tensor& tables, const Tensor& lengths, const Maybe& starts, int64_t tokens) {
  ints(tables, "tables");
  ints(lengths, "lengths");
  want(lengths.dim() == 1 && lengths.is_contiguous(), "lengths", "1-D and contiguous");
  const int64_t n = lengths.size(0);
  if (tables.dim() != 2 || tables.size(0) != n)
    refuse("tables must be [" + std::to_string(n) + ", pages of a sequence], got " + shape_of(tables));
  want(tables.size(1) <= 1 || tables.stride(1) == 1, "tables", "of contiguous rows");
  if (starts) {
    ints(*starts, "starts");
    if (starts->dim() != 1 || starts->size(0) != n + 1 || !starts->is_contiguous())
      refuse("starts must be contiguous [" + std::to_string(n + 1) + "], got " + shape_of(*starts));
  } else if (tokens != n) {
    refuse("without starts a batch has one row a sequence: " + std::to_string(n) + ", got " + std::to_string(tokens));
  }
  return {(const int32_t*)ptr(tables), tables.size(0) > 1 ? tables.stride(0) : 0, tables.size(1),
          (const int32_t*)ptr(lengths), starts ? (const int32_t*)starts->data_ptr() : nullptr, n, tokens};
}
void batch_on(const Tensor& tables, const Tensor& lengths, const Maybe& starts, const Tensor& like) {
  on(tables, like, "tables");
  on(lengths, like, "lengths");
  if (starts) on(*starts, like, "starts");
}

fp8_cache_rows rows_of(const Tensor& t, int64_t tokens, int64_t heads, int64_t head_dim, const char* name, bool output) {
  bf16(t, name);
  if (t.dim() != 3 || t.size(0) != tokens || (heads >= 0 && t.size(1) != heads) || t.size(2) != head_dim)
    refuse(std::string(name) + " must be [" + std::to_string(tokens) + ", " + (heads < 0 ? "heads" : std::to_string(heads)) +
           ", " + std::to_string(head_dim) + "], got " + shape_of(t));
  want(t.stride(2) == 1, name, "of contiguous last dimension");
  if (output && ((t.size(0) > 1 && t.stride(0) == 0) || (t.size(1) > 1 && t.stride(1) == 0)))
    refuse(std::string(name) + " must not be expanded: it is written");
  return {ptr(t), t.stride(0), t.stride(1)};
}
fp8lin::RowSet set_of(const Tensor& t) {
  return {ptr(t), t.size(0), t.size(1), t.size(2), t.stride(0), t.stride(1)};
}
// An output that the caller gives, against an input of the same call
void apart(const Tensor& out, const char* name, const Tensor& in, const char* other, bool or_itself) {
  const fp8lin::RowSet a = set_of(out), b = set_of(in);
  if (or_itself && fp8lin::same_rows(a, b)) return;
  if (fp8lin::overlap(a, b))
    refuse(std::string(name) + " must " + (or_itself ? std::string("be ") + other + " itself or " : "") + "not overlap " + other);
}
void apart(const Tensor& out, const char* name) {
  if (fp8lin::overlaps_itself(set_of(out))) refuse(std::string(name) + " must not overlap itself: it is written");
}
void q_heads_of(const Tensor& q, int64_t heads) {
  if (q.dim() == 3 && (q.size(1) == 0 || q.size(1) % heads))
    refuse("q has " + std::to_string(q.size(1)) + " heads: not a multiple of the cache's " + std::to_string(heads));
}

Maybe append(const Tensor& data, int64_t pages, int64_t page_tokens, int64_t heads, int64_t head_dim, const Tensor& k,
             const Tensor& v, const Tensor& tables, const Tensor& lengths, const Maybe& starts, const Maybe& q,
             const Maybe& freqs, bool interleaved, const Maybe& q_out) {
  const fp8_cache c = cache_of(data, pages, page_tokens, heads, head_dim);
  const int64_t tokens = k.dim() ? k.size(0) : 0;
  const fp8_cache_rows rk = rows_of(k, tokens, heads, head_dim, "k", false), rv = rows_of(v, tokens, heads, head_dim, "v", false);
  const fp8_cache_batch b = batch_of(tables, lengths, starts, tokens);
  int rot = 0;
  if (freqs) {
    want(freqs->scalar_type() == at::kFloat && freqs->dim() == 1 && freqs->is_contiguous(), "freqs", "float32, 1-D and contiguous");
    rot = (int)std::min<int64_t>(2 * freqs->size(0), 1 << 20);
    if (rot % 16 || rot > head_dim)
      refuse("freqs must be half as many as the rotated dimensions, a multiple of 16 up to " + std::to_string(head_dim) +
             ", got " + std::to_string(freqs->size(0)));
  }
  if (q_out && !q) refuse("q_out without q");
  fp8_cache_rows rq = {nullptr, 0, 0}, ro = {nullptr, 0, 0};
  int q_heads = 0;
  if (q) {
    rq = rows_of(*q, tokens, -1, head_dim, "q", false);
    q_heads_of(*q, heads);
    q_heads = (int)q->size(1);
    if (q_out) {
      ro = rows_of(*q_out, tokens, q_heads, head_dim, "q_out", true);
      apart(*q_out, "q_out");
      apart(*q_out, "q_out", *q, "q", true);
      apart(*q_out, "q_out", k, "k", false);
      apart(*q_out, "q_out", v, "v", false);
    }
  }
  no_grad(k, "k");
  no_grad(v, "v");
  if (q) no_grad(*q, "q");
  if (freqs) no_grad(*freqs, "freqs");
  if (q_out) no_grad(*q_out, "q_out");
  on_device(data, "cache");
  on(k, data, "k");
  on(v, data, "v");
  batch_on(tables, lengths, starts, data);
  if (freqs) on(*freqs, data, "freqs");
  Maybe out;
  if (q) {
    on(*q, data, "q");
    if (q_out) on(*q_out, data, "q_out");
    out = q_out ? *q_out : at::empty({tokens, q_heads, head_dim}, q->options());
    ro = {ptr(*out), out->stride(0), out->stride(1)};
  }
  check(api.fp8_cache_append(&c, &b, &rk, &rv, &rq, &ro, q_heads, freqs ? (const float*)ptr(*freqs) : nullptr, rot, interleaved,
                             stream_of(data)),
        "fp8_cache_append");
  wrote(data);
  if (q_out) wrote(*q_out);
  return out;
}

std::pair<Tensor, Tensor> read_back(const Tensor& data, int64_t pages, int64_t page_tokens, int64_t heads, int64_t head_dim,
                                    const Tensor& tables, const Tensor& lengths, const Maybe& starts, int64_t tokens,
                                    const Maybe& k, const Maybe& v) {
  const fp8_cache c = cache_of(data, pages, page_tokens, heads, head_dim);
  if (tokens < 0) refuse("tokens must not be negative");
  const fp8_cache_batch b = batch_of(tables, lengths, starts, tokens);
  if (k) {
    rows_of(*k, tokens, heads, head_dim, "k", true);
    apart(*k, "k");
  }
  if (v) {
    rows_of(*v, tokens, heads, head_dim, "v", true);
    apart(*v, "v");
  }
  if (k && v) apart(*k, "k", *v, "v", false);
  if (k) no_grad(*k, "k");
  if (v) no_grad(*v, "v");
  on_device(data, "cache");
  batch_on(tables, lengths, starts, data);
  if (k) on(*k, data, "k");
  if (v) on(*v, data, "v");
  const auto options = data.options().dtype(at::kBFloat16);
  const Tensor ko = k ? *k : at::empty({tokens, heads, head_dim}, options);
  const Tensor vo = v ? *v : at::empty({tokens, heads, head_dim}, options);
  const fp8_cache_rows rk = {ptr(ko), ko.stride(0), ko.stride(1)}, rv = {ptr(vo), vo.stride(0), vo.stride(1)};
  check(api.fp8_cache_read(&c, &b, &rk, &rv, stream_of(data)), "fp8_cache_read");
  if (k) wrote(*k);
  if (v) wrote(*v);
  return {ko, vo};
}

std::pair<Tensor, Maybe> attention(const Tensor& data, int64_t pages, int64_t page_tokens, int64_t heads, int64_t head_dim,
                                   const Tensor& q, const Tensor& tables, const Tensor& lengths, const Maybe& starts,
                                   double scale, double softcap, int64_t window, bool with_lse, const Maybe& given) {
  const fp8_cache c = cache_of(data, pages, page_tokens, heads, head_dim);
  const int64_t tokens = q.dim() ? q.size(0) : 0;
  const fp8_cache_rows rq = rows_of(q, tokens, -1, head_dim, "q", false);
  q_heads_of(q, heads);
  const int64_t q_heads = q.size(1);
  const fp8_cache_batch b = batch_of(tables, lengths, starts, tokens);
  if (given) {
    rows_of(*given, tokens, q_heads, head_dim, "out", true);
    apart(*given, "out");
    apart(*given, "out", q, "q", true);
  }
  if (!(softcap == 0 || (softcap >= 0x1p-64 && softcap <= 0x1p64))) refuse("softcap must be 0 or between 2^-64 and 2^64");
  if (!(std::fabs(scale) <= 0x1p64)) refuse("scale must be finite, up to 2^64");
  if (window < 0 || window > INT32_MAX) refuse("window must be between 0 and 2^31 - 1");
  no_grad(q, "q");
  if (given) no_grad(*given, "out");
  on_device(data, "cache");
  on(q, data, "q");
  batch_on(tables, lengths, starts, data);
  if (given) on(*given, data, "out");
  const Tensor out = given ? *given : at::empty({tokens, q_heads, head_dim}, q.options());
  const fp8_cache_rows ro = {ptr(out), out.stride(0), out.stride(1)};
  Maybe lse;
  if (with_lse) lse = at::empty({tokens, q_heads}, q.options().dtype(at::kFloat));
  const size_t n = api.fp8_cache_attention_workspace_bytes(&c, &b, (int)q_heads);
  Tensor ws;
  if (n) ws = at::empty({(int64_t)n}, data.options());
  check(api.fp8_cache_attention(&c, &b, &rq, (int)q_heads, (float)scale, (float)softcap, (int)window, &ro,
                                lse ? (float*)ptr(*lse) : nullptr, n ? ws.data_ptr() : nullptr, n, stream_of(data)),
        "fp8_cache_attention");
  if (given) wrote(*given);
  return {out, lse};
}

// A 4-bit weight in one allocation: codes, then scales.
struct Stored4 {
  uint8_t *codes, *scales;
  Stored4(const Tensor& data, int64_t K, int64_t N) {
    const size_t n = api.fp4_codes_bytes(K, N), s = api.fp4_scales_bytes(K, N);
    if (K < 0 || N < 0 || data.scalar_type() != at::kByte || !data.is_contiguous() || (size_t)data.numel() != n + s)
      refuse("a stored 4-bit [" + std::to_string(K) + ", " + std::to_string(N) + "] must be " + std::to_string(n + s) +
             " contiguous bytes (uint8)");
    codes = (uint8_t*)ptr(data);
    scales = codes + n;
  }
};
void matrix(const Tensor& t, const char* name) {
  bf16(t, name);
  want(t.dim() == 2, name, "2-D");
  want(t.stride(1) == 1 || t.size(1) <= 1, name, "of contiguous rows");
}

Tensor fp4_store(const Tensor& W) {
  matrix(W, "W");
  on_device(W, "W");
  const int64_t K = W.size(0), N = W.size(1);
  const Tensor data = at::empty({(int64_t)(api.fp4_codes_bytes(K, N) + api.fp4_scales_bytes(K, N))}, W.options().dtype(at::kByte));
  if (K && N && !data.numel()) refuse("W is too large: at most 2^20 rows and 2^23 columns");
  const Stored4 q(data, K, N);
  check(api.fp4_quantize(ptr(W), W.stride(0), K, N, q.codes, q.scales, stream_of(W)), "fp4_quantize");
  return data;
}

Tensor fp4_restore(const Tensor& data, int64_t K, int64_t N) {
  const Stored4 q(data, K, N);
  on_device(data, "data");
  const Tensor W = at::empty({K, N}, data.options().dtype(at::kBFloat16));
  check(api.fp4_dequantize(q.codes, q.scales, K, N, ptr(W), N, stream_of(data)), "fp4_dequantize");
  return W;
}

Tensor fp4_serve(const Tensor& X, const Tensor& data, int64_t K, int64_t N, const Maybe& given, bool exact) {
  matrix(X, "X");
  if (X.size(1) != K)
    refuse("X " + shape_of(X) + " does not go with the stored weight [" + std::to_string(K) + ", " + std::to_string(N) + "]");
  const Stored4 w(data, K, N);
  const int64_t M = X.size(0);
  if (given) {
    bf16(*given, "Y");
    if (given->dim() != 2 || given->size(0) != M || given->size(1) != N || !given->is_contiguous())
      refuse("Y must be contiguous [" + std::to_string(M) + ", " + std::to_string(N) + "], got " + shape_of(*given));
    // X is read until the last workgroup ends
    const char *x0 = (const char*)ptr(X), *y0 = (const char*)ptr(*given);
    if (x0 && y0 && x0 < y0 + 2 * M * N && y0 < x0 + 2 * ((M - 1) * X.stride(0) + K)) refuse("Y must not overlap X");
  }
  no_grad(X, "X");
  if (given) no_grad(*given, "Y");
  on_device(X, "X");
  on(data, X, "w");
  if (given) on(*given, X, "Y");
  const Tensor Y = given ? *given : at::empty({M, N}, X.options());
  const size_t n = api.fp4_linear_bytes(M, K, N);
  Tensor scratch;
  if (n) scratch = at::empty({(int64_t)n}, data.options());
  check(api.fp4_linear_fwd_cached(ptr(X), X.stride(0), M, K, N, w.codes, w.scales, exact, n ? scratch.data_ptr() : nullptr, n, ptr(Y),
                                  stream_of(X)),
        "fp4_linear_fwd_cached");
  if (given) wrote(*given);
  return Y;
}

}  // namespace

void bind_serve(py::module_& m, void* library) {
  api.open(library);
  m.def("cache_append", &append);
  m.def("cache_read", &read_back);
  m.def("cache_attention", &attention);
  m.def("fp4_store", &fp4_store);
  m.def("fp4_restore", &fp4_restore);
  m.def("fp4_serve", &fp4_serve);
}
