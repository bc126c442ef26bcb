// C-ABI entry points of the block-scaled FP8 operators: argument checks,
// the layout of the caller's workspaces, then kernel launches on the
// caller's stream. No allocation, no host synchronisation.
#include "block.h"

using namespace fp8lin;

namespace {

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool aligned2(const void* p) { return ((uintptr_t)p & 1u) == 0; }
inline bool fmt_ok(int f) { return f == FP8_E4M3 || f == FP8_E5M2; }
inline fp8_status hip_status(hipError_t e) { return e == hipSuccess ? FP8_OK : FP8_ERR_HIP; }

// 256 rows of codes are addressed with 31 bits, as is a matrix of scales
constexpr int64_t kMaxBlockDim = ((int64_t)1 << 23) - kBlk;
inline bool size_ok(int64_t r, int64_t c) {
  return r <= kMaxBlockDim && c <= kMaxBlockDim && round_blk(r) * (round_blk(c) / kBlk) < ((int64_t)1 << 31);
}

// a bf16 argument: null only when empty
inline bool bf16_ok(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  if (rows < 0 || cols < 0 || ld < 0) return false;
  return rows == 0 || cols == 0 || (p && aligned2(p));
}
inline bool codes_ok(const void* c, const void* s, int64_t rows, int64_t cols) {
  return rows == 0 || cols == 0 || (c && s && aligned16(c) && aligned16(s));
}

BlockMat mat(const void* codes, const void* scales, int64_t rows, int64_t cols) {
  return {(uint8_t*)codes, (uint8_t*)scales, round_blk(cols), round_blk(rows), rows, cols};
}
const BlockMat kNone = {nullptr, nullptr, 0, 0, 0, 0};

// Carves pieces of 256 bytes and up from a workspace; with a null base it
// only counts.
struct Carver {
  uint8_t* base;
  size_t at = 0;
  explicit Carver(void* p) : base((uint8_t*)p) {}
  uint8_t* take(size_t n) {
    uint8_t* p = base ? base + at : nullptr;
    at += (n + 255) / 256 * 256;
    return p;
  }
  BlockMat block(int64_t rows, int64_t cols) {
    uint8_t* c = take((size_t)rows * round_blk(cols));
    uint8_t* s = take((size_t)round_blk(rows) * (round_blk(cols) / kBlk));
    return mat(c, s, rows, cols);
  }
};

inline size_t most(size_t a, size_t b) { return a > b ? a : b; }

// ---- one linear: what the forward keeps for the backward, and scratch ----
struct LinearKept {
  BlockMat xt, w;  // X transposed (for dW), W's row form (for dX)
  size_t bytes;
  LinearKept(void* p, int64_t M, int64_t K, int64_t N, int flags) : xt(kNone), w(kNone) {
    Carver c(p);
    if (flags & FP8_BLOCK_NEED_DW) xt = c.block(K, M);
    if (flags & FP8_BLOCK_NEED_DX) w = c.block(K, N);
    bytes = c.at;
  }
};
struct LinearFwd {
  BlockMat x, wt;
  uint8_t* part;
  size_t part_bytes, bytes;
  LinearFwd(void* p, int64_t M, int64_t K, int64_t N, bool with_w) : wt(kNone) {
    Carver c(p);
    x = c.block(M, K);
    if (with_w) wt = c.block(N, K);
    part_bytes = block_gemm_ws_bytes(M, N, K);
    part = c.take(part_bytes);
    bytes = c.at;
  }
};
struct LinearBwd {
  BlockMat dy, dyt;
  uint8_t* part;
  size_t part_bytes, bytes;
  LinearBwd(void* p, int64_t M, int64_t K, int64_t N, int flags) : dy(kNone), dyt(kNone) {
    Carver c(p);
    if (flags & FP8_BLOCK_NEED_DX) dy = c.block(M, N);
    if (flags & FP8_BLOCK_NEED_DW) dyt = c.block(N, M);
    part_bytes = 0;
    if (flags & FP8_BLOCK_NEED_DX) part_bytes = most(part_bytes, block_gemm_ws_bytes(M, K, N));
    if (flags & FP8_BLOCK_NEED_DW) part_bytes = most(part_bytes, block_gemm_ws_bytes(K, N, M));
    part = c.take(part_bytes);
    bytes = c.at;
  }
};

inline fp8_status linear_size(int64_t M, int64_t K, int64_t N) {
  if (M < 0 || K < 0 || N < 0) return FP8_ERR_INVALID;
  return size_ok(M, K) && size_ok(K, M) && size_ok(K, N) && size_ok(N, K) && size_ok(M, N) && size_ok(N, M)
             ? FP8_OK
             : FP8_ERR_UNSUPPORTED;
}
inline bool space_ok(const void* p, size_t have, size_t need) { return need == 0 || (p && aligned16(p) && have >= need); }

struct SwigluKept {
  BlockMat g, u;
  size_t bytes;
  SwigluKept(void* p, int64_t rows, int64_t cols) {
    Carver c(p);
    g = c.block(rows, cols);
    u = c.block(rows, cols);
    bytes = c.at;
  }
};

// ---- the MLP. Blocks of the 2 F gate and up columns never straddle the
// two halves: each half starts at a block of its own (F2 = the halves'
// rounded length apart), in the weight and in the gradient alike.
inline BlockMat half(const BlockMat& b, int64_t f, int i) {
  BlockMat h = b;
  h.cols = f;
  if (b.codes) {
    h.codes += i * round_blk(f);
    h.scales += i * (round_blk(f) / kBlk) * b.srows;
  }
  return h;
}
constexpr int kMlpAll = FP8_BLOCK_NEED_DX | FP8_BLOCK_NEED_DW | FP8_BLOCK_NEED_DW2;
struct MlpKept {
  BlockMat g, u, xt, wgu, wd;
  size_t bytes;
  MlpKept(void* p, int64_t M, int64_t K, int64_t F, int flags) : g(kNone), u(kNone), xt(kNone), wgu(kNone), wd(kNone) {
    Carver c(p);
    if (flags) {
      g = c.block(M, F);
      u = c.block(M, F);
    }
    if (flags & FP8_BLOCK_NEED_DW) xt = c.block(K, M);
    if (flags & FP8_BLOCK_NEED_DX) wgu = c.block(K, 2 * round_blk(F));
    if (flags & (FP8_BLOCK_NEED_DX | FP8_BLOCK_NEED_DW)) wd = c.block(F, K);
    bytes = c.at;
  }
};
struct MlpFwd {
  BlockMat x, wgut, wdt, h;
  uint16_t* gu;
  uint8_t* part;
  size_t part_bytes, bytes;
  MlpFwd(void* p, int64_t M, int64_t K, int64_t F) {
    Carver c(p);
    x = c.block(M, K);
    wgut = c.block(2 * F, K);
    wdt = c.block(K, F);
    h = c.block(M, F);
    gu = (uint16_t*)c.take((size_t)M * 2 * F * 2);
    part_bytes = most(block_gemm_ws_bytes(M, 2 * F, K), block_gemm_ws_bytes(M, K, F));
    part = c.take(part_bytes);
    bytes = c.at;
  }
};
struct MlpBwd {
  BlockMat dy, dyt, dgu, dgut, ht;
  uint16_t* dh;
  uint8_t* part;
  size_t part_bytes, bytes;
  MlpBwd(void* p, int64_t M, int64_t K, int64_t F, int flags)
      : dy(kNone), dyt(kNone), dgu(kNone), dgut(kNone), ht(kNone) {
    const bool dx = flags & FP8_BLOCK_NEED_DX, dw = flags & FP8_BLOCK_NEED_DW, dw2 = flags & FP8_BLOCK_NEED_DW2;
    Carver c(p);
    if (dx || dw) dy = c.block(M, K);
    if (dw2) dyt = c.block(K, M), ht = c.block(F, M);
    if (dx) dgu = c.block(M, 2 * round_blk(F));
    if (dw) dgut = c.block(2 * F, M);
    dh = dx || dw ? (uint16_t*)c.take((size_t)M * F * 2) : nullptr;  // h' needs no dh
    part_bytes = 0;
    if (dx || dw) part_bytes = most(part_bytes, block_gemm_ws_bytes(M, F, K));
    if (dx) part_bytes = most(part_bytes, block_gemm_ws_bytes(M, K, 2 * round_blk(F)));
    if (dw) part_bytes = most(part_bytes, block_gemm_ws_bytes(K, 2 * F, M));
    if (dw2) part_bytes = most(part_bytes, block_gemm_ws_bytes(F, K, M));
    part = c.take(part_bytes);
    bytes = c.at;
  }
};
inline fp8_status mlp_size(int64_t M, int64_t K, int64_t F) {
  if (M < 0 || K < 0 || F < 0) return FP8_ERR_INVALID;
  const int64_t F2 = 2 * round_blk(F);
  return size_ok(M, K) && size_ok(K, M) && size_ok(K, F2) && size_ok(F2, K) && size_ok(M, F2) && size_ok(F2, M)
             ? FP8_OK
             : FP8_ERR_UNSUPPORTED;
}

#define TRY(e)                              \
  do {                                      \
    const hipError_t err_ = (e);            \
    if (err_ != hipSuccess) return FP8_ERR_HIP; \
  } while (0)

}  // namespace

extern "C" {

size_t fp8_block_codes_bytes(int64_t rows, int64_t cols) {
  return rows <= 0 || cols <= 0 ? 0 : (size_t)rows * round_blk(cols);
}
size_t fp8_block_scales_bytes(int64_t rows, int64_t cols) {
  return rows <= 0 || cols <= 0 ? 0 : (size_t)round_blk(rows) * (round_blk(cols) / kBlk);
}

fp8_status fp8_block_quantize(const void* x, int64_t rows, int64_t cols, int64_t ldx, fp8_fmt fmt, uint8_t* row_codes,
                              uint8_t* row_scales, uint8_t* t_codes, uint8_t* t_scales, hipStream_t stream) {
  if (!bf16_ok(x, rows, cols, ldx) || !fmt_ok(fmt) || !!row_codes != !!row_scales || !!t_codes != !!t_scales ||
      !aligned16(row_codes) || !aligned16(row_scales) || !aligned16(t_codes) || !aligned16(t_scales))
    return FP8_ERR_INVALID;
  if (rows > 0 && cols > 0 && !row_codes && !t_codes) return FP8_ERR_INVALID;
  if (!size_ok(rows, cols) || !size_ok(cols, rows)) return FP8_ERR_UNSUPPORTED;
  return hip_status(launch_block_quantize({(const uint16_t*)x, ldx, rows, cols}, fmt,
                                          mat(row_codes, row_scales, rows, cols), mat(t_codes, t_scales, cols, rows), 0,
                                          stream));
}

fp8_status fp8_block_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, fp8_fmt fmt,
                                void* out, int64_t ldo, hipStream_t stream) {
  if (!bf16_ok(out, rows, cols, ldo) || !fmt_ok(fmt) || !codes_ok(codes, scales, rows, cols) || (rows > 1 && ldo < cols))
    return FP8_ERR_INVALID;
  if (!size_ok(rows, cols)) return FP8_ERR_UNSUPPORTED;
  return hip_status(launch_block_dequantize(mat(codes, scales, rows, cols), fmt, (uint16_t*)out, ldo, stream));
}

size_t fp8_block_gemm_workspace_bytes(int64_t M, int64_t N, int64_t R) {
  return M < 0 || N < 0 || R < 0 ? 0 : block_gemm_ws_bytes(M, N, R);
}

fp8_status fp8_block_gemm_plan(int64_t M, int64_t N, int64_t R, int* tile_m, int* tile_n, int* splits) {
  if (M < 0 || N < 0 || R < 0) return FP8_ERR_INVALID;
  if (!size_ok(M, R) || !size_ok(N, R) || !size_ok(M, N)) return FP8_ERR_UNSUPPORTED;
  int bm, bn, s;
  block_gemm_plan(M, N, R, &bm, &bn, &s);
  if (tile_m) *tile_m = bm;
  if (tile_n) *tile_n = bn;
  if (splits) *splits = s;
  return FP8_OK;
}

fp8_status fp8_block_gemm(const uint8_t* A, const uint8_t* sA, fp8_fmt fa, const uint8_t* B, const uint8_t* sB,
                          fp8_fmt fb, int64_t M, int64_t N, int64_t R, void* C, int64_t ldc, void* ws, size_t ws_bytes,
                          hipStream_t stream) {
  if (M < 0 || N < 0 || R < 0 || !fmt_ok(fa) || !fmt_ok(fb) || !codes_ok(A, sA, M, R) || !codes_ok(B, sB, N, R) ||
      !bf16_ok(C, M, N, ldc) || (M > 1 && ldc < N) || !aligned16(ws))
    return FP8_ERR_INVALID;
  if (!size_ok(M, R) || !size_ok(N, R) || !size_ok(M, N)) return FP8_ERR_UNSUPPORTED;
  const BlockGemm g = {mat(A, sA, M, R), mat(B, sB, N, R), fa, fb, (uint16_t*)C, ldc};
  return hip_status(launch_block_gemm(g, ws, ws_bytes, stream));
}

fp8_status fp8_block_linear_bytes(int64_t M, int64_t K, int64_t N, int flags, size_t* kept, size_t* fwd, size_t* bwd) {
  const fp8_status s = linear_size(M, K, N);
  if (s != FP8_OK) return s;
  if (flags & ~(FP8_BLOCK_NEED_DX | FP8_BLOCK_NEED_DW) || !kept || !fwd || !bwd) return FP8_ERR_INVALID;
  *kept = LinearKept(nullptr, M, K, N, flags).bytes;
  *fwd = LinearFwd(nullptr, M, K, N, true).bytes;
  *bwd = LinearBwd(nullptr, M, K, N, flags).bytes;
  return FP8_OK;
}

fp8_status fp8_block_linear_fwd(const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t M, int64_t K, int64_t N,
                                int flags, void* kept, size_t kept_bytes, void* scratch, size_t scratch_bytes, void* Y,
                                hipStream_t stream) {
  const fp8_status s = linear_size(M, K, N);
  if (s != FP8_OK) return s;
  if (flags & ~(FP8_BLOCK_NEED_DX | FP8_BLOCK_NEED_DW) || !bf16_ok(X, M, K, ldx) || !bf16_ok(W, K, N, ldw) ||
      !bf16_ok(Y, M, N, N))
    return FP8_ERR_INVALID;
  const LinearKept k(kept, M, K, N, flags);
  const LinearFwd f(scratch, M, K, N, true);
  if (!space_ok(kept, kept_bytes, k.bytes) || !space_ok(scratch, scratch_bytes, f.bytes)) return FP8_ERR_INVALID;
  const BlockQuant q[] = {{{(const uint16_t*)X, ldx, M, K}, f.x, k.xt}, {{(const uint16_t*)W, ldw, K, N}, k.w, f.wt}};
  TRY(launch_block_quantize_many(q, 2, stream));
  return hip_status(launch_block_gemm({f.x, f.wt, FP8_E4M3, FP8_E4M3, (uint16_t*)Y, N}, f.part, f.part_bytes, stream));
}

fp8_status fp8_block_linear_bwd(const void* dY, int64_t lddy, int64_t M, int64_t K, int64_t N, int flags,
                                const void* kept, size_t kept_bytes, void* scratch, size_t scratch_bytes, void* dX,
                                void* dW, hipStream_t stream) {
  const fp8_status s = linear_size(M, K, N);
  if (s != FP8_OK) return s;
  const bool dx = flags & FP8_BLOCK_NEED_DX, dw = flags & FP8_BLOCK_NEED_DW;
  if (flags & ~(FP8_BLOCK_NEED_DX | FP8_BLOCK_NEED_DW) || !bf16_ok(dY, M, N, lddy) || (dx && !bf16_ok(dX, M, K, K)) ||
      (dw && !bf16_ok(dW, K, N, N)))
    return FP8_ERR_INVALID;
  const LinearKept k((void*)kept, M, K, N, flags);
  const LinearBwd b(scratch, M, K, N, flags);
  if (!space_ok(kept, kept_bytes, k.bytes) || !space_ok(scratch, scratch_bytes, b.bytes)) return FP8_ERR_INVALID;
  TRY(launch_block_quantize({(const uint16_t*)dY, lddy, M, N}, FP8_E5M2, b.dy, b.dyt, 0, stream));
  if (dx) TRY(launch_block_gemm({b.dy, k.w, FP8_E5M2, FP8_E4M3, (uint16_t*)dX, K}, b.part, b.part_bytes, stream));
  if (dw) TRY(launch_block_gemm({k.xt, b.dyt, FP8_E4M3, FP8_E5M2, (uint16_t*)dW, N}, b.part, b.part_bytes, stream));
  return FP8_OK;
}

size_t fp8_block_linear_cached_bytes(int64_t M, int64_t K, int64_t N) {
  return linear_size(M, K, N) == FP8_OK ? LinearFwd(nullptr, M, K, N, false).bytes : 0;
}

fp8_status fp8_block_linear_fwd_cached(const void* X, int64_t ldx, int64_t M, int64_t K, int64_t N,
                                       const uint8_t* w_codes, const uint8_t* w_scales, void* scratch,
                                       size_t scratch_bytes, void* Y, hipStream_t stream) {
  const fp8_status s = linear_size(M, K, N);
  if (s != FP8_OK) return s;
  if (!bf16_ok(X, M, K, ldx) || !codes_ok(w_codes, w_scales, N, K) || !bf16_ok(Y, M, N, N)) return FP8_ERR_INVALID;
  const LinearFwd f(scratch, M, K, N, false);
  if (!space_ok(scratch, scratch_bytes, f.bytes)) return FP8_ERR_INVALID;
  const Bf16Mat x = {(const uint16_t*)X, ldx, M, K};
  const BlockMat w = mat(w_codes, w_scales, N, K);
  if (block_serve_fused(M, K)) return hip_status(launch_block_serve_fused(x, w, (uint16_t*)Y, stream));
  TRY(launch_block_quantize(x, FP8_E4M3, f.x, kNone, 0, stream));
  if (block_serve_takes(M, N)) return hip_status(launch_block_serve(f.x, w, (uint16_t*)Y, stream));
  return hip_status(launch_block_gemm({f.x, w, FP8_E4M3, FP8_E4M3, (uint16_t*)Y, N}, f.part, f.part_bytes, stream));
}

int fp8_block_linear_few(int64_t M, int64_t K, int64_t N) {
  return linear_size(M, K, N) == FP8_OK && block_serve_fused(M, K);
}

fp8_status fp8_block_linear_fwd_few(const void* X, int64_t ldx, int64_t M, int64_t K, int64_t N, const uint8_t* w_codes,
                                    const uint8_t* w_scales, void* Y, hipStream_t stream) {
  const fp8_status s = linear_size(M, K, N);
  if (s != FP8_OK) return s;
  if (!bf16_ok(X, M, K, ldx) || !codes_ok(w_codes, w_scales, N, K) || !bf16_ok(Y, M, N, N)) return FP8_ERR_INVALID;
  if (!block_serve_fused(M, K)) return FP8_ERR_UNSUPPORTED;
  return hip_status(launch_block_serve_fused({(const uint16_t*)X, ldx, M, K}, mat(w_codes, w_scales, N, K), (uint16_t*)Y,
                                             stream));
}

size_t fp8_swiglu_kept_bytes(int64_t rows, int64_t cols) {
  return rows < 0 || cols < 0 || !size_ok(rows, cols) ? 0 : SwigluKept(nullptr, rows, cols).bytes;
}

fp8_status fp8_swiglu_fwd(const void* gate, int64_t ldg, const void* up, int64_t ldu, int64_t rows, int64_t cols,
                          void* h, void* kept, size_t kept_bytes, hipStream_t stream) {
  if (!bf16_ok(gate, rows, cols, ldg) || !bf16_ok(up, rows, cols, ldu) || !bf16_ok(h, rows, cols, cols))
    return FP8_ERR_INVALID;
  if (!size_ok(rows, cols)) return FP8_ERR_UNSUPPORTED;
  BlockMat g = kNone, u = kNone;
  if (kept) {
    const SwigluKept k(kept, rows, cols);
    if (!space_ok(kept, kept_bytes, k.bytes)) return FP8_ERR_INVALID;
    g = k.g;
    u = k.u;
  }
  return hip_status(launch_swiglu_fwd({(const uint16_t*)gate, ldg, rows, cols}, {(const uint16_t*)up, ldu, rows, cols},
                                      (uint16_t*)h, cols, kNone, g, u, stream));
}

fp8_status fp8_swiglu_bwd(const void* dh, int64_t lddh, int64_t rows, int64_t cols, const void* kept, size_t kept_bytes,
                          void* dgate, void* dup, hipStream_t stream) {
  if (!bf16_ok(dh, rows, cols, lddh) || !aligned2(dgate) || !aligned2(dup) ||
      (rows > 0 && cols > 0 && !dgate && !dup))
    return FP8_ERR_INVALID;
  if (!size_ok(rows, cols)) return FP8_ERR_UNSUPPORTED;
  const SwigluKept k((void*)kept, rows, cols);
  if (!space_ok(kept, kept_bytes, k.bytes)) return FP8_ERR_INVALID;
  return hip_status(launch_swiglu_bwd({(const uint16_t*)dh, lddh, rows, cols}, k.g, k.u, (uint16_t*)dgate, cols,
                                      (uint16_t*)dup, cols, stream));
}

fp8_status fp8_block_mlp_bytes(int64_t M, int64_t K, int64_t F, int flags, size_t* kept, size_t* fwd, size_t* bwd) {
  const fp8_status s = mlp_size(M, K, F);
  if (s != FP8_OK) return s;
  if (flags & ~kMlpAll || !kept || !fwd || !bwd) return FP8_ERR_INVALID;
  *kept = MlpKept(nullptr, M, K, F, flags).bytes;
  *fwd = MlpFwd(nullptr, M, K, F).bytes;
  *bwd = MlpBwd(nullptr, M, K, F, flags).bytes;
  return FP8_OK;
}

fp8_status fp8_block_mlp_fwd(const void* X, int64_t ldx, const void* Wgu, int64_t ldwgu, const void* Wd, int64_t ldwd,
                             int64_t M, int64_t K, int64_t F, int flags, void* kept, size_t kept_bytes, void* scratch,
                             size_t scratch_bytes, void* Y, hipStream_t stream) {
  const fp8_status s = mlp_size(M, K, F);
  if (s != FP8_OK) return s;
  if (flags & ~kMlpAll || !bf16_ok(X, M, K, ldx) || !bf16_ok(Wgu, K, 2 * F, ldwgu) || !bf16_ok(Wd, F, K, ldwd) ||
      !bf16_ok(Y, M, K, K))
    return FP8_ERR_INVALID;
  const MlpKept k(kept, M, K, F, flags);
  const MlpFwd f(scratch, M, K, F);
  if (!space_ok(kept, kept_bytes, k.bytes) || !space_ok(scratch, scratch_bytes, f.bytes)) return FP8_ERR_INVALID;
  const uint16_t* w = (const uint16_t*)Wgu;
  const BlockQuant q[] = {{{(const uint16_t*)X, ldx, M, K}, f.x, k.xt},
                          {{(const uint16_t*)Wd, ldwd, F, K}, k.wd, f.wdt},
                          {{w, ldwgu, K, 2 * F}, k.wgu, f.wgut}};
  if (F % kBlk == 0 || !k.wgu.codes) {
    TRY(launch_block_quantize_many(q, 3, stream));
  } else {
    TRY(launch_block_quantize_many(q, 2, stream));
    // a half's blocks start at its own first column
    for (int i = 0; i < 2; ++i) {
      BlockMat t = f.wgut;
      t.rows = F;
      TRY(launch_block_quantize({w + i * F, ldwgu, K, F}, FP8_E4M3, half(k.wgu, F, i), t, i * F, stream));
    }
  }
  TRY(launch_block_gemm({f.x, f.wgut, FP8_E4M3, FP8_E4M3, f.gu, 2 * F}, f.part, f.part_bytes, stream));
  TRY(launch_swiglu_fwd({f.gu, 2 * F, M, F}, {f.gu + F, 2 * F, M, F}, nullptr, 0, f.h, k.g, k.u, stream));
  return hip_status(launch_block_gemm({f.h, f.wdt, FP8_E4M3, FP8_E4M3, (uint16_t*)Y, K}, f.part, f.part_bytes, stream));
}

fp8_status fp8_block_mlp_bwd(const void* dY, int64_t lddy, int64_t M, int64_t K, int64_t F, int flags, const void* kept,
                             size_t kept_bytes, void* scratch, size_t scratch_bytes, void* dX, void* dWgu, void* dWd,
                             hipStream_t stream) {
  const fp8_status s = mlp_size(M, K, F);
  if (s != FP8_OK) return s;
  const bool dx = flags & FP8_BLOCK_NEED_DX, dw = flags & FP8_BLOCK_NEED_DW, dw2 = flags & FP8_BLOCK_NEED_DW2;
  if (flags & ~kMlpAll || !bf16_ok(dY, M, K, lddy) || (dx && !bf16_ok(dX, M, K, K)) ||
      (dw && !bf16_ok(dWgu, K, 2 * F, 2 * F)) || (dw2 && !bf16_ok(dWd, F, K, K)))
    return FP8_ERR_INVALID;
  const MlpKept k((void*)kept, M, K, F, flags);
  const MlpBwd b(scratch, M, K, F, flags);
  if (!space_ok(kept, kept_bytes, k.bytes) || !space_ok(scratch, scratch_bytes, b.bytes)) return FP8_ERR_INVALID;
  TRY(launch_block_quantize({(const uint16_t*)dY, lddy, M, K}, FP8_E5M2, b.dy, b.dyt, 0, stream));
  if (dx || dw) TRY(launch_block_gemm({b.dy, k.wd, FP8_E5M2, FP8_E4M3, b.dh, F}, b.part, b.part_bytes, stream));
  if (flags) {
    const Bf16Mat dh = dx || dw ? Bf16Mat{b.dh, F, M, F} : Bf16Mat{nullptr, 0, M, F};
    TRY(launch_swiglu_bwd_quant(dh, k.g, k.u, half(b.dgu, F, 0), half(b.dgu, F, 1), b.dgut, b.ht, stream));
  }
  if (dx) TRY(launch_block_gemm({b.dgu, k.wgu, FP8_E5M2, FP8_E4M3, (uint16_t*)dX, K}, b.part, b.part_bytes, stream));
  if (dw) TRY(launch_block_gemm({k.xt, b.dgut, FP8_E4M3, FP8_E5M2, (uint16_t*)dWgu, 2 * F}, b.part, b.part_bytes, stream));
  if (dw2) TRY(launch_block_gemm({b.ht, b.dyt, FP8_E4M3, FP8_E5M2, (uint16_t*)dWd, K}, b.part, b.part_bytes, stream));
  return FP8_OK;
}

}  // extern "C"
