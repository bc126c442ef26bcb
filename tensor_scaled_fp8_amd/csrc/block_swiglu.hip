// SwiGLU with 8-bit checkpoints. Forward, from the bf16 gate g and up u:
//   h = g s u,  s = 1 / (1 + exp(-g)),
// and the E4M3 block-scaled forms g', u' that the backward reads in place
// of g and u (half their bytes). Backward, at g', u':
//   dg = dh u' s' (1 + g' (1 - s')),  du = dh g' s',  h' = g' s' u'.
// Everything is computed in 32 bits and rounded once, to bf16 or to a
// block-scaled code. Bound by HBM: every input read once, every output
// written once, the maxima of a block taken in registers.
#include "block_quant.h"

namespace fp8lin {
namespace {

// v_exp and v_rcp are within 1 ulp or so of 32 bits, far below the
// outputs' 8 bits; exp overflows to inf for g < -88, whose reciprocal is
// the right 0
__device__ inline float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

struct Grads {
  float dg, du, h;
};
__device__ inline Grads grads(float g, float u, float dh) {
  const float s = sigmoid(g);
  const float gs = g * s;
  return {dh * u * s * (1.0f + g * (1.0f - s)), dh * gs, gs * u};
}

template <int RPT>
__global__ __launch_bounds__(256) void swiglu_fwd_kernel(Bf16Mat gate, Bf16Mat up, uint16_t* __restrict__ h, int64_t ldh,
                                                         BlockMat hq, BlockMat gq, BlockMat uq, int tiles_c) {
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * (16 * RPT), c0 = (int64_t)(blockIdx.x % tiles_c) * kBlk;
  const int t = threadIdx.x;
  const int64_t rr = r0 + (t >> 4), cx = c0 + 8 * (t & 15);
  bq_u32x4 wg[RPT], wu[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    wg[i] = wu[i] = (bq_u32x4){0, 0, 0, 0};
    if (rr + 16 * i < gate.rows) {
      wg[i] = load8(gate.p + (rr + 16 * i) * gate.ld, cx, gate.cols);
      wu[i] = load8(up.p + (rr + 16 * i) * up.ld, cx, gate.cols);
    }
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int64_t r = rr + 16 * i;
    float g[8], u[8], y[8];
    widen8(wg[i], g);
    widen8(wu[i], u);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = g[k] * sigmoid(g[k]) * u[k];
    if (h && r < gate.rows) store8(h + r * ldh, cx, gate.cols, y);
    if (hq.codes) quant_row8<FP8_E4M3>(y, hq, r, cx);
    if (gq.codes) {
      quant_row8<FP8_E4M3>(g, gq, r, cx);
      quant_row8<FP8_E4M3>(u, uq, r, cx);
    }
  }
}

template <int RPT>
__global__ __launch_bounds__(256) void swiglu_bwd_kernel(Bf16Mat dh, BlockMat gq, BlockMat uq,
                                                         uint16_t* __restrict__ dg, int64_t lddg,
                                                         uint16_t* __restrict__ du, int64_t lddu, int tiles_c) {
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * (16 * RPT), c0 = (int64_t)(blockIdx.x % tiles_c) * kBlk;
  const int t = threadIdx.x;
  const int64_t rr = r0 + (t >> 4), cx = c0 + 8 * (t & 15);
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int64_t r = rr + 16 * i;
    if (r >= dh.rows) continue;
    float g[8], u[8], d[8], a[8], b[8];
    widen8(load8(dh.p + r * dh.ld, cx, dh.cols), d);
    load_row8<FP8_E4M3>(gq, r, cx, g);
    load_row8<FP8_E4M3>(uq, r, cx, u);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const Grads x = grads(g[k], u[k], d[k]);
      a[k] = x.dg;
      b[k] = x.du;
    }
    if (dg) store8(dg + r * lddg, cx, dh.cols, a);
    if (du) store8(du + r * lddu, cx, dh.cols, b);
  }
}

// One 128 x 128 tile: the E5M2 row and transposed forms of dg and du, and
// the E4M3 transposed form of h'. The three are made one after the other
// from the same loaded operands, so 64 results are live at a time. dh.p
// null: h' only.
__global__ __launch_bounds__(256) void swiglu_bwd_quant_kernel(Bf16Mat dh, BlockMat gq, BlockMat uq, BlockMat dgq,
                                                               BlockMat duq, BlockMat dgut, BlockMat ht, int tiles_c) {
  __shared__ QuantLds lds;
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * kBlk, c0 = (int64_t)(blockIdx.x % tiles_c) * kBlk;
  const int t = threadIdx.x, rg = t >> 4, cc = t & 15;
  const int64_t rr = r0 + 8 * rg, cx = c0 + 8 * cc;
  bq_u32x4 wd[8];
  uint2 wg[8], wu[8];
  float sg[8], su[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wd[i] = (bq_u32x4){0, 0, 0, 0};
    wg[i] = wu[i] = make_uint2(0, 0);
    sg[i] = su[i] = 0.0f;
    const int64_t r = rr + i;
    if (r < dh.rows) {
      if (dh.p) wd[i] = load8(dh.p + r * dh.ld, cx, dh.cols);
      wg[i] = *(const uint2*)(gq.codes + r * gq.pitch + cx);
      wu[i] = *(const uint2*)(uq.codes + r * uq.pitch + cx);
      sg[i] = scale_value(gq.scales[cx / kBlk * gq.srows + scale_pos(r)]);
      su[i] = scale_value(uq.scales[cx / kBlk * uq.srows + scale_pos(r)]);
    }
  }
  const int64_t f = dh.cols;
  float v[8][8];
  auto fill = [&](auto pick) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float d[8], g[8], u[8];
      widen8(wd[i], d);
      uncode8<FP8_E4M3>(wg[i], sg[i], g);
      uncode8<FP8_E4M3>(wu[i], su[i], u);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = pick(grads(g[k], u[k], d[k]));
    }
  };
  if (ht.codes) {
    fill([](const Grads& x) { return x.h; });
    quant_cols<FP8_E4M3>(v, ht, 0, r0, c0, lds);
  }
  if (!dh.p) return;
  fill([](const Grads& x) { return x.dg; });
  if (dgq.codes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) quant_row8<FP8_E5M2>(v[i], dgq, rr + i, cx);
  }
  if (dgut.codes) {
    BlockMat o = dgut;
    o.rows = f;  // dg's rows of the transposed form are 0 .. f - 1, du's f .. 2 f - 1
    quant_cols<FP8_E5M2>(v, o, 0, r0, c0, lds);
  }
  fill([](const Grads& x) { return x.du; });
  if (duq.codes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) quant_row8<FP8_E5M2>(v[i], duq, rr + i, cx);
  }
  if (dgut.codes) {
    BlockMat o = dgut;
    o.rows = f;
    quant_cols<FP8_E5M2>(v, o, f, r0, c0, lds);
  }
}

inline bool few_rows(int64_t rows, int64_t cols) { return (rows + 127) / 128 * ((cols + 127) / 128) < 1024; }

}  // namespace

hipError_t launch_swiglu_fwd(const Bf16Mat& gate, const Bf16Mat& up, uint16_t* h, int64_t ldh, const BlockMat& hq,
                             const BlockMat& gq, const BlockMat& uq, hipStream_t st) {
  if (gate.rows == 0 || gate.cols == 0) return hipSuccess;
  const int64_t tc = (gate.cols + kBlk - 1) / kBlk;
  if (few_rows(gate.rows, gate.cols))
    swiglu_fwd_kernel<1><<<dim3((unsigned)((gate.rows + 15) / 16 * tc)), 256, 0, st>>>(gate, up, h, ldh, hq, gq, uq,
                                                                                      (int)tc);
  else
    swiglu_fwd_kernel<4><<<dim3((unsigned)((gate.rows + 63) / 64 * tc)), 256, 0, st>>>(gate, up, h, ldh, hq, gq, uq,
                                                                                      (int)tc);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const Bf16Mat& dh, const BlockMat& gq, const BlockMat& uq, uint16_t* dg, int64_t lddg,
                             uint16_t* du, int64_t lddu, hipStream_t st) {
  if (dh.rows == 0 || dh.cols == 0) return hipSuccess;
  const int64_t tc = (dh.cols + kBlk - 1) / kBlk;
  if (few_rows(dh.rows, dh.cols))
    swiglu_bwd_kernel<1><<<dim3((unsigned)((dh.rows + 15) / 16 * tc)), 256, 0, st>>>(dh, gq, uq, dg, lddg, du, lddu,
                                                                                    (int)tc);
  else
    swiglu_bwd_kernel<4><<<dim3((unsigned)((dh.rows + 63) / 64 * tc)), 256, 0, st>>>(dh, gq, uq, dg, lddg, du, lddu,
                                                                                    (int)tc);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd_quant(const Bf16Mat& dh, const BlockMat& gq, const BlockMat& uq, const BlockMat& dgq,
                                   const BlockMat& duq, const BlockMat& dgut, const BlockMat& ht, hipStream_t st) {
  if (dh.rows == 0 || dh.cols == 0) return hipSuccess;
  const int64_t tc = (dh.cols + kBlk - 1) / kBlk;
  swiglu_bwd_quant_kernel<<<dim3((unsigned)((dh.rows + kBlk - 1) / kBlk * tc)), 256, 0, st>>>(dh, gq, uq, dgq, duq,
                                                                                            dgut, ht, (int)tc);
  return hipGetLastError();
}

}  // namespace fp8lin
