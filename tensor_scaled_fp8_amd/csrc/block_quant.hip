// Block-scaled FP8 store and restore (formulas in block.h):
//   bias = floor(log2(fmt max / amax)) over each block of 128, code =
//   fp8(v 2^bias) to nearest even; back, bf16(code 2^-bias).
// One pass over the bf16 input: a block's 128 values are in registers when
// its maximum is known, so the tensor is read once whether the row form,
// the transposed form (blocks down the columns) or both are written. Bound
// by HBM: 2 bytes in and 1 out an element and form, 1/128 more for scales.
#include "block_quant.h"

namespace fp8lin {
namespace {

// 128 x 128 tile per workgroup: transposed form, and the row form if ROW
template <int FMT, bool ROW>
__global__ __launch_bounds__(256) void block_quant_tile_kernel(Bf16Mat x, BlockMat row, BlockMat tr, int64_t t_row0,
                                                               int tiles_c) {
  __shared__ QuantLds lds;
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * kBlk, c0 = (int64_t)(blockIdx.x % tiles_c) * kBlk;
  const int t = threadIdx.x, rg = t >> 4, cc = t & 15;
  const int64_t rr = r0 + 8 * rg, cx = c0 + 8 * cc;
  bq_u32x4 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = (bq_u32x4){0, 0, 0, 0};
    if (rr + i < x.rows) w[i] = load8(x.p + (rr + i) * x.ld, cx, x.cols);
  }
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) widen8(w[i], v[i]);
  if constexpr (ROW) {
#pragma unroll
    for (int i = 0; i < 8; ++i) quant_row8<FMT>(v[i], row, rr + i, cx);
  }
  quant_cols<FMT>(v, tr, t_row0, r0, c0, lds);
}

// row form only: 16 RPT rows x 128 columns per workgroup
template <int FMT, int RPT>
__global__ __launch_bounds__(256) void block_quant_rows_kernel(Bf16Mat x, BlockMat row, int tiles_c) {
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * (16 * RPT), c0 = (int64_t)(blockIdx.x % tiles_c) * kBlk;
  const int t = threadIdx.x;
  const int64_t rr = r0 + (t >> 4), cx = c0 + 8 * (t & 15);
  bq_u32x4 w[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    w[i] = (bq_u32x4){0, 0, 0, 0};
    if (rr + 16 * i < x.rows) w[i] = load8(x.p + (rr + 16 * i) * x.ld, cx, x.cols);
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    float f[8];
    widen8(w[i], f);
    quant_row8<FMT>(f, row, rr + 16 * i, cx);
  }
}

template <int FMT, int RPT>
__global__ __launch_bounds__(256) void block_dequant_kernel(BlockMat q, uint16_t* __restrict__ out, int64_t ld,
                                                            int tiles_c) {
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * (16 * RPT), c0 = (int64_t)(blockIdx.x % tiles_c) * kBlk;
  const int t = threadIdx.x;
  const int64_t rr = r0 + (t >> 4), cx = c0 + 8 * (t & 15);
  float f[RPT][8];
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    if (rr + 16 * i < q.rows) load_row8<FMT>(q, rr + 16 * i, cx, f[i]);
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    if (rr + 16 * i < q.rows) store8(out + (rr + 16 * i) * ld, cx, q.cols, f[i]);
}

// rows a thread takes in the row kernels: 8 keeps many loads in flight, 1
// spreads a small matrix over the chip
inline bool few_rows(int64_t rows, int64_t cols) { return (rows + 127) / 128 * ((cols + 127) / 128) < 1024; }

template <int FMT>
hipError_t quantize(const Bf16Mat& x, const BlockMat& row, const BlockMat& t, int64_t t_row0, hipStream_t st) {
  const int64_t tc = (x.cols + kBlk - 1) / kBlk;
  const dim3 tiles((unsigned)((x.rows + kBlk - 1) / kBlk * tc));
  if (t.codes) {
    if (row.codes) block_quant_tile_kernel<FMT, true><<<tiles, 256, 0, st>>>(x, row, t, t_row0, (int)tc);
    else block_quant_tile_kernel<FMT, false><<<tiles, 256, 0, st>>>(x, row, t, t_row0, (int)tc);
  } else if (few_rows(x.rows, x.cols)) {
    block_quant_rows_kernel<FMT, 1><<<dim3((unsigned)((x.rows + 15) / 16 * tc)), 256, 0, st>>>(x, row, (int)tc);
  } else {
    block_quant_rows_kernel<FMT, 8><<<tiles, 256, 0, st>>>(x, row, (int)tc);
  }
  return hipGetLastError();
}

template <int FMT>
hipError_t dequantize(const BlockMat& q, uint16_t* out, int64_t ld, hipStream_t st) {
  const int64_t tc = (q.cols + kBlk - 1) / kBlk;
  if (few_rows(q.rows, q.cols))
    block_dequant_kernel<FMT, 1><<<dim3((unsigned)((q.rows + 15) / 16 * tc)), 256, 0, st>>>(q, out, ld, (int)tc);
  else
    block_dequant_kernel<FMT, 8><<<dim3((unsigned)((q.rows + 127) / 128 * tc)), 256, 0, st>>>(q, out, ld, (int)tc);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_quantize(const Bf16Mat& x, int fmt, const BlockMat& row, const BlockMat& t, int64_t t_row0,
                                 hipStream_t st) {
  if (x.rows == 0 || x.cols == 0 || (!row.codes && !t.codes)) return hipSuccess;
  return fmt == FP8_E5M2 ? quantize<FP8_E5M2>(x, row, t, t_row0, st) : quantize<FP8_E4M3>(x, row, t, t_row0, st);
}

hipError_t launch_block_dequantize(const BlockMat& q, int fmt, uint16_t* out, int64_t ld, hipStream_t st) {
  if (q.rows == 0 || q.cols == 0) return hipSuccess;
  return fmt == FP8_E5M2 ? dequantize<FP8_E5M2>(q, out, ld, st) : dequantize<FP8_E4M3>(q, out, ld, st);
}

}  // namespace fp8lin
