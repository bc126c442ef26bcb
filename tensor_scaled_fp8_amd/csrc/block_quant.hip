// Block-scaled FP8 store and restore (formulas in block.h):
//   bias = floor(log2(fmt max / amax)) over each block of 128, code =
//   fp8(v 2^bias) to nearest even; back, bf16(code 2^-bias).
// One pass over the bf16 input: a block's 128 values are in registers when
// its maximum is known, so the tensor is read once whether the row form,
// the transposed form (blocks down the columns) or both are written. Bound
// by HBM: 2 bytes in and 1 out an element and form, 1/128 more for scales.
// Measured: 12288 x 36864 in both forms 342 us, 5.3 TB/s; 4096 x 4096 15.4 us,
// 4.4 TB/s; 4096 x 28672 in row form 56 us, 6.3 TB/s, and back 52 us.
#include "block_quant.h"

namespace fp8lin {
namespace {

// 128 x 128 tile per workgroup: transposed form, and the row form if ROW.
// Thread t has rows 8 (t / 16) .. + 7, columns 8 (t % 16) .. + 7 as packed
// bf16 (32 registers), so a row's block lies in 16 neighbouring lanes and a
// column's in 16 lane groups of all four waves: its maximum is reduced
// within a wave, then over LDS by one thread a column.
template <int FMT, bool ROW>
__device__ __forceinline__ void quant_tile(const Bf16Mat& x, const BlockMat& row, const BlockMat& tr, int64_t t_row0,
                                           int tiles_c, int at) {
  __shared__ uint4 tile[kBlk * kBlk / 16];
  __shared__ uint32_t cmax[4][kBlk / 2];  // of each wave, two columns' bf16 magnitudes a dword
  __shared__ float cscale[kBlk];
  __shared__ uint8_t rbyte[kBlk];         // in the scales' order
  const int64_t r0 = (int64_t)(at / tiles_c) * kBlk, c0 = (int64_t)(at % tiles_c) * kBlk;
  const int t = threadIdx.x, rg = t >> 4, cc = t & 15;
  const int64_t rr = r0 + 8 * rg, cx = c0 + 8 * cc;
  bq_u32x4 w[8];
  load_rows<8, 1>(x, rr, cx, r0 + kBlk <= x.rows && c0 + kBlk <= x.cols, w);
  bq_u32x4 cm = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bq_u32x4 a = w[i] & 0x7FFF7FFFu;
#pragma unroll
    for (int d = 0; d < 4; ++d) cm[d] = pk_max(cm[d], a[d]);
  }
  if constexpr (ROW) {
    uint2 q[8];
    uint32_t byte[8];
    rows_codes<FMT>(w, q, byte);
    const __amdgpu_buffer_rsrc_t r = tile_rsrc(row, r0, kBlk);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      put_codes(r, q[i], (8 * rg + i) * (int)row.pitch + (int)cx);
      if (cc == 0) rbyte[(8 * (rg & 1) + i) * 8 + (rg >> 1)] = (uint8_t)byte[i];
    }
  }
  // dword R of the four in the R-th 16 lanes
  cmax[t >> 6][4 * cc + (rg & 3)] =
      swap16_max(swap32_max(cm[0], cm[2], pk_max), swap32_max(cm[1], cm[3], pk_max), pk_max);
  __syncthreads();
  if (t < kBlk) {
    const int sh = 16 * (t & 1);
    const uint32_t m =
        pk_max(pk_max(cmax[0][t >> 1], cmax[1][t >> 1]), pk_max(cmax[2][t >> 1], cmax[3][t >> 1])) >> sh << 16;
    const uint32_t byte = scale_byte<FMT>(m);
    cscale[t] = m < 0x7F800000u ? scale_value(byte) : -1.0f;
    if (c0 + t < tr.rows) tr.scales[r0 / kBlk * tr.srows + scale_pos(t_row0 + c0 + t)] = (uint8_t)byte;
  } else if (ROW) {
    const int p = t - kBlk;
    if (r0 + 16 * (p & 7) + (p >> 3) < row.rows) row.scales[c0 / kBlk * row.srows + r0 + p] = rbyte[p];
  }
  __syncthreads();
  float s[8];  // negative: an infinity or a NaN in the column
  bool odd = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    s[j] = cscale[8 * cc + j];
    odd |= s[j] < 0;
  }
  odd = __builtin_expect(__any(odd), 0);
  uint8_t* const l8 = (uint8_t*)tile;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t p[4];  // rows 2 k, 2 k + 1 of column j
#pragma unroll
    for (int k = 0; k < 4; ++k)
      p[k] = __builtin_amdgcn_perm(w[2 * k + 1][j >> 1], w[2 * k][j >> 1], j & 1 ? 0x07060302 : 0x05040100);
    if (__builtin_expect(odd, 0)) {
#pragma unroll
      for (int k = 0; k < 4; ++k) p[k] = clamp_pair<FMT>(p[k], s[j] < 0);
      s[j] = __builtin_fabsf(s[j]);
    }
    *(uint2*)(l8 + 16 * lds_chunk(8 * cc + j, rg >> 1) + 8 * (rg & 1)) =
        make_uint2(code4<FMT>(p[0], p[1], s[j]), code4<FMT>(p[2], p[3], s[j]));
  }
  __syncthreads();
  put_tile<256>(tile, tr, t_row0 + c0, tr.rows - c0, r0);
}

template <int FMT, bool ROW>
__global__ __launch_bounds__(256) void block_quant_tile_kernel(Bf16Mat x, BlockMat row, BlockMat tr, int64_t t_row0,
                                                               int tiles_c) {
  quant_tile<FMT, ROW>(x, row, tr, t_row0, tiles_c, blockIdx.x);
}

// both forms of several matrices: first[i] is the first workgroup of the i-th
struct QuantSets {
  BlockQuant q[kMaxQuant];
  int tiles_c[kMaxQuant], first[kMaxQuant];
};
template <int FMT>
__global__ __launch_bounds__(256) void block_quant_many_kernel(QuantSets s) {
  int i = 0;
#pragma unroll
  for (int k = 1; k < kMaxQuant; ++k) i += (int)blockIdx.x >= s.first[k];
  const BlockQuant& q = s.q[i];
  quant_tile<FMT, true>(q.x, q.row, q.t, 0, s.tiles_c[i], blockIdx.x - s.first[i]);
}

// row form only: 16 RPT rows x 128 columns per workgroup
template <int FMT, int RPT>
__global__ __launch_bounds__(256) void block_quant_rows_kernel(Bf16Mat x, BlockMat row, int tiles_c) {
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * (16 * RPT), c0 = (int64_t)(blockIdx.x % tiles_c) * kBlk;
  const int t = threadIdx.x;
  const int64_t rr = r0 + (t >> 4), cx = c0 + 8 * (t & 15);
  bq_u32x4 w[RPT];
  load_rows<RPT, 16>(x, rr, cx, r0 + 16 * RPT <= x.rows && c0 + kBlk <= x.cols, w);
  uint2 q[RPT];
  uint32_t byte[RPT];
  rows_codes<FMT>(w, q, byte);
  const __amdgpu_buffer_rsrc_t r = tile_rsrc(row, r0, 16 * RPT);
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    put_codes(r, q[i], ((t >> 4) + 16 * i) * (int)row.pitch + (int)cx);
    put_byte(row, rr + 16 * i, cx, byte[i]);
  }
}

template <int FMT, int RPT>
__global__ __launch_bounds__(256) void block_dequant_kernel(BlockMat q, uint16_t* __restrict__ out, int64_t ld,
                                                            int tiles_c) {
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * (16 * RPT), c0 = (int64_t)(blockIdx.x % tiles_c) * kBlk;
  const int t = threadIdx.x;
  const int64_t rr = r0 + (t >> 4), cx = c0 + 8 * (t & 15);
  uint2 c[RPT];
  float s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    c[i] = make_uint2(0, 0);
    s[i] = 1.0f;
    if (rr + 16 * i < q.rows) {
      c[i] = row_codes_at(q, rr + 16 * i, cx);
      s[i] = row_scale_at(q, rr + 16 * i, cx);
    }
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    if (rr + 16 * i < q.rows) store8(out + (rr + 16 * i) * ld, cx, q.cols, uncode8_bf16<FMT>(c[i], s[i]));
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

hipError_t launch_block_quantize_many(const BlockQuant* q, int n, hipStream_t st) {
  QuantSets s = {};
  int64_t tiles = 0;
  bool one = n <= kMaxQuant;
  for (int i = 0; i < n && one; ++i) {
    const Bf16Mat& x = q[i].x;
    one = x.rows > 0 && x.cols > 0 && q[i].row.codes && q[i].t.codes;
    s.q[i] = q[i];
    s.tiles_c[i] = (int)((x.cols + kBlk - 1) / kBlk);
    s.first[i] = (int)tiles;
    tiles += (x.rows + kBlk - 1) / kBlk * s.tiles_c[i];
    one = one && tiles < ((int64_t)1 << 23);  // 2^31 threads
  }
  if (!one) {
    for (int i = 0; i < n; ++i) {
      const hipError_t e = launch_block_quantize(q[i].x, FP8_E4M3, q[i].row, q[i].t, 0, st);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  for (int i = n; i < kMaxQuant; ++i) s.first[i] = 0x7FFFFFFF;
  block_quant_many_kernel<FP8_E4M3><<<dim3((unsigned)tiles), 256, 0, st>>>(s);
  return hipGetLastError();
}

hipError_t launch_block_dequantize(const BlockMat& q, int fmt, uint16_t* out, int64_t ld, hipStream_t st) {
  if (q.rows == 0 || q.cols == 0) return hipSuccess;
  return fmt == FP8_E5M2 ? dequantize<FP8_E5M2>(q, out, ld, st) : dequantize<FP8_E4M3>(q, out, ld, st);
}

}  // namespace fp8lin
