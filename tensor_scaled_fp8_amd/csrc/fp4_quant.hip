// Storing a weight in 4 bits and restoring it: a thread takes one group of 32
// along K of one column, so a wave reads 64 columns of a row at a time and
// writes 16 bytes a lane. Done once a weight.
#include "fp4.h"

namespace fp8lin {
namespace {

// where column n's group g of 32 lies
__device__ inline int64_t code_at(int64_t n, int64_t g, int64_t kblocks) {
  return ((n >> 4) * kblocks + (g >> 2)) * 1024 + 256 * (g & 3) + 16 * (n & 15);
}
__device__ inline int64_t scale_at(int64_t n, int64_t g, int64_t kblocks) {
  const int64_t b = g >> 2;
  return ((n >> 4) * (kblocks >> 2) + (b >> 2)) * 256 + 64 * (g & 3) + 4 * (n & 15) + (b & 3);
}

// 127 - floor(log2(6 / amax)) from the bits of amax in 32 bits; 0 and infinity: 127
__device__ inline uint32_t scale_byte4(uint32_t mag) {
  const int e = (int)((mag + 0x3FFFFFu) >> 23) - 2;  // carries if the significand is above 1.5
  return mag - 1u < 0x7F7FFFFFu ? (uint32_t)(e > 1 ? e : 1) : 127u;
}

__global__ __launch_bounds__(256) void fp4_quant_kernel(const uint16_t* __restrict__ w, int64_t ld, Fp4Mat q) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x, g = blockIdx.y, kblocks = fp4_kblocks(q.K);
  if (n >= (q.N + 15) / 16 * 16) return;
  uint32_t v[32], mag = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] = n < q.N && 32 * g + i < q.K ? w[(32 * g + i) * ld + n] : 0;
    mag = umax(mag, v[i] & 0x7FFFu);
  }
  const bool bad = mag > 0x7F80u;
  const uint32_t byte = bad ? 255u : scale_byte4(mag << 16);
  const float s = bad ? 1.0f : scale_value(byte), most = 6.0f * s;
  bq_u32x4 c;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t word = 0;
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fminf(fmaxf(__uint_as_float(v[8 * k + i] << 16), -most), most);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f[0], f[1], s, 0);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f[2], f[3], s, 1);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f[4], f[5], s, 2);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f[6], f[7], s, 3);
    c[k] = bad ? 0x22222222u : word;
  }
  *(bq_u32x4*)(q.codes + code_at(n, g, kblocks)) = c;
  q.scales[scale_at(n, g, kblocks)] = (uint8_t)byte;
}

__global__ __launch_bounds__(256) void fp4_dequant_kernel(Fp4Mat q, uint16_t* __restrict__ w, int64_t ld) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x, g = blockIdx.y, kblocks = fp4_kblocks(q.K);
  if (n >= q.N) return;
  const bq_u32x4 c = *(const bq_u32x4*)(q.codes + code_at(n, g, kblocks));
  const uint32_t byte = q.scales[scale_at(n, g, kblocks)];
  const bool bad = byte == 255u;
  const float s = scale_value(byte);
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (32 * g + i >= q.K) break;
    // 2^e (1 + m / 2) from sign, 2 exponent bits and 1 mantissa bit
    const uint32_t x = c[i >> 3] >> (4 * (i & 7)), e = x >> 1 & 3u, m = x & 1u;
    const float a = e ? (float)((2u + m) << (e - 1)) * 0.5f : 0.5f * (float)m;
    const float f = (x & 8u ? -a : a) * s;
    w[(32 * g + i) * ld + n] = bad ? 0x7FC0u : (uint16_t)pack_bf16(f, 0.0f);
  }
}

// X quantised for the product: 16 lanes a block of 128, 16 blocks a workgroup
__global__ __launch_bounds__(256) void fp4_x_kernel(Bf16Mat x, Fp4X q, int nk) {
  const int t = threadIdx.x, c8 = 8 * (t & 15), r = t >> 4;
  const int64_t mt = blockIdx.x / nk, row = mt * 16 + r;
  const int kb = (int)(blockIdx.x % nk);
  bq_u32x4 v[1];
  load_rows<1, 1, false>(x, row, (int64_t)kb * kBlk + c8, mt * 16 + 16 <= x.rows && (int64_t)(kb + 1) * kBlk <= x.cols, v);
  uint2 c[1];
  uint32_t byte[1];
  rows_codes<FP8_E4M3>(v, c, byte);
  if (row >= x.rows) return;
  uint8_t* o = q.codes + ((mt * nk + kb) * 2 + (c8 >> 6)) * 1024 + ((c8 >> 4 & 3) * 16 + r) * 16 + (c8 & 15);
  *(uint2*)o = c[0];
  if (c8 == 0) q.scales[(mt * ((nk + 3) / 4) + (kb >> 2)) * 64 + 4 * r + (kb & 3)] = (uint8_t)byte[0];
}

}  // namespace

hipError_t launch_fp4_x(const Bf16Mat& x, const Fp4X& q, hipStream_t st) {
  const int nk = (int)fp4_xblocks(x.cols);
  if (x.rows == 0 || nk == 0) return hipSuccess;
  fp4_x_kernel<<<(unsigned)((x.rows + 15) / 16 * nk), 256, 0, st>>>(x, q, nk);
  return hipGetLastError();
}

hipError_t launch_fp4_quantize(const uint16_t* w, int64_t ld, const Fp4Mat& q, hipStream_t st) {
  if (q.K == 0 || q.N == 0) return hipSuccess;
  fp4_quant_kernel<<<dim3((unsigned)((q.N + 255) / 256), (unsigned)(4 * fp4_kblocks(q.K))), 256, 0, st>>>(w, ld, q);
  return hipGetLastError();
}

hipError_t launch_fp4_dequantize(const Fp4Mat& q, uint16_t* w, int64_t ld, hipStream_t st) {
  if (q.K == 0 || q.N == 0) return hipSuccess;
  fp4_dequant_kernel<<<dim3((unsigned)((q.N + 255) / 256), (unsigned)((q.K + 31) / 32)), 256, 0, st>>>(q, w, ld);
  return hipGetLastError();
}

}  // namespace fp8lin
