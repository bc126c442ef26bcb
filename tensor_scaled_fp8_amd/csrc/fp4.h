// Shared declarations of the 4-bit weight (fp4_*.hip).
//
// W [K, N] as the scaled matrix instruction 16x16x128 takes it: a panel of 16
// columns and 128 of K is one instruction's operand, 16 contiguous bytes a
// lane (lane 16 G + r: column r, elements 32 G ..+31, one scale), so a wave
// streams a panel's K in whole lines. A lane's scale bytes of four such
// k-blocks make one word.
#pragma once

#include "block_quant.h"
#include "fp8lin_serve.h"

namespace fp8lin {

__host__ __device__ inline int64_t fp4_kblocks(int64_t K) { return (K + 511) / 512 * 4; }  // of 128, as stored

struct Fp4Mat {
  uint8_t *codes, *scales;
  int64_t K, N;
};
hipError_t launch_fp4_quantize(const uint16_t* w, int64_t ld, const Fp4Mat& q, hipStream_t st);
hipError_t launch_fp4_dequantize(const Fp4Mat& q, uint16_t* w, int64_t ld, hipStream_t st);
// Y [x.rows, w.N] = X W of a stored X [M, K]
hipError_t launch_fp4_linear(const BlockMat& x, const Fp4Mat& w, uint16_t* y, hipStream_t st);

}  // namespace fp8lin
