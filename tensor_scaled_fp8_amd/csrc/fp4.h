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

// X [M, K] quantised (E4M3, a scale for each 128 of a row) in the order that
// the instructions take it: for each 16 rows and each 128 of K two pieces of
// 1024 bytes, byte 16 (16 G + r) + i of piece p being element 64 p + 16 G + i
// of row r; scale bytes [16 rows][4 blocks of 128] as words. The pad of a last
// part block is zero; rows past the last are not written.
struct Fp4X {
  uint8_t *codes, *scales;
  int64_t M, K;
};
__host__ __device__ inline int64_t fp4_xblocks(int64_t K) { return (K + 127) / 128; }
inline size_t fp4_x_codes(int64_t M, int64_t K) { return (size_t)((M + 15) / 16) * fp4_xblocks(K) * 2048; }
inline size_t fp4_x_scales(int64_t M, int64_t K) { return (size_t)((M + 15) / 16) * ((fp4_xblocks(K) + 3) / 4) * 64; }
hipError_t launch_fp4_x(const Bf16Mat& x, const Fp4X& q, hipStream_t st);

// Y [M, N] = X W. Of few rows (and blocks of K) X is quantised by the
// product's own launch; otherwise it comes quantised. Up to kFp4Few rows, and
// up to kFp4FewExact of an exact product, it is of bf16 operands in the form
// that waits for W's bytes; above, of the 8-bit and 4-bit codes, or of bf16 if
// exact. us by 4096 x 12288 and 8192 x 8192: 32 rows 14.2 and 17.6 (of the
// codes 14.3 and 21.0); 64 rows, exact, 18.3 and 24.3 (by the exact form of
// many rows 19.6 and 29.7), of the codes 15.1 and 22.3.
constexpr int64_t kFp4Few = 32, kFp4FewExact = 64;
bool fp4_fused(int64_t M, int64_t K);
struct Fp4Form {
  int kind;             // FP4_FUSED, _FEW, _MANY or _EXACT
  int mf, nb, groups;   // 16-row fragments of X and 16-column ones of W a wave, groups of waves over K
  int cols;             // of Y a workgroup (fused, few)
};
Fp4Form fp4_form(int64_t M, int64_t K, int64_t N, bool exact);
// Y of an empty sum (K = 0): the product's kernels have no block of K to stand on
hipError_t launch_fp4_zero(uint16_t* y, int64_t n, hipStream_t st);
hipError_t launch_fp4_fused(const Bf16Mat& x, const Fp4Mat& w, uint16_t* y, hipStream_t st);
hipError_t launch_fp4_linear(const Fp4X& x, const Fp4Mat& w, uint16_t* y, bool exact, hipStream_t st);

}  // namespace fp8lin
