// Shared declarations of the block-scaled FP8 sources (block_*.hip).
//
// A block-scaled matrix holds, for each row and each block of 128
// consecutive columns, FP8 codes and one power-of-two scale:
//   value(r, c) = code(r, c) * 2^(scale byte(r, c / 128) - 127).
// Codes are row-major with the pitch rounded up to 128 (zero codes in the
// pad), so a block is one 128-byte cache line and a GEMM never meets a
// partial one. The scale byte is the E8M0 exponent the scaled MFMA takes.
// Scales are stored block-major, srows (rows rounded up to 128) bytes for
// each block of 128 columns, with the rows of each group of 128 permuted by
// scale_pos: an MFMA lane holds rows l % 16, 16 + l % 16, ... of the group,
// so its eight scale bytes are eight consecutive bytes.
#pragma once

#include "fp8lin_internal.h"

namespace fp8lin {

constexpr int kBlk = 128;
__host__ __device__ inline int64_t round_blk(int64_t n) { return (n + kBlk - 1) / kBlk * kBlk; }

// place of a row's scale byte within a column block's srows bytes
__host__ __device__ inline int64_t scale_pos(int64_t row) {
  return (row & ~(int64_t)127) | ((row & 15) << 3) | ((row >> 4) & 7);
}

// A block-scaled matrix as the kernels take it. codes and scales may point
// into a larger one (at a column block): pitch and srows are the larger's.
struct BlockMat {
  uint8_t* codes;   // null: not wanted (an output) 
  uint8_t* scales;
  int64_t pitch;    // bytes from a row of codes to the next
  int64_t srows;    // bytes from a column block of scales to the next
  int64_t rows, cols;
};

// A bf16 matrix with a row pitch in elements (any alignment of 2 bytes).
struct Bf16Mat {
  const uint16_t* p;
  int64_t ld, rows, cols;
};

hipError_t launch_block_quantize(const Bf16Mat& x, int fmt, const BlockMat& row, const BlockMat& t, int64_t t_row0,
                                 hipStream_t st);
// E4M3 forms of up to kMaxQuant matrices, by one launch where all want both
// forms (a training step's X and weights: two launches of 2 us each on the
// host less in an MLP)
constexpr int kMaxQuant = 3;
struct BlockQuant {
  Bf16Mat x;
  BlockMat row, t;
};
hipError_t launch_block_quantize_many(const BlockQuant* q, int n, hipStream_t st);
hipError_t launch_block_dequantize(const BlockMat& q, int fmt, uint16_t* out, int64_t ld, hipStream_t st);

// C [M, N] bf16 (row pitch ldc) = sum over k of A(m, k) B(n, k): A [M, R]
// and B [N, R] block-scaled over the same R. ws: FP32 partials of a split
// reduction (block_gemm_ws_bytes of them), or null: never split.
struct BlockGemm {
  BlockMat A, B;
  int fa, fb;
  uint16_t* C;
  int64_t ldc;
};
size_t block_gemm_ws_bytes(int64_t M, int64_t N, int64_t R);
void block_gemm_plan(int64_t M, int64_t N, int64_t R, int* tile_m, int* tile_n, int* splits);
hipError_t launch_block_gemm(const BlockGemm& g, void* ws, size_t ws_bytes, hipStream_t st);

// Y [M, N] bf16 (dense) = X [M, K] W for few rows of X, W stored as w [N, K]
// in E4M3. Fused: X is bf16 and of at most kServeBlocks blocks of 128 (two
// rows of K = 8192: 20.1 us against 21.6 with X quantised by a launch of its
// own, which is what more blocks cost). Otherwise X comes stored, of at most
// 16 rows, or 32 where a workgroup has 16 columns or more to read it for (32
// rows by 12288: 19.1 us; the tiled product 24).
constexpr int64_t kServeBlocks = 256;
bool block_serve_fused(int64_t M, int64_t K);
bool block_serve_takes(int64_t M, int64_t N);
hipError_t launch_block_serve_fused(const Bf16Mat& x, const BlockMat& w, uint16_t* y, hipStream_t st);
hipError_t launch_block_serve(const BlockMat& xq, const BlockMat& w, uint16_t* y, hipStream_t st);

// SwiGLU: h = g sigmoid(g) u. Outputs that are null are not written:
// h bf16 [rows, cols]; hq its E4M3 form; gq, uq the E4M3 forms of g and u.
hipError_t launch_swiglu_fwd(const Bf16Mat& gate, const Bf16Mat& up, uint16_t* h, int64_t ldh, const BlockMat& hq,
                             const BlockMat& gq, const BlockMat& uq, hipStream_t st);
// gradients from the 8-bit g and u: dg, du bf16
hipError_t launch_swiglu_bwd(const Bf16Mat& dh, const BlockMat& gq, const BlockMat& uq, uint16_t* dg, int64_t lddg,
                             uint16_t* du, int64_t lddu, hipStream_t st);
// the same gradients straight to E5M2: dgq, duq [rows, cols] (row form of
// the concatenated gradient, in halves), dgut [2 cols, rows] (transposed,
// dg's rows then du's) and ht [cols, rows] the E4M3 transposed h
hipError_t launch_swiglu_bwd_quant(const Bf16Mat& dh, const BlockMat& gq, const BlockMat& uq, const BlockMat& dgq,
                                   const BlockMat& duq, const BlockMat& dgut, const BlockMat& ht, hipStream_t st);

}  // namespace fp8lin
