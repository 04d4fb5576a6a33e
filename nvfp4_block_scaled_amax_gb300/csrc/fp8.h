// fp8.h -- internal launchers of the E4M3 cast with a scale for each block of
// 128 (fp8_cast.cu) and of the product of such operands (fp8_matmul.cu);
// arguments validated by the C-ABI layer (experts_api.cu).
#pragma once

#include "kernels.h"

namespace nvfp4 {

constexpr int kFp8Block = 128;
inline int64_t fp8_blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

struct Fp8CastArgs {
  int64_t batch, M, N;
  bool bf16;
  int block_rows;  // 1 or 128
  uint8_t* data_row;
  float* scale_row;
  uint8_t* data_col;
  float* scale_col;
};
cudaError_t launch_fp8_cast(const void* x, const Fp8CastArgs& a, const LaunchCtx& ctx);

struct Fp8MatmulArgs {
  const uint8_t* a;     // [a_rows, a_cols]
  const float* sa;      // [blocks(a_cols), a_rows]
  const uint8_t* b;     // [experts, b_rows, a_cols]; wgrad: [b_rows, a_cols]
  const float* sb;
  int64_t a_rows, a_cols, b_rows;
  int b_block_rows;     // 1 or 128
  int experts;
  const int32_t* offsets;  // device, NULL: one member of all of A's rows (wgrad: of all columns)
  bool wgrad;
  void* out;
  bool out_bf16;
};
cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, const LaunchCtx& ctx);

// Tensor map of a row-major byte matrix, box 128 bytes x `box_rows` rows,
// 128-byte swizzle, zero fill outside.
cudaError_t make_fp8_tensor_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int box_rows);

// Tensor map of `batch` row-major matrices M x N of `bytes`-byte elements
// (1: bytes, 2: BF16, 4: FP32), box 128 bytes x 128 rows of one matrix, 128-byte
// swizzle, zero fill outside the matrix.  Needs a 16-byte aligned base and row
// pitch.
cudaError_t make_batch_tensor_map(CUtensorMap* map, const void* p, int bytes, int64_t batch, int64_t M, int64_t N);

// Tensor map of a product [rows][cols] in BF16 or FP32: box 128 bytes x 32
// rows, 128-byte swizzle.  Needs a 16-byte aligned base and row pitch.
cudaError_t make_matmul_out_map(CUtensorMap* map, void* out, bool bf16, int64_t rows, int64_t cols);

}  // namespace nvfp4
