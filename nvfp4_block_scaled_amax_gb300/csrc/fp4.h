// fp4.h -- internal launchers of the 4-bit operators: the MXFP4 cast and its
// reading back (mxfp4_cast.cu), the product of 4-bit operands (fp4_matmul.cu,
// fp4_matmul_thin.cu) and the gated expert layer for a few tokens
// (expert_mlp.cu); arguments validated by the C-ABI layer (fp4_api.cu).
#pragma once

#include "kernels.h"

namespace nvfp4 {

struct MxCastArgs {
  int64_t M, N;
  bool bf16, swizzled;
  uint8_t* data_row;
  uint8_t* scale_row;
  uint8_t* data_col;
  uint8_t* scale_col;
};
cudaError_t launch_mxfp4_cast(const void* x, const MxCastArgs& a, const LaunchCtx& ctx);
cudaError_t launch_mxfp4_dequantize(const uint8_t* data, const uint8_t* scale, int64_t rows, int64_t cols, bool swizzled,
                                    void* out, bool out_bf16, const LaunchCtx& ctx);

// One operand of a product: [rows][K/2] codes, their scales, and an amax for
// the whole (amax_rows 1) or for each row; NULL: MXFP4, none.
struct Fp4Side {
  const uint8_t* data;
  const uint8_t* scale;
  const float* amax;
  int64_t rows;
  int amax_per_row, swizzled;
};

struct Fp4MatmulArgs {
  Fp4Side a, b;
  int64_t K;
  int block;  // 16: NVFP4, 32: MXFP4
  void* out;  // [a.rows][b.rows]
  bool out_bf16;
};
cudaError_t launch_fp4_matmul(const Fp4MatmulArgs& a, const LaunchCtx& ctx);

constexpr int kMaxTopk = 64;
constexpr int kMaxMlpSlots = 1024;
constexpr int kMaxMlpWidth = 10240;  // hidden and inner sizes

// The gated expert layer for a few tokens (Fp4Side: of all experts; rows and
// swizzled unused, amax_per_row: one amax an expert).
struct ExpertMlpArgs {
  const void* x;   // [tokens][hidden] BF16
  Fp4Side up;      // [experts][2 inner][hidden / 2]: gate rows, then up rows
  Fp4Side down;    // [experts][hidden][inner / 2]
  int block;
  const int32_t* ids;   // [tokens][topk]
  const float* gates;
  int64_t tokens, hidden, inner;
  int topk, experts;
  void* workspace;
  void* y;         // [tokens][hidden] BF16
};
size_t expert_mlp_workspace(const ExpertMlpArgs& a);  // (of its sizes and block)
cudaError_t launch_expert_mlp(const ExpertMlpArgs& a, const LaunchCtx& ctx);

// Tensor map of a row-major byte matrix, box 128 bytes x `box_rows` rows,
// 128-byte swizzle, zero fill outside (fp8.h).
cudaError_t make_fp8_tensor_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int box_rows);
// The same for stores of 4-bit codes: box 64 bytes x 128 rows, 64-byte swizzle.
cudaError_t make_fp4_tensor_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols);
// Swizzled scales: a row for each 128 rows of the operand, `bytes` long; box
// `box_bytes` (at most 2048) x `box_rows`, no swizzle, zero fill outside.
cudaError_t make_scale_tensor_map(CUtensorMap* map, const void* p, int64_t rows, int64_t bytes, int box_bytes,
                                  int box_rows);
// Tensor map of a product (fp8.h).
cudaError_t make_matmul_out_map(CUtensorMap* map, void* out, bool bf16, int64_t rows, int64_t cols);

}  // namespace nvfp4
