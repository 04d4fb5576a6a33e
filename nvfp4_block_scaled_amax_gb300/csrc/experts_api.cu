// experts_api.cu -- the C ABI of the expert-layer operators (include/nvfp4.h):
// host-side validation before anything is enqueued, then the launches.
#include "fp8.h"
#include "nvfp4.h"
#include "tokens.h"

namespace nvfp4 {

nvfp4_status make_launch_ctx(void* stream, LaunchCtx* ctx);

namespace {

static_assert(NVFP4_MAX_EXPERTS == kMaxExperts, "expert table size");

nvfp4_status status_of(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }
bool aligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
constexpr int64_t kLimit = (int64_t)1 << 31;  // rows, columns, slots
bool size_ok(int64_t v) { return v >= 0 && v < kLimit; }

int64_t capacity(int64_t slots, int experts, int align) {
  return (slots + (int64_t)experts * (align - 1)) / align * align;
}

nvfp4_status check_sort(int64_t tokens, int topk, int experts, int align) {
  if (!size_ok(tokens) || topk < 1 || topk > NVFP4_MAX_TOPK || experts < 1 || experts > kMaxExperts || align < 1 ||
      align > NVFP4_MAX_ALIGN)
    return NVFP4_ERR_SHAPE;
  if (!size_ok(tokens * topk) || !size_ok(capacity(tokens * topk, experts, align))) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

nvfp4_status check_sort_call(const int32_t* ids, int64_t tokens, int topk, int experts, int align,
                             const int32_t* offsets, const int32_t* row_of_slot, const int32_t* slot_of_row,
                             int64_t rows, const void* scratch, size_t scratch_bytes) {
  nvfp4_status st = check_sort(tokens, topk, experts, align);
  if (st != NVFP4_OK) return st;
  if (rows != capacity(tokens * topk, experts, align)) return NVFP4_ERR_SHAPE;
  if (offsets == nullptr || (tokens > 0 && (ids == nullptr || row_of_slot == nullptr)) ||
      (rows > 0 && slot_of_row == nullptr))
    return NVFP4_ERR_NULL;
  const size_t need = sizeof(int) * (size_t)sort_scratch_ints(tokens * topk, experts);
  if (scratch_bytes < need) return NVFP4_ERR_SHAPE;
  if (need > 0 && scratch == nullptr) return NVFP4_ERR_NULL;
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(row_of_slot, 4) || !aligned(slot_of_row, 4) ||
      !aligned(scratch, 4))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

// Checks of the calls that move rows: sizes, and 16-byte rows.
nvfp4_status check_rows(int dtype, int64_t tokens, int64_t width, int topk, int64_t rows) {
  if (dtype != NVFP4_BF16 && dtype != NVFP4_FP32) return NVFP4_ERR_DTYPE;
  if (!size_ok(tokens) || !size_ok(width) || !size_ok(rows) || topk < 1 || topk > NVFP4_MAX_TOPK ||
      !size_ok(tokens * topk))
    return NVFP4_ERR_SHAPE;
  if (width * (dtype == NVFP4_BF16 ? 2 : 4) % 16 != 0) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

SortArgs sort_args(const int32_t* ids, int64_t tokens, int topk, int experts, int align, int32_t* offsets,
                   int32_t* row_of_slot, int32_t* slot_of_row, int64_t rows, void* scratch) {
  SortArgs a = {};
  a.ids = ids;
  a.slots = tokens * topk;
  a.experts = experts;
  a.align = align;
  a.rows = rows;
  a.offsets = offsets;
  a.row_of_slot = row_of_slot;
  a.slot_of_row = slot_of_row;
  a.scratch = static_cast<int32_t*>(scratch);
  return a;
}

TokenArgs token_args(int dtype, int64_t tokens, int64_t width, int topk, int64_t rows, const int32_t* row_of_slot,
                     const int32_t* slot_of_row, const float* weights) {
  TokenArgs a = {};
  a.tokens = tokens;
  a.width = width;
  a.rows = rows;
  a.topk = topk;
  a.bf16 = dtype == NVFP4_BF16;
  a.row_of_slot = row_of_slot;
  a.slot_of_row = slot_of_row;
  a.weights = weights;
  return a;
}

nvfp4_status matmul(Fp8MatmulArgs m, int out_dtype, void* stream) {
  if (out_dtype != NVFP4_BF16 && out_dtype != NVFP4_FP32) return NVFP4_ERR_DTYPE;
  if (m.b_block_rows != 1 && m.b_block_rows != kFp8Block) return NVFP4_ERR_SHAPE;
  if (!size_ok(m.a_rows) || !size_ok(m.a_cols) || !size_ok(m.b_rows) || m.a_cols % 16 != 0) return NVFP4_ERR_SHAPE;
  if (m.experts < 1 || m.experts > kMaxExperts) return NVFP4_ERR_SHAPE;
  // one coordinate and one tile index for the whole call
  if (!size_ok(m.experts * m.b_rows) || !size_ok(m.experts * m.a_rows)) return NVFP4_ERR_SHAPE;
  const int64_t tiles = (fp8_blocks(m.a_rows) + 1) * (fp8_blocks(m.b_rows) + 1);
  if (!size_ok(tiles) || !size_ok(2 * tiles * m.experts)) return NVFP4_ERR_SHAPE;
  if (!aligned(m.a, 16) || !aligned(m.b, 16) || !aligned(m.out, 16) || !aligned(m.sa, 4) || !aligned(m.sb, 4) ||
      !aligned(m.offsets, 4))
    return NVFP4_ERR_ALIGN;
  if (m.a_rows > 0 && m.b_rows > 0) {
    if (m.out == nullptr) return NVFP4_ERR_NULL;
    if (m.a_cols > 0 && (m.a == nullptr || m.sa == nullptr || m.b == nullptr || m.sb == nullptr))
      return NVFP4_ERR_NULL;
  }
  LaunchCtx ctx;
  nvfp4_status st = make_launch_ctx(stream, &ctx);
  if (st != NVFP4_OK) return st;
  m.out_bf16 = out_dtype == NVFP4_BF16;
  return status_of(launch_fp8_matmul(m, ctx));
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

nvfp4_status nvfp4_token_rows(int64_t tokens, int topk, int num_experts, int align, int64_t* rows,
                              size_t* scratch_bytes) {
  if (rows == nullptr || scratch_bytes == nullptr) return NVFP4_ERR_NULL;
  nvfp4_status st = check_sort(tokens, topk, num_experts, align);
  if (st != NVFP4_OK) return st;
  *rows = capacity(tokens * topk, num_experts, align);
  *scratch_bytes = sizeof(int) * (size_t)sort_scratch_ints(tokens * topk, num_experts);
  return NVFP4_OK;
}

nvfp4_status nvfp4_sort_tokens(const int32_t* expert_ids, int64_t tokens, int topk, int num_experts, int align,
                               int32_t* offsets, int32_t* row_of_slot, int32_t* slot_of_row, int64_t rows,
                               void* scratch, size_t scratch_bytes, void* stream) {
  nvfp4_status st = check_sort_call(expert_ids, tokens, topk, num_experts, align, offsets, row_of_slot, slot_of_row,
                                    rows, scratch, scratch_bytes);
  if (st != NVFP4_OK) return st;
  LaunchCtx ctx;
  if ((st = make_launch_ctx(stream, &ctx)) != NVFP4_OK) return st;
  return status_of(launch_sort_tokens(
      sort_args(expert_ids, tokens, topk, num_experts, align, offsets, row_of_slot, slot_of_row, rows, scratch), ctx));
}

nvfp4_status nvfp4_gather_tokens(const void* x, int dtype, int64_t tokens, int64_t width, int topk,
                                 const int32_t* row_of_slot, const int32_t* slot_of_row, int64_t rows, void* out,
                                 void* stream) {
  nvfp4_status st = check_rows(dtype, tokens, width, topk, rows);
  if (st != NVFP4_OK) return st;
  if ((tokens > 0 && row_of_slot == nullptr) || (rows > 0 && slot_of_row == nullptr)) return NVFP4_ERR_NULL;
  if (width > 0 && ((tokens > 0 && x == nullptr) || (rows > 0 && out == nullptr))) return NVFP4_ERR_NULL;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(row_of_slot, 4) || !aligned(slot_of_row, 4))
    return NVFP4_ERR_ALIGN;
  LaunchCtx ctx;
  if ((st = make_launch_ctx(stream, &ctx)) != NVFP4_OK) return st;
  return status_of(launch_gather_tokens(
      x, out, token_args(dtype, tokens, width, topk, rows, row_of_slot, slot_of_row, nullptr), ctx));
}

nvfp4_status nvfp4_dispatch_tokens(const void* x, int dtype, int64_t tokens, int64_t width,
                                   const int32_t* expert_ids, int topk, int num_experts, int align,
                                   int32_t* offsets, int32_t* row_of_slot, int32_t* slot_of_row, int64_t rows,
                                   void* out, void* scratch, size_t scratch_bytes, void* stream) {
  nvfp4_status st = check_sort_call(expert_ids, tokens, topk, num_experts, align, offsets, row_of_slot, slot_of_row,
                                    rows, scratch, scratch_bytes);
  if (st != NVFP4_OK) return st;
  if ((st = check_rows(dtype, tokens, width, topk, rows)) != NVFP4_OK) return st;
  if (width > 0 && ((tokens > 0 && x == nullptr) || (rows > 0 && out == nullptr))) return NVFP4_ERR_NULL;
  if (!aligned(x, 16) || !aligned(out, 16)) return NVFP4_ERR_ALIGN;
  LaunchCtx ctx;
  if ((st = make_launch_ctx(stream, &ctx)) != NVFP4_OK) return st;
  const SortArgs s =
      sort_args(expert_ids, tokens, topk, num_experts, align, offsets, row_of_slot, slot_of_row, rows, scratch);
  const TokenArgs a = token_args(dtype, tokens, width, topk, rows, row_of_slot, slot_of_row, nullptr);
  return status_of(launch_dispatch_tokens(s, x, out, a, ctx));
}

nvfp4_status nvfp4_combine_tokens(const void* rows_in, int dtype, int64_t tokens, int64_t width, int topk,
                                  const int32_t* row_of_slot, int64_t rows, const float* weights, void* y,
                                  void* stream) {
  nvfp4_status st = check_rows(dtype, tokens, width, topk, rows);
  if (st != NVFP4_OK) return st;
  if (tokens > 0 && row_of_slot == nullptr) return NVFP4_ERR_NULL;
  if (tokens > 0 && width > 0 && (y == nullptr || (rows > 0 && rows_in == nullptr))) return NVFP4_ERR_NULL;
  if (!aligned(rows_in, 16) || !aligned(y, 16) || !aligned(row_of_slot, 4) || !aligned(weights, 4))
    return NVFP4_ERR_ALIGN;
  LaunchCtx ctx;
  if ((st = make_launch_ctx(stream, &ctx)) != NVFP4_OK) return st;
  return status_of(launch_combine_tokens(
      rows_in, y, token_args(dtype, tokens, width, topk, rows, row_of_slot, nullptr, weights), ctx));
}

nvfp4_status nvfp4_combine_tokens_grad(const void* dy, const void* rows_in, int dtype, int64_t tokens, int64_t width,
                                       int topk, const int32_t* row_of_slot, const int32_t* slot_of_row,
                                       int64_t rows, const float* weights, void* drows, float* dweights,
                                       void* stream) {
  nvfp4_status st = check_rows(dtype, tokens, width, topk, rows);
  if (st != NVFP4_OK) return st;
  if ((tokens > 0 && row_of_slot == nullptr) || (rows > 0 && slot_of_row == nullptr)) return NVFP4_ERR_NULL;
  if (!size_ok(tokens + (rows + 31) / 32)) return NVFP4_ERR_SHAPE;  // one CTA each
  if (width > 0 && ((tokens > 0 && dy == nullptr) || (rows > 0 && (rows_in == nullptr || drows == nullptr))))
    return NVFP4_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(rows_in, 16) || !aligned(drows, 16) || !aligned(row_of_slot, 4) ||
      !aligned(slot_of_row, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
    return NVFP4_ERR_ALIGN;
  LaunchCtx ctx;
  if ((st = make_launch_ctx(stream, &ctx)) != NVFP4_OK) return st;
  return status_of(launch_combine_tokens_grad(
      dy, rows_in, drows, dweights, token_args(dtype, tokens, width, topk, rows, row_of_slot, slot_of_row, weights),
      ctx));
}

nvfp4_status nvfp4_fp8_quantize(const void* x, int dtype, int64_t batch, int64_t M, int64_t N, int block_rows,
                                uint8_t* data_row, float* scale_row, uint8_t* data_col, float* scale_col,
                                unsigned flags, void* stream) {
  if (flags & ~(NVFP4_ROWWISE | NVFP4_COLWISE)) return NVFP4_ERR_FLAGS;
  const bool row = flags & NVFP4_ROWWISE, col = flags & NVFP4_COLWISE;
  if (!row && !col) return NVFP4_ERR_FLAGS;
  if (dtype != NVFP4_BF16 && dtype != NVFP4_FP32) return NVFP4_ERR_DTYPE;
  if (block_rows != 1 && block_rows != kFp8Block) return NVFP4_ERR_SHAPE;
  if (!size_ok(batch) || !size_ok(M) || !size_ok(N) || !size_ok(batch * M) || !size_ok(batch * N))
    return NVFP4_ERR_SHAPE;
  if (N % 16 != 0 || (col && M % 16 != 0)) return NVFP4_ERR_SHAPE;
  if (!size_ok(fp8_blocks(M) * fp8_blocks(N)) || !size_ok(batch * fp8_blocks(M) * fp8_blocks(N)))
    return NVFP4_ERR_SHAPE;
  if (batch > 0 && M > 0 && N > 0) {
    if (x == nullptr) return NVFP4_ERR_NULL;
    if ((row && (data_row == nullptr || scale_row == nullptr)) || (col && (data_col == nullptr || scale_col == nullptr)))
      return NVFP4_ERR_NULL;
  }
  if (!aligned(x, 16) || (row && (!aligned(data_row, 16) || !aligned(scale_row, 4))) ||
      (col && (!aligned(data_col, 16) || !aligned(scale_col, 4))))
    return NVFP4_ERR_ALIGN;
  LaunchCtx ctx;
  nvfp4_status st = make_launch_ctx(stream, &ctx);
  if (st != NVFP4_OK) return st;
  Fp8CastArgs a = {};
  a.batch = batch;
  a.M = M;
  a.N = N;
  a.bf16 = dtype == NVFP4_BF16;
  a.block_rows = block_rows;
  a.data_row = row ? data_row : nullptr;
  a.scale_row = row ? scale_row : nullptr;
  a.data_col = col ? data_col : nullptr;
  a.scale_col = col ? scale_col : nullptr;
  return status_of(launch_fp8_cast(x, a, ctx));
}

nvfp4_status nvfp4_fp8_matmul(const uint8_t* a, const float* a_scale, const uint8_t* b, const float* b_scale,
                              int b_block_rows, int64_t M, int64_t N, int64_t K, void* out, int out_dtype,
                              void* stream) {
  Fp8MatmulArgs m = {};
  m.a = a;
  m.sa = a_scale;
  m.b = b;
  m.sb = b_scale;
  m.a_rows = M;
  m.a_cols = K;
  m.b_rows = N;
  m.b_block_rows = b_block_rows;
  m.experts = 1;
  m.out = out;
  return matmul(m, out_dtype, stream);
}

nvfp4_status nvfp4_fp8_matmul_grouped(const uint8_t* a, const float* a_scale, const uint8_t* b, const float* b_scale,
                                      int b_block_rows, int64_t rows, int64_t N, int64_t K, int num_experts,
                                      const int32_t* offsets, void* out, int out_dtype, void* stream) {
  if (offsets == nullptr) return NVFP4_ERR_NULL;
  Fp8MatmulArgs m = {};
  m.a = a;
  m.sa = a_scale;
  m.b = b;
  m.sb = b_scale;
  m.a_rows = rows;
  m.a_cols = K;
  m.b_rows = N;
  m.b_block_rows = b_block_rows;
  m.experts = num_experts;
  m.offsets = offsets;
  m.out = out;
  return matmul(m, out_dtype, stream);
}

nvfp4_status nvfp4_fp8_matmul_grouped_wgrad(const uint8_t* a, const float* a_scale, const uint8_t* b,
                                            const float* b_scale, int64_t M, int64_t N, int64_t rows,
                                            int num_experts, const int32_t* offsets, void* out, int out_dtype,
                                            void* stream) {
  if (offsets == nullptr) return NVFP4_ERR_NULL;
  Fp8MatmulArgs m = {};
  m.a = a;
  m.sa = a_scale;
  m.b = b;
  m.sb = b_scale;
  m.a_rows = M;
  m.a_cols = rows;
  m.b_rows = N;
  m.b_block_rows = 1;
  m.experts = num_experts;
  m.offsets = offsets;
  m.wgrad = true;
  m.out = out;
  return matmul(m, out_dtype, stream);
}

}  // extern "C"
