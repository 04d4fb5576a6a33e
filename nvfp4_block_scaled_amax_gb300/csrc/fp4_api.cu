// fp4_api.cu -- the C ABI of the 4-bit operators (include/nvfp4.h): host-side
// validation before anything is enqueued, then the launches.
#include "fp4.h"
#include "nvfp4.h"

namespace nvfp4 {

nvfp4_status make_launch_ctx(void* stream, LaunchCtx* ctx);

namespace {

nvfp4_status status_of(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }
bool aligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
constexpr int64_t kLimit = (int64_t)1 << 31;  // rows, columns, tiles
bool size_ok(int64_t v) { return v >= 0 && v < kLimit; }
int64_t blocks128(int64_t n) { return (n + 127) / 128; }

nvfp4_status check_operand(const nvfp4_operand* o, int block, int64_t rows, int64_t K) {
  if (o->flags & ~(NVFP4_SWIZZLED | NVFP4_ROW_SCALED)) return NVFP4_ERR_FLAGS;
  if (block == 32 && (o->amax != nullptr || (o->flags & NVFP4_ROW_SCALED))) return NVFP4_ERR_FLAGS;
  const bool swizzled = o->flags & NVFP4_SWIZZLED;
  if (swizzled && (rows % 128 != 0 || K % 128 != 0)) return NVFP4_ERR_ALIGN;
  if (rows > 0 && K > 0 && (o->data == nullptr || o->scale == nullptr || (block == 16 && o->amax == nullptr)))
    return NVFP4_ERR_NULL;
  if (!aligned(o->data, 16) || (swizzled && !aligned(o->scale, 16)) || !aligned(o->amax, 4)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

static_assert(NVFP4_MAX_TOPK == kMaxTopk, "limits of the header");
static_assert(NVFP4_MAX_MLP_SLOTS == kMaxMlpSlots && NVFP4_MAX_MLP_WIDTH == kMaxMlpWidth, "limits of the header");

nvfp4_status check_mlp(int64_t tokens, int topk, int experts, int64_t hidden, int64_t inner) {
  if (tokens < 0 || tokens > kMaxMlpSlots || topk < 1 || topk > NVFP4_MAX_TOPK || tokens * topk > kMaxMlpSlots)
    return NVFP4_ERR_SHAPE;
  if (experts < 1 || experts > NVFP4_MAX_EXPERTS) return NVFP4_ERR_SHAPE;
  for (int64_t v : {hidden, inner})
    if (v < 0 || v > kMaxMlpWidth || v % 32 != 0) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

// A stack of weight matrices.
nvfp4_status check_experts(const nvfp4_operand* o, int block, bool any) {
  if (o->flags & NVFP4_SWIZZLED) return NVFP4_ERR_FLAGS;
  return check_operand(o, block, any, any);
}

Fp4Side side(const nvfp4_operand* o, int64_t rows) {
  return {o->data, o->scale, o->amax, rows, (o->flags & NVFP4_ROW_SCALED) != 0, (o->flags & NVFP4_SWIZZLED) != 0};
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

nvfp4_status nvfp4_mxfp4_quantize(const void* x, int dtype, int64_t M, int64_t N, uint8_t* data_row,
                                  uint8_t* scale_row, uint8_t* data_col, uint8_t* scale_col, unsigned flags,
                                  void* stream) {
  if (flags & ~(NVFP4_ROWWISE | NVFP4_COLWISE | NVFP4_SWIZZLED)) return NVFP4_ERR_FLAGS;
  const bool row = flags & NVFP4_ROWWISE, col = flags & NVFP4_COLWISE, swizzled = flags & NVFP4_SWIZZLED;
  if (!row && !col) return NVFP4_ERR_FLAGS;
  if (dtype != NVFP4_BF16 && dtype != NVFP4_FP32) return NVFP4_ERR_DTYPE;
  if (M < 0 || N < 0 || !size_ok(M + 512) || !size_ok(N + 512) || N % 32 != 0 || (col && M % 32 != 0))
    return NVFP4_ERR_SHAPE;
  if (swizzled && (M % 128 != 0 || N % 128 != 0)) return NVFP4_ERR_ALIGN;
  if (M > 0 && N > 0 && (x == nullptr || (row && (data_row == nullptr || scale_row == nullptr)) ||
                         (col && (data_col == nullptr || scale_col == nullptr))))
    return NVFP4_ERR_NULL;
  if (!aligned(x, 16) || (row && !aligned(data_row, 16)) || (col && !aligned(data_col, 16))) return NVFP4_ERR_ALIGN;
  if (swizzled && ((row && !aligned(scale_row, 16)) || (col && !aligned(scale_col, 16)))) return NVFP4_ERR_ALIGN;
  LaunchCtx ctx;
  const nvfp4_status st = make_launch_ctx(stream, &ctx);
  if (st != NVFP4_OK) return st;
  MxCastArgs a = {};
  a.M = M;
  a.N = N;
  a.bf16 = dtype == NVFP4_BF16;
  a.swizzled = swizzled;
  a.data_row = row ? data_row : nullptr;
  a.scale_row = row ? scale_row : nullptr;
  a.data_col = col ? data_col : nullptr;
  a.scale_col = col ? scale_col : nullptr;
  return status_of(launch_mxfp4_cast(x, a, ctx));
}

nvfp4_status nvfp4_mxfp4_dequantize(const uint8_t* data, const uint8_t* scale, int64_t rows, int64_t cols,
                                    unsigned flags, void* out, int out_dtype, void* stream) {
  if (flags & ~NVFP4_SWIZZLED) return NVFP4_ERR_FLAGS;
  if (out_dtype != NVFP4_BF16 && out_dtype != NVFP4_FP32) return NVFP4_ERR_DTYPE;
  if (!size_ok(rows) || !size_ok(cols) || cols % 32 != 0) return NVFP4_ERR_SHAPE;
  if ((flags & NVFP4_SWIZZLED) && (rows % 128 != 0 || cols % 128 != 0)) return NVFP4_ERR_ALIGN;
  if (rows > 0 && cols > 0 && (data == nullptr || scale == nullptr || out == nullptr)) return NVFP4_ERR_NULL;
  if (!aligned(data, 16) || !aligned(out, 32)) return NVFP4_ERR_ALIGN;
  LaunchCtx ctx;
  const nvfp4_status st = make_launch_ctx(stream, &ctx);
  if (st != NVFP4_OK) return st;
  return status_of(launch_mxfp4_dequantize(data, scale, rows, cols, (flags & NVFP4_SWIZZLED) != 0, out,
                                           out_dtype == NVFP4_BF16, ctx));
}

nvfp4_status nvfp4_fp4_matmul(const nvfp4_operand* a, const nvfp4_operand* b, int block, int64_t M, int64_t N,
                              int64_t K, void* out, int out_dtype, void* stream) {
  if (a == nullptr || b == nullptr) return NVFP4_ERR_NULL;
  if (out_dtype != NVFP4_BF16 && out_dtype != NVFP4_FP32) return NVFP4_ERR_DTYPE;
  if (block != 16 && block != 32) return NVFP4_ERR_SHAPE;
  // (a row index past the last tile; a tile's sum within the limit of a wait)
  if (M < 0 || N < 0 || K < 0 || !size_ok(M + 512) || !size_ok(N + 512) || K > NVFP4_MAX_FP4_K || K % 32 != 0)
    return NVFP4_ERR_SHAPE;
  if (!size_ok(blocks128(M) * blocks128(N))) return NVFP4_ERR_SHAPE;  // one tile index
  nvfp4_status st = check_operand(a, block, M, K);
  if (st != NVFP4_OK) return st;
  if ((st = check_operand(b, block, N, K)) != NVFP4_OK) return st;
  if (M > 0 && N > 0 && out == nullptr) return NVFP4_ERR_NULL;
  if (!aligned(out, 16)) return NVFP4_ERR_ALIGN;
  LaunchCtx ctx;
  if ((st = make_launch_ctx(stream, &ctx)) != NVFP4_OK) return st;
  Fp4MatmulArgs m = {};
  m.a = side(a, M);
  m.b = side(b, N);
  m.K = K;
  m.block = block;
  m.out = out;
  m.out_bf16 = out_dtype == NVFP4_BF16;
  return status_of(launch_fp4_matmul(m, ctx));
}

nvfp4_status nvfp4_expert_mlp_workspace(int64_t tokens, int topk, int num_experts, int64_t hidden, int64_t inner,
                                        int block, size_t* bytes) {
  if (bytes == nullptr) return NVFP4_ERR_NULL;
  if (block != 16 && block != 32) return NVFP4_ERR_SHAPE;
  const nvfp4_status st = check_mlp(tokens, topk, num_experts, hidden, inner);
  if (st != NVFP4_OK) return st;
  ExpertMlpArgs a = {};
  a.tokens = tokens;
  a.topk = topk;
  a.experts = num_experts;
  a.hidden = hidden;
  a.inner = inner;
  a.block = block;
  *bytes = expert_mlp_workspace(a);
  return NVFP4_OK;
}

nvfp4_status nvfp4_expert_mlp(const void* x, int64_t tokens, int64_t hidden, int64_t inner, const nvfp4_operand* up,
                              const nvfp4_operand* down, int block, const int32_t* expert_ids, const float* gates,
                              int topk, int num_experts, void* workspace, size_t workspace_bytes, void* y,
                              void* stream) {
  if (up == nullptr || down == nullptr) return NVFP4_ERR_NULL;
  if (block != 16 && block != 32) return NVFP4_ERR_SHAPE;
  nvfp4_status st = check_mlp(tokens, topk, num_experts, hidden, inner);
  if (st != NVFP4_OK) return st;
  const bool any = tokens > 0 && hidden > 0 && inner > 0;
  if ((st = check_experts(up, block, any)) != NVFP4_OK) return st;
  if ((st = check_experts(down, block, any)) != NVFP4_OK) return st;
  if (tokens > 0 && hidden > 0 && y == nullptr) return NVFP4_ERR_NULL;
  if (any && (x == nullptr || expert_ids == nullptr || gates == nullptr || workspace == nullptr)) return NVFP4_ERR_NULL;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(workspace, 128) || !aligned(expert_ids, 4) || !aligned(gates, 4))
    return NVFP4_ERR_ALIGN;
  ExpertMlpArgs a = {};
  a.x = x;
  a.up = side(up, 0);
  a.down = side(down, 0);
  a.block = block;
  a.ids = expert_ids;
  a.gates = gates;
  a.tokens = tokens;
  a.hidden = hidden;
  a.inner = inner;
  a.topk = topk;
  a.experts = num_experts;
  a.workspace = workspace;
  a.y = y;
  if (any && workspace_bytes < expert_mlp_workspace(a)) return NVFP4_ERR_SHAPE;
  LaunchCtx ctx;
  if ((st = make_launch_ctx(stream, &ctx)) != NVFP4_OK) return st;
  return status_of(launch_expert_mlp(a, ctx));
}

}  // extern "C"
