// tokens.h -- internal launchers of the token sort, gather and combine
// kernels (tokens.cu); arguments validated by the C-ABI layer (experts_api.cu).
#pragma once

#include "kernels.h"

namespace nvfp4 {

constexpr int kMaxExperts = 1024;

// Chunks the sort cuts `slots` into (one CTA each), and the bytes of scratch
// it needs: a count per chunk and expert (none for a single chunk).
int sort_chunks(int64_t slots, const LaunchCtx& ctx);
int64_t sort_scratch_ints(int64_t slots, int experts);

struct SortArgs {
  const int32_t* ids;   // [slots], outside 0..experts-1: dropped
  int64_t slots;
  int experts, align;
  int64_t rows;         // capacity
  int32_t* offsets;     // [experts + 1]
  int32_t* row_of_slot; // [slots]
  int32_t* slot_of_row; // [rows]
  int32_t* scratch;
};
cudaError_t launch_sort_tokens(const SortArgs& a, const LaunchCtx& ctx);

struct TokenArgs {
  int64_t tokens, width, rows;
  int topk;
  bool bf16;
  const int32_t* row_of_slot;
  const int32_t* slot_of_row;
  const float* weights;  // [tokens, topk] or NULL (all 1)
};
// out[r] = x[slot_of_row[r] / topk], zero where there is no slot.
cudaError_t launch_gather_tokens(const void* x, void* out, const TokenArgs& a, const LaunchCtx& ctx);
// The sort, then the gather; in one launch where there are few slots.
cudaError_t launch_dispatch_tokens(const SortArgs& s, const void* x, void* out, const TokenArgs& t,
                                   const LaunchCtx& ctx);
cudaError_t launch_combine_tokens(const void* rows, void* y, const TokenArgs& a, const LaunchCtx& ctx);
cudaError_t launch_combine_tokens_grad(const void* dy, const void* rows, void* drows, float* dweights,
                                       const TokenArgs& a, const LaunchCtx& ctx);

}  // namespace nvfp4
