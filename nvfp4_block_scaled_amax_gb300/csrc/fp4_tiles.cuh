// fp4_tiles.cuh -- what the product kernels of 4-bit operands share: the
// block-scaled MMA, scales on their way into tensor memory, and the factor of
// the output.
//
// A stage holds 256 elements (128 bytes of codes) of the contracted dimension.
// The MMA of 64 elements takes the scales of its rows from tensor memory: 32
// lanes, four rows 32 apart in four columns, four scales (16 elements each, or
// 32) to a column's word.  That is the order of a 512-byte tile of the 128x4
// layout, so a swizzled operand's scales are copied to shared memory as they
// stand; compact ones are put into that order by warps that read them a row at
// a time.
#pragma once

#include "fp4.h"
#include "fp8_tiles.cuh"

namespace nvfp4 {
namespace fp4 {

using fp8::cluster_arrive;
using fp8::cluster_arrive_relaxed;
using fp8::cluster_rank;
using fp8::cluster_sync;
using fp8::cluster_wait;
using fp8::elect_one;
using fp8::map_to_cta;
using fp8::mbar_arrive;
using fp8::mbar_arrive_cluster;
using fp8::mbar_arrive_cluster_release;
using fp8::mbar_wait;
using fp8::mbar_wait_cluster;
using fp8::operand_desc;
using fp8::report_timeout;
using fp8::store_async;
using fp8::tma_load;
using fp8::tma_load_pair;
using fp8::tma_store;
using fp8::tmem_alloc_pair;
using fp8::tmem_dealloc_pair;
using fp8::tmem_read;
using fp8::umma_commit_pair;
using fp8::warp_index;

constexpr int kStageK = 256;      // elements of a stage
constexpr int kStageRow = 128;    // their bytes in a row
constexpr int kScaleTile = 512;   // bytes of 128 rows x 4 scales

struct MatmulKernelArgs {
  Fp4Side a, b;
  int64_t K;
  void* out;
  int out_bf16, out_map;
  int tiles_a, tiles_b;
  unsigned* status;
};

// kBlock 16: NVFP4 (E4M3 scales), 32: MXFP4 (powers of two).
template <int kBlock>
struct Format {
  static constexpr int kRowBytes = kStageK / kBlock;       // scales of a row and stage
  static constexpr int kTiles = kRowBytes / 4;             // tiles of 128 rows x 4 scales in a stage
  static constexpr int kScaleBytes = kTiles * kScaleTile;  // of 128 rows and a stage
  static constexpr int kCols = 4 * kTiles;                 // tensor-memory columns they take
  // Instruction descriptor: E2M1 A and B, both K-major, FP32 D, the scales' type.
  static constexpr __host__ __device__ uint32_t idesc(int m, int n) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((kBlock == 32 ? 1u : 0u) << 23) |
           ((uint32_t)(m >> 7) << 27);
  }
  // Column of the stage's first that holds step k's scales, and the
  // descriptor's bits that select the half of its words (MXFP4 uses two scales a
  // step).
  static constexpr __device__ int col(int k) { return kBlock == 32 ? 4 * (k >> 1) : 4 * k; }
  static constexpr __device__ uint32_t half(int k) {
    return kBlock == 32 && (k & 1) ? (2u << 4) | (2u << 29) : 0u;
  }
};

// D (tensor memory) = A * B (+ D when accumulate) over 64 elements, with the
// scales at sa and sb; issued by one thread.
template <int kGroup, int kBlock>
__device__ __forceinline__ void umma_fp4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sa,
                                         uint32_t sb, uint32_t accumulate) {
  if constexpr (kGroup == 2 && kBlock == 16)
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p;\n}" ::"r"(
                     d_tmem),
                 "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb)
                 : "memory");
  else if constexpr (kGroup == 2)
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n}" ::"r"(
                     d_tmem),
                 "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb)
                 : "memory");
  else if constexpr (kBlock == 16)
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p;\n}" ::"r"(
                     d_tmem),
                 "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb)
                 : "memory");
  else
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n}" ::"r"(
                     d_tmem),
                 "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb)
                 : "memory");
}

// One tile of scales (32 x 16 bytes) from shared memory into four columns, the
// same in all four groups of 32 lanes; before the MMAs that the thread issues
// later, after those it issued earlier.
template <int kGroup>
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t desc) {
  if constexpr (kGroup == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Descriptor of a tile of scales: no swizzle, 8 rows of 16 bytes a core matrix.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) { return umma_smem_desc(addr, 16, 128, 0); }

// Bytes of a swizzled operand's scales of 128 rows in the stage from element
// k0 on, and where they begin.
template <int kBlock>
__device__ __forceinline__ uint32_t swizzled_bytes(int64_t K, int64_t k0) {
  const int64_t tiles = (K - k0) / (4 * kBlock);  // (K is a multiple of 128)
  return (uint32_t)(tiles < Format<kBlock>::kTiles ? tiles : Format<kBlock>::kTiles) * kScaleTile;
}
template <int kBlock>
__device__ __forceinline__ const uint8_t* swizzled_at(const Fp4Side& s, int64_t K, int64_t row, int64_t k0) {
  return s.scale + ((row >> 7) * (K / (4 * kBlock)) + k0 / (4 * kBlock)) * kScaleTile;
}

// The scales of one row and stage, compact, as words; zeros past the row's end
// and for a row that does not exist (n 0).  n: bytes there are.
template <int kWords>
__device__ __forceinline__ void compact_scales(const uint8_t* p, int n, uint32_t (&v)[kWords]) {
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
  if (n == 4 * kWords && off % (4 * kWords) == 0) {
    if constexpr (kWords == 4) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
      v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    } else {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
      v[0] = w.x, v[1] = w.y;
    }
    return;
  }
  // Words that hold a byte of the row, moved into place.
  const uint32_t sh = (off & 3) * 8;
  const uint32_t* q = reinterpret_cast<const uint32_t*>(p - (off & 3));
  uint32_t w[kWords + 1];
#pragma unroll
  for (int i = 0; i <= kWords; ++i) w[i] = 4 * i < n + (int)(off & 3) && n > 0 ? __ldg(q + i) : 0u;
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    const int left = n - 4 * i;  // bytes of this word that the row has
    const uint32_t x = __funnelshift_r(w[i], w[i + 1], sh);
    v[i] = left >= 4 ? x : left <= 0 ? 0u : x & ((1u << (8 * left)) - 1);
  }
}

// The factor of an output: value * first * second, in that order.  One
// product where it is a normal number; else one after the other, the larger
// first where both together are too small, the smaller first where they are too
// large: a sum (0, or 2^-20 to 2^60) times both may be a normal number all the
// same.
struct Factor {
  float first, second;
  __device__ __forceinline__ float operator()(float v) const { return __fmul_rn(__fmul_rn(v, first), second); }
};
__device__ __forceinline__ Factor factor(float a, float b) {
  const float both = __fmul_rn(a, b);
  if (both < 0x1p-126f && a > 0.0f && b > 0.0f) return {fmaxf(a, b), fminf(a, b)};
  if (both > 0x1.fffffep127f && a <= 0x1.fffffep127f && b <= 0x1.fffffep127f) return {fminf(a, b), fmaxf(a, b)};
  return {both, 1.0f};
}
// amax / 2688 of a row (1 of an MXFP4 operand).
__device__ __forceinline__ float row_factor(const Fp4Side& s, int64_t row) {
  if (s.amax == nullptr) return 1.0f;
  return __fdiv_rn(s.amax[s.amax_per_row ? (row < s.rows ? row : s.rows - 1) : 0], 2688.0f);
}

// fp4_matmul_thin.cu
struct ThinPlan {
  int bn, split;
  int64_t tiles;
};
ThinPlan thin_plan(const Fp4MatmulArgs& a, const LaunchCtx& ctx);
cudaError_t launch_matmul_thin(const Fp4MatmulArgs& a, MatmulKernelArgs p, const LaunchCtx& ctx);

}  // namespace fp4
}  // namespace nvfp4
