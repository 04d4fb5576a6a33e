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
using fp8::mbar_wait_acquire;
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

// Compact scales on their way into the order of the swizzled layout: stage i's
// words of 128 rows from row0 on, a lane taking four rows 32 apart (zeros past the
// rows there are, past `limit` of the 128, and past a row's end).  A stage's scales
// of a row are 16 (MXFP4: 8) bytes; where rows are not multiples of so many they
// lie at any alignment and are put together from two aligned groups of so many
// bytes, each of which holds at least one byte of the row.
//
// A kernel may begin before the one that writes its operands ends, so scales are
// not constant while it runs: no .nc loads.  Warps that read ahead of the wait for the
// kernel before fence first (stale_lines_gone).  L1 is of use where a row's stages share
// sectors (4096 x 4096 x 4128 44 us, past L1 54); whole sectors are better off without
// it (8192 x 8192 x 8192 167 us past L1, 179 through it).
template <int kBlock>
struct CompactScales {
  static constexpr int kWords = Format<kBlock>::kTiles, kGroup = 4 * kWords;
  const uint8_t* scale;
  int64_t pitch, rows;
  bool whole;  // every stage of every row is a group
  bool pairs;  // and every two stages are two, aligned as such

  __device__ __forceinline__ CompactScales(const uint8_t* at, int64_t K, int64_t rows_)
      : scale(at), pitch(K / kBlock), rows(rows_),
        whole(pitch % kGroup == 0 && (reinterpret_cast<uintptr_t>(at) & (kGroup - 1)) == 0),
        pairs(pitch % (2 * kGroup) == 0 && (reinterpret_cast<uintptr_t>(at) & (2 * kGroup - 1)) == 0) {}

  static __device__ __forceinline__ void group(const uint8_t* p, bool there, uint32_t* w) {
    if constexpr (kWords == 4) {
      const uint4* q = reinterpret_cast<const uint4*>(p);
      const uint4 v = there ? *q : make_uint4(0, 0, 0, 0);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2* q = reinterpret_cast<const uint2*>(p);
      const uint2 v = there ? *q : make_uint2(0, 0);
      w[0] = v.x, w[1] = v.y;
    }
  }
  // gap: rows between the first 64 and the other 64.
  __device__ __forceinline__ void read(int64_t row0, int limit, int i, uint32_t (&v)[4][kWords], int64_t gap = 0) const {
    const int lane = threadIdx.x & 31;
    const uint8_t* p = scale + (row0 + lane) * pitch + (int64_t)i * kGroup;
    auto row = [&](int g) { return 32 * g + (g < 2 ? 0 : gap); };  // after the lane's first
    if (whole) {
#pragma unroll
      for (int g = 0; g < 4; ++g)
        group(p + row(g) * pitch, row0 + lane + row(g) < rows && lane + 32 * g < limit, v[g]);
      return;
    }
    const int n = (int)min((int64_t)kGroup, pitch - (int64_t)i * kGroup);  // bytes of the stage
    uint32_t w[4][2 * kWords];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint8_t* q = p + row(g) * pitch;
      const int off = (int)(reinterpret_cast<uintptr_t>(q) & (kGroup - 1));
      const bool there = row0 + lane + row(g) < rows && lane + 32 * g < limit;
      group(q - off, there, w[g]);
      group(q - off + kGroup, there && off + n > kGroup, w[g] + kWords);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int off = (int)(reinterpret_cast<uintptr_t>(p + row(g) * pitch) & (kGroup - 1));
      uint32_t(&all)[2 * kWords] = w[g];
      if constexpr (kWords == 4) {
#pragma unroll
        for (int k = 0; k < 6; ++k) all[k] = off & 8 ? all[k + 2] : all[k];
      }
#pragma unroll
      for (int k = 0; k <= kWords; ++k) all[k] = off & 4 && k + 1 < 2 * kWords ? all[k + 1] : all[k];
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        const uint32_t x = __funnelshift_r(all[k], all[k + 1], 8 * (off & 3));
        const int left = n - 4 * k;  // bytes of this word that the row has
        v[g][k] = left >= 4 ? x : left <= 0 ? 0u : x & ((1u << (8 * left)) - 1);
      }
    }
  }
  // Stages i and, if there is one, i + 1: where rows allow it, both at once.
  __device__ __forceinline__ void read_two(int64_t row0, int i, bool two, uint32_t (&v)[2][4][kWords]) const {
    const int64_t row = row0 + (threadIdx.x & 31);
    const uint8_t* p = scale + row * pitch + (int64_t)i * kGroup;
    if (!whole) {
      const int n = (int)min((int64_t)2 * kGroup, pitch - (int64_t)i * kGroup);  // bytes of the stages
      uint32_t w[4][3 * kWords];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint8_t* q = p + 32 * g * pitch;
        const int off = (int)(reinterpret_cast<uintptr_t>(q) & (kGroup - 1));
        const bool there = row + 32 * g < rows;
#pragma unroll
        for (int k = 0; k < 3; ++k) group(q - off + k * kGroup, there && off + n > k * kGroup, w[g] + k * kWords);
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int off = (int)(reinterpret_cast<uintptr_t>(p + 32 * g * pitch) & (kGroup - 1));
        uint32_t(&all)[3 * kWords] = w[g];
        if constexpr (kWords == 4) {
#pragma unroll
          for (int k = 0; k < 10; ++k) all[k] = off & 8 ? all[k + 2] : all[k];
        }
#pragma unroll
        for (int k = 0; k <= 2 * kWords; ++k) all[k] = off & 4 ? all[k + 1] : all[k];
#pragma unroll
        for (int k = 0; k < 2 * kWords; ++k) {
          const uint32_t x = __funnelshift_r(all[k], all[k + 1], 8 * (off & 3));
          const int left = n - 4 * k;  // bytes of this word that the row has
          v[k / kWords][g][k % kWords] = left >= 4 ? x : left <= 0 ? 0u : x & ((1u << (8 * left)) - 1);
        }
      }
      return;
    }
#pragma unroll
    for (int g = 0; g < 4; ++g, p += 32 * pitch) {
      uint32_t w[2 * kWords] = {};
      if (!pairs) {
        group(p, row + 32 * g < rows, w);
        group(p + kGroup, row + 32 * g < rows && two, w + kWords);
      } else if (row + 32 * g < rows) {
        if constexpr (kWords == 4) {
          asm volatile("ld.global.cg.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                       : "l"(p));
        } else {
          const uint4 q = *reinterpret_cast<const uint4*>(p);
          w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        }
      }
#pragma unroll
      for (int k = 0; k < kWords; ++k) v[0][g][k] = w[k], v[1][g][k] = w[kWords + k];
    }
  }
  static __device__ __forceinline__ void write(uint32_t to, const uint32_t (&v)[4][kWords]) {
#pragma unroll
    for (int j = 0; j < kWords; ++j)
      sts_v4(to + j * kScaleTile + 16 * (threadIdx.x & 31), v[0][j], v[1][j], v[2][j], v[3][j]);
  }
};

// Ahead of the wait for the kernel before, a warp reads what kernels wrote that were over
// before that one let this one begin.  They have written to L2, but L1 may hold lines of
// the same memory from earlier calls (weights that are loaded anew in place); loads
// behind a fence do not take those.  (Reading past L1 instead: 13 tokens, 4 of 16 experts of
// 2720 x 1184 29.5 us, with the fence 27.8, as without either.)
__device__ __forceinline__ void stale_lines_gone() { __threadfence(); }

// The stages are dealt out to the warps that do this, so that the loads of
// several are in flight; to no more warps than there are slots, for a warp's stage
// may not be two uses of its slot ahead: the barrier's parity would be that of a
// phase long over.
constexpr int kScaleWarps = 4;
__device__ __forceinline__ int active_scale_warps(int stages) {
  return stages >= kScaleWarps ? kScaleWarps : stages >= 2 ? 2 : 1;
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
// Whether factor(a, b) is one product for every lane's a and each lane's two b.
__device__ __forceinline__ bool one_product(float a, float b0, float b1) {
  uint32_t lo = 0x7F7FFFFFu, hi = 0;  // the least positive b and the largest finite one, as bits
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t bits = __float_as_uint(i == 0 ? b0 : b1);
    if (bits - 1u < 0x7F7FFFFFu) lo = min(lo, bits), hi = max(hi, bits);
  }
  lo = __reduce_min_sync(0xFFFFFFFFu, lo);
  hi = __reduce_max_sync(0xFFFFFFFFu, hi);
  return __all_sync(0xFFFFFFFFu, !(a > 0.0f && __fmul_rn(a, __uint_as_float(lo)) < 0x1p-126f) &&
                                     !(a <= 0x1.fffffep127f && __fmul_rn(a, __uint_as_float(hi)) > 0x1.fffffep127f));
}
// amax / 2688 of a row (1 of an MXFP4 operand).
__device__ __forceinline__ float row_factor(const Fp4Side& s, int64_t row) {
  if (s.amax == nullptr) return 1.0f;
  return __fdiv_rn(s.amax[s.amax_per_row ? (row < s.rows ? row : s.rows - 1) : 0], 2688.0f);
}

// fp4_matmul_thin.cu: at most kThinRows rows of A
constexpr int kThinRows = 64;
struct ThinPlan {
  int bn, split;
  int64_t tiles;
};
ThinPlan thin_plan(const Fp4MatmulArgs& a, const LaunchCtx& ctx);
cudaError_t launch_matmul_thin(const Fp4MatmulArgs& a, MatmulKernelArgs p, const LaunchCtx& ctx);

}  // namespace fp4
}  // namespace nvfp4
