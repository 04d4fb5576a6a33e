// fp8_cast.cu -- the cast to E4M3 with one FP32 scale for each block of 128,
// rows and transposed columns in one pass.
//
// For a block (128 consecutive elements of a row, or a 128 x 128 tile) with
// a = max(max|x|, 2^-100):  s = a / 448,  r = 448 / a  (IEEE FP32 divisions)
// and q = E4M3_rn_satfinite(x * r).  The floor keeps s and r normal numbers
// for a block of zeros or of tiny values.  The column-wise output is the
// same cast of x transposed.
//
// A 128 x 128 tile holds whole blocks of both directions, so one CTA casts it
// from registers with one read of x: TMA brings the tile, a thread takes 8
// rows x 8 columns (the next tile's copy starts at once), maxima meet over
// the 16 lanes of a row and, through shared memory, over the 16 row groups
// of a column, and both directions' codes leave through shared memory by TMA,
// which also cuts off what lies past the edges.  Memory-bound: 2 or 4 bytes
// in and 1 byte per direction out for every element.
#include "common.cuh"
#include "dependent.h"
#include "fp8.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;
constexpr int kCodeBytes = kTile * kTile;
constexpr float kFloor = 7.888609052210118e-31f;  // 2^-100

struct CastKernelArgs {
  int64_t M, N;
  int tiles_m, tiles_n;
  int64_t tiles;
  float* scale_row;
  float* scale_col;
  unsigned* status;
};

template <bool kBf16>
struct Smem {
  static constexpr int kInBytes = kTile * kTile * (kBf16 ? 2 : 4);
  static constexpr int kBytes = 1024 + kInBytes + 2 * kCodeBytes;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(src)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
// Per BF16 half, the larger magnitude (its sign is of no use): one instruction
// where masking the signs away takes two more on the same pipe.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two FP32 values -> two E4M3 codes, v0 in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float v0, float v1) {
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(v1), "f"(v0));
  return h;
}

// kBoth: row-wise and column-wise codes; otherwise one direction (kRow).
template <bool kBf16, bool kRow, bool kCol, bool kTileScale>
__global__ void __launch_bounds__(kThreads, kBf16 ? 3 : 2)
fp8_cast_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap rmap,
                const __grid_constant__ CUtensorMap cmap, const __grid_constant__ CastKernelArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full;
  __shared__ __align__(16) float row_max[kTile], col_max[kThreads / 32][kTile], row_fac[kTile], col_fac[kTile];
  const uint32_t in = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t out_row = in + Smem<kBf16>::kInBytes, out_col = out_row + kCodeBytes;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int g = lane & 15;            // columns 8 g .. 8 g + 7
  const int rg = 2 * w + (lane >> 4);  // rows 8 rg .. 8 rg + 7
  if (tid == 0) {
    mbar_init(&full, 1);
    fence_mbar_init();
    tma_prefetch_desc(&xmap);
    if (kRow) tma_prefetch_desc(&rmap);
    if (kCol) tma_prefetch_desc(&cmap);
  }
  grid_begin();
  __syncthreads();
  constexpr int kBox = kBf16 ? 64 : 32;  // columns of an input box (128 bytes)
  auto load = [&](int64_t t) {
    const int64_t per = (int64_t)a.tiles_m * a.tiles_n, b = t / per, i = t - b * per;
    const int32_t m = (int32_t)(i / a.tiles_n) * kTile, n = (int32_t)(i % a.tiles_n) * kTile;
    mbar_arrive_expect_tx(&full, Smem<kBf16>::kInBytes);
#pragma unroll
    for (int k = 0; k < kTile / kBox; ++k) tma_load_3d(in + k * kTile * 128, &xmap, n + k * kBox, m, (int32_t)b, &full);
  };
  if (tid == 0 && blockIdx.x < a.tiles) load(blockIdx.x);
  uint32_t phase = 0;
  for (int64_t t = blockIdx.x; t < a.tiles; t += gridDim.x) {
    const bool ok = mbar_wait_bounded(&full, phase, a.status);
    phase ^= 1;
    // 8 x 8 elements: BF16 in four words a row, FP32 in eight
    constexpr int kW = kBf16 ? 4 : 8;
    uint32_t x[8][kW];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 8 * rg + i;  // r & 7 == i
      if constexpr (kBf16) {
        const uint4 v = lds128(in + (g >> 3) * (kTile * 128) + r * 128 + (((g & 7) ^ i) * 16));
        x[i][0] = v.x; x[i][1] = v.y; x[i][2] = v.z; x[i][3] = v.w;
      } else {
        // the two halves in either order, so that eight lanes touch eight different 16-byte places
        const uint32_t row = in + (g >> 2) * (kTile * 128) + r * 128;
        const int odd = (g >> 2) & 1;
        const uint4 p = lds128(row + (((2 * (g & 3) + odd) ^ i) * 16));
        const uint4 q = lds128(row + (((2 * (g & 3) + 1 - odd) ^ i) * 16));
        x[i][0] = odd ? q.x : p.x; x[i][1] = odd ? q.y : p.y; x[i][2] = odd ? q.z : p.z; x[i][3] = odd ? q.w : p.w;
        x[i][4] = odd ? p.x : q.x; x[i][5] = odd ? p.y : q.y; x[i][6] = odd ? p.z : q.z; x[i][7] = odd ? p.w : q.w;
      }
    }
    // everyone has its elements, and (below) the previous codes are stored
    if (tid == 0) bulk_wait_read_all();
    if (!__syncthreads_and(ok)) break;
    if (tid == 0 && t + gridDim.x < a.tiles) load(t + gridDim.x);
    const int64_t per = (int64_t)a.tiles_m * a.tiles_n, b = t / per, ti = t - b * per;
    const int tm = (int)(ti / a.tiles_n), tn = (int)(ti % a.tiles_n);
    const int64_t m0 = (int64_t)tm * kTile, n0 = (int64_t)tn * kTile;

    // Maxima of the thread's rows and columns, then over the 16 lanes of a row
    // and the two row groups of a warp.
    if constexpr (kBf16) {
      uint32_t rm[4], cm[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) cm[k] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (kRow || kTileScale) m = larger(m, x[i][k]);
          if (kCol && !kTileScale) cm[k] = larger(cm[k], x[i][k]);
        }
        // the larger half of rows i and i + 1 side by side in one word
        m = larger(m, __byte_perm(m, m, 0x1032));
        if (i & 1) rm[i >> 1] = __byte_perm(rm[i >> 1], m, 0x5410); else rm[i >> 1] = m;
      }
      if (kRow || kTileScale) {
#pragma unroll
        for (int d = 1; d < 16; d <<= 1)
#pragma unroll
          for (int k = 0; k < 4; ++k) rm[k] = larger(rm[k], __shfl_xor_sync(0xFFFFFFFFu, rm[k], d));
        if (g == 0) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<float2*>(&row_max[8 * rg + 2 * k]) = make_float2(fabsf(bf16_lo(rm[k])), fabsf(bf16_hi(rm[k])));
        }
      }
      if (kCol && !kTileScale) {
#pragma unroll
        for (int k = 0; k < 4; ++k) cm[k] = larger(cm[k], __shfl_xor_sync(0xFFFFFFFFu, cm[k], 16));
        if (lane < 16) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<float4*>(&col_max[w][8 * g + 4 * k]) =
                make_float4(fabsf(bf16_lo(cm[2 * k])), fabsf(bf16_hi(cm[2 * k])), fabsf(bf16_lo(cm[2 * k + 1])),
                            fabsf(bf16_hi(cm[2 * k + 1])));
        }
      }
    } else {
      float rm[8], cm[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) cm[k] = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        rm[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float v = fabsf(__uint_as_float(x[i][k]));
          if (kRow || kTileScale) rm[i] = fmaxf(rm[i], v);
          if (kCol && !kTileScale) cm[k] = fmaxf(cm[k], v);
        }
      }
      if (kRow || kTileScale) {
#pragma unroll
        for (int d = 1; d < 16; d <<= 1)
#pragma unroll
          for (int i = 0; i < 8; ++i) rm[i] = fmaxf(rm[i], __shfl_xor_sync(0xFFFFFFFFu, rm[i], d));
        if (g == 0) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<float4*>(&row_max[8 * rg + 4 * k]) =
                make_float4(rm[4 * k], rm[4 * k + 1], rm[4 * k + 2], rm[4 * k + 3]);
        }
      }
      if (kCol && !kTileScale) {
#pragma unroll
        for (int k = 0; k < 8; ++k) cm[k] = fmaxf(cm[k], __shfl_xor_sync(0xFFFFFFFFu, cm[k], 16));
        if (lane < 16) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<float4*>(&col_max[w][8 * g + 4 * k]) =
                make_float4(cm[4 * k], cm[4 * k + 1], cm[4 * k + 2], cm[4 * k + 3]);
        }
      }
    }
    __syncthreads();
    float rf[8], cf[8];  // encode factors of the thread's rows and columns
    if constexpr (kTileScale) {
      float m = fmaxf(fmaxf(row_max[lane], row_max[lane + 32]), fmaxf(row_max[lane + 64], row_max[lane + 96]));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
      m = fmaxf(m, kFloor);
      const float f = __fdiv_rn(448.0f, m);
      if (tid == 0) {
        const float s = __fdiv_rn(m, 448.0f);
        if (kRow) a.scale_row[(b * a.tiles_m + tm) * a.tiles_n + tn] = s;
        if (kCol) a.scale_col[(b * a.tiles_n + tn) * a.tiles_m + tm] = s;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) rf[i] = cf[i] = f;
    } else {
      if (tid < kTile) {
        if constexpr (kRow) {
          const float m = fmaxf(row_max[tid], kFloor);
          row_fac[tid] = __fdiv_rn(448.0f, m);
          if (m0 + tid < a.M) a.scale_row[(b * a.tiles_n + tn) * a.M + m0 + tid] = __fdiv_rn(m, 448.0f);
        }
      } else if constexpr (kCol) {
        const int c = tid - kTile;
        float m = kFloor;
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) m = fmaxf(m, col_max[k][c]);
        col_fac[c] = __fdiv_rn(448.0f, m);
        if (n0 + c < a.N) a.scale_col[(b * a.tiles_m + tm) * a.N + n0 + c] = __fdiv_rn(m, 448.0f);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (kRow) *reinterpret_cast<float4*>(&rf[4 * k]) = *reinterpret_cast<const float4*>(&row_fac[8 * rg + 4 * k]);
        if (kCol) *reinterpret_cast<float4*>(&cf[4 * k]) = *reinterpret_cast<const float4*>(&col_fac[8 * g + 4 * k]);
      }
    }
    auto value = [&](int i, int k) {  // element of row i, column k
      if constexpr (kBf16) return k & 1 ? bf16_hi(x[i][k >> 1]) : bf16_lo(x[i][k >> 1]);
      else return __uint_as_float(x[i][k]);
    };
    // Four rows at a time, unpacked once for both directions.
    uint32_t c[8][2];  // [column][rows 0-3, 4-7]
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = value(4 * h + i, k);
      if constexpr (kRow) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = rf[4 * h + i];
          uint32_t q[2];
#pragma unroll
          for (int k = 0; k < 2; ++k)
            q[k] = e4m3x2(__fmul_rn(v[i][4 * k], f), __fmul_rn(v[i][4 * k + 1], f)) |
                   e4m3x2(__fmul_rn(v[i][4 * k + 2], f), __fmul_rn(v[i][4 * k + 3], f)) << 16;
          sts_v2(out_row + (8 * rg + 4 * h + i) * 128 + (((g >> 1) ^ (4 * h + i)) * 16) + (g & 1) * 8, q[0], q[1]);
        }
      }
      if constexpr (kCol) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          c[k][h] = e4m3x2(__fmul_rn(v[0][k], cf[k]), __fmul_rn(v[1][k], cf[k])) |
                    e4m3x2(__fmul_rn(v[2][k], cf[k]), __fmul_rn(v[3][k], cf[k])) << 16;
      }
    }
    if constexpr (kCol) {
      // Lane g stores its column k ^ (g & 7) in turn k (three rounds of swaps
      // arrange them), so that a turn's stores fall into different banks.
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) {
        const bool swap = g & d;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (!(k & d)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t p = c[k][i], q = c[k | d][i];
              c[k][i] = swap ? q : p;
              c[k | d][i] = swap ? p : q;
            }
          }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int kk = k ^ (g & 7);  // column 8 g + kk, a row of the output
        sts_v2(out_col + (8 * g + kk) * 128 + (((rg >> 1) ^ kk) * 16) + (rg & 1) * 8, c[k][0], c[k][1]);
      }
    }
    fence_proxy_async_shared();
    __syncthreads();
    if (tid == 0) {
      if (kRow) tma_store_3d(&rmap, out_row, (int32_t)n0, (int32_t)m0, (int32_t)b);
      if (kCol) tma_store_3d(&cmap, out_col, (int32_t)m0, (int32_t)n0, (int32_t)b);
      bulk_commit();
    }
  }
  if (tid == 0) bulk_wait_all();
}

template <bool kBf16, bool kRow, bool kCol, bool kTileScale>
cudaError_t launch(const CUtensorMap& x, const CUtensorMap& r, const CUtensorMap& c, const CastKernelArgs& k,
                   const LaunchCtx& ctx) {
  const auto kernel = fp8_cast_kernel<kBf16, kRow, kCol, kTileScale>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), Smem<kBf16>::kBytes, allowed);
  if (e != cudaSuccess) return e;
  const int64_t room = (int64_t)ctx.num_sms * (kBf16 ? 3 : 2);
  CUtensorMap maps[3] = {x, r, c};
  CastKernelArgs args = k;
  void* p[] = {&maps[0], &maps[1], &maps[2], &args};
  return launch_dependent(reinterpret_cast<const void*>(kernel), dim3((unsigned)(k.tiles < room ? k.tiles : room)),
                    dim3(kThreads), Smem<kBf16>::kBytes, ctx.stream, p);
}

template <bool kBf16, bool kTileScale>
cudaError_t launch_directions(const CUtensorMap& x, const CUtensorMap& r, const CUtensorMap& c, bool row, bool col,
                              const CastKernelArgs& k, const LaunchCtx& ctx) {
  if (row && col) return launch<kBf16, true, true, kTileScale>(x, r, c, k, ctx);
  if (row) return launch<kBf16, true, false, kTileScale>(x, r, c, k, ctx);
  return launch<kBf16, false, true, kTileScale>(x, r, c, k, ctx);
}

}  // namespace

cudaError_t launch_fp8_cast(const void* x, const Fp8CastArgs& a, const LaunchCtx& ctx) {
  if (a.batch == 0 || a.M == 0 || a.N == 0) return cudaSuccess;
  CUtensorMap xm, rm = {}, cm = {};
  cudaError_t e = make_batch_tensor_map(&xm, x, a.bf16 ? 2 : 4, a.batch, a.M, a.N);
  if (e == cudaSuccess && a.data_row) e = make_batch_tensor_map(&rm, a.data_row, 1, a.batch, a.M, a.N);
  if (e == cudaSuccess && a.data_col) e = make_batch_tensor_map(&cm, a.data_col, 1, a.batch, a.N, a.M);
  if (e != cudaSuccess) return e;
  CastKernelArgs k = {};
  k.M = a.M;
  k.N = a.N;
  k.tiles_m = (int)fp8_blocks(a.M);
  k.tiles_n = (int)fp8_blocks(a.N);
  k.tiles = a.batch * k.tiles_m * k.tiles_n;
  k.scale_row = a.scale_row;
  k.scale_col = a.scale_col;
  k.status = ctx.status;
  const bool row = a.data_row != nullptr, col = a.data_col != nullptr;
  if (a.bf16)
    return a.block_rows == 1 ? launch_directions<true, false>(xm, rm, cm, row, col, k, ctx)
                             : launch_directions<true, true>(xm, rm, cm, row, col, k, ctx);
  return a.block_rows == 1 ? launch_directions<false, false>(xm, rm, cm, row, col, k, ctx)
                           : launch_directions<false, true>(xm, rm, cm, row, col, k, ctx);
}

}  // namespace nvfp4
