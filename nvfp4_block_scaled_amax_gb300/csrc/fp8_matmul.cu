// fp8_matmul.cu -- the product of E4M3 operands with a scale for each block of
// 128 along the contracted dimension:
//     c[m][n] = sum_b sa[b][m] sb[b][n] sum_{k in b} a[m][k] b[n][k].
// The inner sum of a block runs on the tensor cores (tcgen05 kind::f8f6f4,
// FP32 accumulation in tensor memory); the outer sum is held in FP32
// registers, one fused multiply-add per block and element.
//
// With member offsets, A's rows are cut into members, member e = rows
// offsets[e] .. offsets[e + 1], each multiplied by its own B; rows past the
// last member are zero.  In the weight-gradient form the members cut the
// contracted dimension instead (in blocks of 128) and each gives a product
// of its own; an empty member's product is zero.
//
// Warp-specialised persistent kernel, one CTA per SM: warp 8 streams 128-byte
// slices of both operands through a TMA ring, warp 9 issues the MMAs of each
// block into one of two tensor-memory accumulators, and warps 0-7 read the
// finished accumulator and add it, scaled, to their registers while the next
// block is multiplied.
#include <cudaTypedefs.h>

#include "common.cuh"
#include "fp8.h"
#include "tokens.h"

namespace nvfp4 {
namespace {

constexpr int kBM = 128, kBN = 128, kBK = 128;
constexpr int kStages = 6;
constexpr int kStageA = kBM * kBK, kStageB = kBN * kBK, kStageBytes = kStageA + kStageB;
constexpr int kSumWarps = 8;
constexpr int kThreads = 32 * (kSumWarps + 2);
constexpr int kColsPerThread = kBN / 2;

struct KernelArgs {
  const float* sa;
  const float* sb;
  int64_t a_rows, a_cols, b_rows;
  int b_block_rows, experts, wgrad;
  const int32_t* offsets;
  void* out;
  int out_bf16;
  unsigned* status;
};

struct Barriers {
  uint64_t full[kStages], empty[kStages], tfull[2], tempty[2];
  uint32_t tmem;
};

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Instruction descriptor of kind::f8f6f4: E4M3 A and B, both K-major, FP32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
               " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
               "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
               : "memory");
}

// Tiles of all members in one list: first[i] is the first tile of member i
// (forward: one more member, the rows past the last one, with nothing to sum).
struct TileList {
  int* first;  // shared, [members + 1]
  int members;
  int64_t tiles_n;
};

struct Tile {
  int64_t a_row, b_row, n0, out_row;
  int rows, cols;  // of the tile, inside the output
  int kb0, nkb;    // blocks of the contracted dimension
  int member;
};

__device__ __forceinline__ int64_t clamp_offset(const KernelArgs& p, int e) {
  const int64_t limit = p.wgrad ? p.a_cols : p.a_rows;
  const int64_t v = p.offsets[e];
  return v < 0 ? 0 : v > limit ? limit : v;
}
__device__ __forceinline__ void member_range(const KernelArgs& p, int e, int64_t& begin, int64_t& end) {
  const int64_t limit = p.wgrad ? p.a_cols : p.a_rows;
  if (p.offsets == nullptr) {
    begin = 0;
    end = limit;
  } else if (e == p.experts) {  // the rows past the last member
    begin = clamp_offset(p, e);
    end = limit;
  } else {
    begin = clamp_offset(p, e);
    end = clamp_offset(p, e + 1);
    if (end < begin) end = begin;
  }
}

__device__ __forceinline__ Tile tile_at(const KernelArgs& p, const TileList& l, int t) {
  int lo = 0, hi = l.members;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (l.first[mid] <= t) lo = mid; else hi = mid;
  }
  Tile r;
  r.member = lo;
  const int i = t - l.first[lo];
  int64_t begin, end;
  member_range(p, lo, begin, end);
  const int64_t M = p.wgrad ? p.a_rows : end - begin;
  const int mt = (int)((M + kBM - 1) / kBM);
  const int64_t m0 = (int64_t)(i % mt) * kBM;
  r.n0 = (int64_t)(i / mt) * kBN;
  r.rows = (int)min((int64_t)kBM, M - m0);
  r.cols = (int)min((int64_t)kBN, p.b_rows - r.n0);
  if (p.wgrad) {
    r.a_row = m0;
    r.b_row = r.n0;
    r.out_row = lo * p.a_rows + m0;
    r.kb0 = (int)(begin / kBK);
    r.nkb = (int)((end + kBK - 1) / kBK) - r.kb0;
    if (begin == end) r.nkb = 0;
  } else {
    r.a_row = begin + m0;
    r.out_row = r.a_row;
    const bool tail = lo == p.experts;
    r.b_row = tail ? 0 : lo * p.b_rows + r.n0;
    r.kb0 = 0;
    r.nkb = tail ? 0 : (int)((p.a_cols + kBK - 1) / kBK);
  }
  return r;
}

__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__global__ void __launch_bounds__(kThreads, 1)
fp8_matmul_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                  const __grid_constant__ KernelArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Barriers* bar = reinterpret_cast<Barriers*>(smem + kStages * kStageBytes);
  TileList list;
  list.first = reinterpret_cast<int*>(bar + 1);
  list.members = p.offsets == nullptr ? 1 : p.experts + (p.wgrad ? 0 : 1);
  list.tiles_n = (p.b_rows + kBN - 1) / kBN;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (w == 0) {
    int run = 0;
    for (int e0 = 0; e0 < list.members; e0 += 32) {
      const int e = e0 + lane;
      int tiles = 0;
      if (e < list.members) {
        int64_t begin, end;
        member_range(p, e, begin, end);
        const int64_t M = p.wgrad ? p.a_rows : end - begin;
        tiles = (int)((M + kBM - 1) / kBM * list.tiles_n);
      }
      int incl = tiles;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += v;
      }
      if (e < list.members) list.first[e] = run + incl - tiles;
      run += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (lane == 0) list.first[list.members] = run;
  } else if (w == kSumWarps) {
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) {
        mbar_init(&bar->full[i], 1);
        mbar_init(&bar->empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar->tfull[i], 1);
        mbar_init(&bar->tempty[i], kSumWarps);
      }
      fence_mbar_init();
      tma_prefetch_desc(&amap);
      tma_prefetch_desc(&bmap);
    }
  } else if (w == kSumWarps + 1) {
    tmem_alloc(&bar->tmem, 2 * kBN);
  }
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  const uint32_t tmem = bar->tmem;
  const int tiles = list.first[list.members];

  if (w == kSumWarps) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const Tile tl = tile_at(p, list, t);
        for (int kb = 0; kb < tl.nkb; ++kb, ++it) {
          const uint32_t s = it % kStages;
          if (!mbar_wait_bounded(&bar->empty[s], ((it / kStages) & 1) ^ 1, p.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bar->full[s], kStageBytes);
          const uint32_t dst = smem_u32(smem + s * kStageBytes);
          tma_load(dst, &amap, (tl.kb0 + kb) * kBK, (int32_t)tl.a_row, &bar->full[s]);
          tma_load(dst + kStageA, &bmap, (tl.kb0 + kb) * kBK, (int32_t)tl.b_row, &bar->full[s]);
        }
      }
      if (!ok)  // let the copies in flight land before the CTA leaves
        for (uint32_t i = it < kStages ? 0 : it - kStages; i < it; ++i)
          mbar_wait_bounded(&bar->full[i % kStages], (i / kStages) & 1, p.status);
    }
    __syncwarp();
  } else if (w == kSumWarps + 1) {
    if (lane == 0) {
      constexpr uint32_t kIdesc = idesc_e4m3(kBM, kBN);
      uint32_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const int nkb = tile_at(p, list, t).nkb;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const uint32_t s = it % kStages, buf = it & 1;
          if (!mbar_wait_bounded(&bar->tempty[buf], ((it >> 1) & 1) ^ 1, p.status) ||
              !mbar_wait_bounded(&bar->full[s], (it / kStages) & 1, p.status)) {
            ok = false;
            break;
          }
          tcgen05_after_sync();
          const uint32_t a = smem_u32(smem + s * kStageBytes), b = a + kStageA;
#pragma unroll
          for (int k = 0; k < kBK / 32; ++k)  // 32 bytes further inside the 128-byte swizzled rows
            umma_e4m3(tmem + buf * kBN, umma_smem_desc(a + 32 * k, 16, 1024, 2), umma_smem_desc(b + 32 * k, 16, 1024, 2),
                      kIdesc, k > 0);
          umma_commit(&bar->empty[s]);
          umma_commit(&bar->tfull[buf]);
        }
      }
    }
    __syncwarp();
  } else {
    const int q = w & 3, half = w >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16) + half * kColsPerThread;
    const int64_t kblocks = (p.a_cols + kBK - 1) / kBK, nblocks = (p.b_rows + kBN - 1) / kBN;
    uint32_t it = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const Tile tl = tile_at(p, list, t);
      float acc[kColsPerThread];
#pragma unroll
      for (int i = 0; i < kColsPerThread; ++i) acc[i] = 0.0f;
      const int row = 32 * q + lane;
      const int64_t arow = min(tl.a_row + row, p.a_rows - 1);
      const int64_t c0 = tl.n0 + half * kColsPerThread;
      const int64_t member = p.wgrad || tl.nkb == 0 ? 0 : tl.member;
      for (int kb = 0; kb < tl.nkb; ++kb, ++it) {
        const uint32_t buf = it & 1;
        const float sa = p.sa[(tl.kb0 + kb) * p.a_rows + arow];
        if (!mbar_wait_bounded(&bar->tfull[buf], (it >> 1) & 1, p.status)) {
          ok = false;
          break;
        }
        __syncwarp();
        tcgen05_after_sync();
        uint32_t v[kColsPerThread / 32][32];
#pragma unroll
        for (int c = 0; c < kColsPerThread / 32; ++c) tmem_ld32_nowait(lane_base + buf * kBN + 32 * c, v[c]);
        tmem_ld_wait();
        tcgen05_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->tempty[buf]);
        if (p.b_block_rows == 128) {
          const float s = __fmul_rn(sa, p.sb[(member * nblocks + tl.n0 / kBN) * kblocks + tl.kb0 + kb]);
#pragma unroll
          for (int c = 0; c < kColsPerThread / 32; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[32 * c + i] = __fmaf_rn(__uint_as_float(v[c][i]), s, acc[32 * c + i]);
        } else {
          const float* sb = p.sb + (member * kblocks + tl.kb0 + kb) * p.b_rows;
#pragma unroll
          for (int c = 0; c < kColsPerThread / 32; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int64_t n = min(c0 + 32 * c + i, p.b_rows - 1);
              acc[32 * c + i] =
                  __fmaf_rn(__fmul_rn(__uint_as_float(v[c][i]), __ldg(sb + n)), sa, acc[32 * c + i]);
            }
        }
      }
      if (!ok || row >= tl.rows) continue;
      const int64_t at = (tl.out_row + row) * p.b_rows + c0;
#pragma unroll
      for (int i = 0; i < kColsPerThread; ++i) {
        if (c0 + i >= p.b_rows) continue;
        if (p.out_bf16) {
          uint16_t h;
          asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(acc[i]));
          static_cast<uint16_t*>(p.out)[at + i] = h;
        } else {
          static_cast<float*>(p.out)[at + i] = acc[i];
        }
      }
    }
  }
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  if (w == kSumWarps + 1) tmem_dealloc(tmem, 2 * kBN);
}

}  // namespace

cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, const LaunchCtx& ctx) {
  if (a.a_rows == 0 || a.b_rows == 0) return cudaSuccess;
  const int64_t out_rows = a.wgrad ? a.a_rows * a.experts : a.a_rows;
  if (a.a_cols == 0)
    return cudaMemsetAsync(a.out, 0, (size_t)out_rows * a.b_rows * (a.out_bf16 ? 2 : 4), ctx.stream);
  CUtensorMap amap, bmap;
  cudaError_t e = make_fp8_tensor_map(&amap, a.a, a.a_rows, a.a_cols, kBM);
  if (e != cudaSuccess) return e;
  e = make_fp8_tensor_map(&bmap, a.b, a.wgrad ? a.b_rows : a.b_rows * a.experts, a.a_cols, kBN);
  if (e != cudaSuccess) return e;
  KernelArgs p = {};
  p.sa = a.sa;
  p.sb = a.sb;
  p.a_rows = a.a_rows;
  p.a_cols = a.a_cols;
  p.b_rows = a.b_rows;
  p.b_block_rows = a.b_block_rows;
  p.experts = a.experts;
  p.wgrad = a.wgrad;
  p.offsets = a.offsets;
  p.out = a.out;
  p.out_bf16 = a.out_bf16;
  p.status = ctx.status;
  // No more tiles than this, whatever the offsets.
  const int64_t tn = (a.b_rows + kBN - 1) / kBN;
  const int64_t tm = (a.a_rows + kBM - 1) / kBM;
  const int64_t tiles = tn * (a.wgrad ? tm * a.experts : tm + (a.offsets ? a.experts : 0));
  const unsigned grid = (unsigned)(tiles < ctx.num_sms ? tiles : ctx.num_sms);
  const int smem = 1024 + kStages * kStageBytes + (int)sizeof(Barriers) + 4 * (kMaxExperts + 2);
  e = cudaFuncSetAttribute(fp8_matmul_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  fp8_matmul_kernel<<<grid, kThreads, smem, ctx.stream>>>(amap, bmap, p);
  return cudaGetLastError();
}

}  // namespace nvfp4
