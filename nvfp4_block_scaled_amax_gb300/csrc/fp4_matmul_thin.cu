// fp4_matmul_thin.cu -- the product of fp4_matmul.cu for few rows of A (a
// decoding step, a small matrix).
//
// The operands change places: a CTA's tile is 128 rows of B (the weights, on
// the tensor-memory lanes) by kBN = 16, 32 or 64 rows of A (the columns),
// so that few rows waste little of an MMA and every weight is read once per kBN
// rows.  The contracted dimension of a tile is split over a cluster of 2, 4
// or 8 CTAs where there are too few tiles to fill the machine: each CTA sums its
// share of the stages, sends every column of its partial sums to the CTA of
// the cluster that owns the column (through distributed shared memory, counted
// on the owner's barrier), and the owner adds the shares in the order of
// their rank, so the result does not depend on timing.
//
// One row through 5120 x 4096 (NVFP4, swizzled weights) takes 5.2 us in a graph, of which
// the weights' bytes are 1.8: the start of the launch, the first copies' latency,
// the cluster's join and the end are one after the other.  Eight rows through
// 10240 x 8192 take 10.6 us, 4.5 TB/s.
//
// Warps 0-3 write the results, warp 4 issues the copies, warp 5 the MMAs (two
// accumulators, so that a tile is multiplied while the one before it is
// written), warps 6-9 put compact scales in order, a stage each in turn: A's, which
// so few rows always are, and B's if they are not swizzled.
#include "fp4_tiles.cuh"

namespace nvfp4 {
namespace fp4 {
namespace {

constexpr int kOutWarps = 4;
constexpr int kThreads = 32 * (kOutWarps + 2 + kScaleWarps);
constexpr int kWeights = 128;  // rows of B in a tile
constexpr int kMaxStages = 8;

struct Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2];
  uint64_t got, taken;  // the cluster's partial sums: all are here / all have been added
  uint32_t tmem;
  uint32_t pad;
};

template <int kBN, int kBlock>
struct Layout {
  using F = Format<kBlock>;
  static constexpr int kCodes = (kWeights + kBN) * kStageRow;
  static constexpr int kStageBytes = kCodes + 2 * F::kScaleBytes;  // a multiple of 1024
  static constexpr int kCols = 2 * kBN + 2 * F::kCols;
  static constexpr int kTmemCols = kCols <= 64 ? 64 : kCols <= 128 ? 128 : 256;
  static_assert(kCols <= 256, "two CTAs share an SM's tensor memory");
  // Columns a CTA of a cluster owns (of few columns and many CTAs, the last CTAs own none).
  static __host__ __device__ int own(int split) { return split == 1 ? 0 : kBN / split < 4 ? 4 : kBN / split; }
  static __host__ __device__ int share_floats(int split) { return split * own(split) * kWeights; }
  static int rest(int split) { return 4 * share_floats(split) + (int)sizeof(Barriers); }
};

template <int kBN, int kBlock>
__global__ void __launch_bounds__(kThreads, 2)
matmul_thin_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                   const __grid_constant__ MatmulKernelArgs p, int stages, int split) {
  using L = Layout<kBN, kBlock>;
  using F = Format<kBlock>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* shares = reinterpret_cast<float*>(smem + stages * L::kStageBytes);  // [rank of the sender][own columns / 4][row of B][4]
  const int own = L::own(split);
  Barriers* bar = reinterpret_cast<Barriers*>(shares + L::share_floats(split));
  const int w = warp_index(), lane = threadIdx.x & 31;
  const int rank = split > 1 ? (int)cluster_rank() : 0;

  if (w == kOutWarps) {
    if (lane == 0) {
      for (int i = 0; i < stages; ++i) {
        mbar_init(&bar->full[i], 2);  // the copies, and compact scales
        mbar_init(&bar->empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar->tfull[i], 1);
        mbar_init(&bar->tempty[i], kOutWarps);
      }
      mbar_init(&bar->got, 1);
      mbar_init(&bar->taken, kOutWarps * split);
      fence_mbar_init();
      tma_prefetch_desc(&amap);
      tma_prefetch_desc(&bmap);
    }
  } else if (w == kOutWarps + 1) {
    tmem_alloc(&bar->tmem, L::kTmemCols);
  }
  __syncwarp();
  if (split > 1) cluster_arrive();  // (the barriers are set up)
  grid_begin();
  tcgen05_before_sync();
  __syncthreads();
  if (split > 1) cluster_wait();
  tcgen05_after_sync();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, bar->tmem, 0);
  const int lg_split = __ffs(split) - 1;
  const int t0 = blockIdx.x >> lg_split, step = gridDim.x >> lg_split, tiles = p.tiles_a * p.tiles_b;
  const int nkb = (int)((p.K + kStageK - 1) / kStageK);
  const int full_stages = (int)(p.K / kStageK), last_steps = (int)((p.K % kStageK + 63) / 64);  // of 64 elements
  const int kb0 = (int)(((int64_t)nkb * rank) >> lg_split), kb1 = (int)(((int64_t)nkb * (rank + 1)) >> lg_split);
  bool ok = true;

  if (w == kOutWarps) {
    uint32_t s = 0, phase = 1, sent = 0;
    for (int t = t0; t < tiles && ok; t += step) {
      const int64_t n0 = (int64_t)(t / p.tiles_a) * kWeights, m0 = (int64_t)(t % p.tiles_a) * kBN;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&bar->empty[s], phase)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const int64_t k0 = (int64_t)kb * kStageK;
          const uint32_t scales = swizzled_bytes<kBlock>(p.K, k0);
          const uint32_t dst = smem_u32(smem + s * L::kStageBytes), full = smem_u32(&bar->full[s]);
          mbar_arrive_expect_tx(&bar->full[s], L::kCodes + (p.b.swizzled ? scales : 0));
          tma_load(dst, &bmap, kb * kStageRow, (int32_t)n0, full);
          tma_load(dst + kWeights * kStageRow, &amap, kb * kStageRow, (int32_t)m0, full);
          if (p.b.swizzled) bulk_load(dst + L::kCodes, swizzled_at<kBlock>(p.b, p.K, n0, k0), scales, &bar->full[s]);
        }
        __syncwarp();
        ++sent;
        if (++s == (uint32_t)stages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) {
      report_timeout(p.status);
      // let the copies in flight land
      for (uint32_t i = sent < (uint32_t)stages ? 0 : sent - stages; i < sent; ++i)
        mbar_wait(&bar->full[i % stages], (i / stages) & 1);
    }
  } else if (w == kOutWarps + 1) {
    constexpr uint32_t kIdesc = F::idesc(kWeights, kBN);
    const uint64_t desc0 = operand_desc(smem_u32(smem));
    const uint64_t sdesc0 = scale_desc(smem_u32(smem) + L::kCodes);
    const uint32_t sb = tmem + 2 * kBN, sa = sb + F::kCols;
    uint32_t s = 0, phase = 0, buf = 0, tphase = 1;
    for (int t = t0; t < tiles && ok; t += step) {
      if (!mbar_wait(&bar->tempty[buf], tphase)) {
        ok = false;
        break;
      }
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&bar->full[s], phase)) {
          ok = false;
          break;
        }
        tcgen05_after_sync();
        const uint64_t b = desc0 + s * (L::kStageBytes / 16), a = b + kWeights * kStageRow / 16;
        const uint64_t ds = sdesc0 + s * (L::kStageBytes / 16);
        const uint32_t add = kb > kb0;
        auto copy = [&](int j) {
          scales_to_tmem<1>(sb + 4 * j, ds + j * (kScaleTile / 16));
          scales_to_tmem<1>(sa + 4 * j, ds + (F::kScaleBytes + j * kScaleTile) / 16);
        };
        auto multiply = [&](int k) {
          umma_fp4<1, kBlock>(tmem + buf * kBN, b + 2 * k, a + 2 * k, kIdesc | F::half(k), sb + F::col(k),
                              sa + F::col(k), k > 0 ? 1 : add);
        };
        if (elect_one()) {
          if (kb < full_stages) {
#pragma unroll
            for (int j = 0; j < F::kTiles; ++j) copy(j);
#pragma unroll
            for (int k = 0; k < 4; ++k) multiply(k);
          } else {
            for (int j = 0; j * 4 * kBlock < last_steps * 64; ++j) copy(j);
            for (int k = 0; k < last_steps; ++k) multiply(k);
          }
          umma_commit(&bar->empty[s]);
          if (kb + 1 == kb1) umma_commit(&bar->tfull[buf]);
        }
        __syncwarp();
        if (++s == (uint32_t)stages) {
          s = 0;
          phase ^= 1;
        }
      }
      buf ^= 1;
      tphase ^= buf ^ 1;
    }
    if (!ok) report_timeout(p.status);
  } else if (w > kOutWarps + 1) {
    const int mine = w - kOutWarps - 2, active = active_scale_warps(stages);
    if (mine < active) {
      uint32_t s = 0, phase = 1, it = 0;
      const CompactScales<kBlock> of_a(p.a.scale, p.K, p.a.rows), of_b(p.b.scale, p.K, p.b.rows);
      for (int t = t0; t < tiles && ok; t += step) {
        const int64_t n0 = (int64_t)(t / p.tiles_a) * kWeights, m0 = (int64_t)(t % p.tiles_a) * kBN;
        for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
          if ((it & (active - 1)) == (uint32_t)mine) {
            uint32_t va[4][F::kTiles], vb[4][F::kTiles];
            if (!p.b.swizzled) of_b.read(n0, kWeights, kb, vb);
            of_a.read(m0, kBN, kb, va);
            ok = mbar_wait(&bar->empty[s], phase);
            if (ok) {
              const uint32_t dst = smem_u32(smem + s * L::kStageBytes) + L::kCodes;
              if (!p.b.swizzled) of_b.write(dst, vb);
              of_a.write(dst + F::kScaleBytes, va);
              fence_proxy_async_shared();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar->full[s]);
            }
          }
          if (++s == (uint32_t)stages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) report_timeout(p.status);
    }
  } else {
    const uint32_t lane_base = tmem + ((uint32_t)(32 * w) << 16);
    const int n_in_tile = 32 * w + lane;
    uint32_t buf = 0, tphase = 0, round = 0;
    for (int t = t0; t < tiles && ok; t += step) {
      const int64_t n0 = (int64_t)(t / p.tiles_a) * kWeights, m0 = (int64_t)(t % p.tiles_a) * kBN;
      const int rows = (int)min((int64_t)kBN, p.a.rows - m0);
      const bool there = n0 + n_in_tile < p.b.rows;
      const float fb = row_factor(p.b, n0 + n_in_tile);
      const Factor whole = factor(p.a.amax_per_row ? 1.0f : row_factor(p.a, 0), fb);
      // with an amax for each row of A: lane l has those of columns l and 32 + l
      float fa[2] = {};
      if (p.a.amax_per_row)
#pragma unroll
        for (int k = 0; k < (kBN + 31) / 32; ++k) fa[k] = row_factor(p.a, m0 + 32 * k + lane);
      auto store = [&](int c, float v) {  // (by whole warps)
        const float mine = __shfl_sync(0xFFFFFFFFu, c < 32 ? fa[0] : fa[1], c & 31);
        if (c >= rows || !there) return;
        v = p.a.amax_per_row ? factor(mine, fb)(v) : whole(v);
        const int64_t at = (m0 + c) * p.b.rows + n0 + n_in_tile;
        if (p.out_bf16) {
          uint16_t h;
          asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
          static_cast<uint16_t*>(p.out)[at] = h;
        } else {
          static_cast<float*>(p.out)[at] = v;
        }
      };
      ok = mbar_wait(&bar->tfull[buf], tphase);
      if (!ok) break;
      __syncwarp();
      tcgen05_after_sync();
      constexpr int kChunk = kBN < 32 ? kBN : 32;
      auto release = [&]() {
        tcgen05_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->tempty[buf]);
      };
      if (split == 1) {
#pragma unroll 1
        for (int c = 0; c < kBN && c < rows; c += kChunk) {
          uint32_t v[kChunk];
          tmem_read(lane_base + buf * kBN + c, v);
#pragma unroll
          for (int i = 0; i < kChunk; ++i) store(c + i, __uint_as_float(v[i]));
        }
        release();
      } else {
        // Column c belongs to rank c / own.  Columns travel in fours.
        const int lg = __ffs(own) - 1;
        ok = mbar_wait_cluster(&bar->taken, (round & 1) ^ 1, p.status);
        if (!ok) break;
        const int held = max(0, min(own, rows - rank * own));  // columns of this CTA that exist
        if (w == 0 && lane == 0) mbar_arrive_expect_tx(&bar->got, split * kWeights * 4 * ((held + 3) & ~3));
        const uint32_t mine = smem_u32(shares) + 4 * (rank * own * kWeights + 4 * n_in_tile), got = smem_u32(&bar->got);
#pragma unroll 1
        for (int c = 0; c < kBN && c < rows; c += kChunk) {
          uint32_t v[kChunk];
          tmem_read(lane_base + buf * kBN + c, v);
#pragma unroll
          for (int i = 0; i < kChunk; i += 4) {
            const int col = c + i;
            if (col >= rows) break;
            store_async(map_to_cta(mine + 4 * (col & (own - 1)) * kWeights, col >> lg), __uint_as_float(v[i]),
                        __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]),
                        map_to_cta(got, col >> lg));
          }
        }
        release();
        ok = mbar_wait_cluster(&bar->got, round & 1, p.status);
        if (!ok) break;
#pragma unroll 1
        for (int c = 0; c < held; c += 4) {
          float4 part[8];  // all read before the first is added
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r < split) part[r] = *reinterpret_cast<const float4*>(shares + (r * own + c) * kWeights + 4 * n_in_tile);
          float4 sum = part[0];
#pragma unroll
          for (int r = 1; r < 8; ++r)
            if (r < split)
              sum = make_float4(__fadd_rn(sum.x, part[r].x), __fadd_rn(sum.y, part[r].y), __fadd_rn(sum.z, part[r].z),
                                __fadd_rn(sum.w, part[r].w));
          const int at = rank * own + c;
          store(at, sum.x);
          store(at + 1, sum.y);
          store(at + 2, sum.z);
          store(at + 3, sum.w);
        }
        if (t + step < tiles) {
          __syncwarp();
          if (lane < split) mbar_arrive_cluster_release(map_to_cta(smem_u32(&bar->taken), lane));
        }
        ++round;
      }
      buf ^= 1;
      tphase ^= buf ^ 1;
    }
    if (!ok) report_timeout(p.status);
  }
  __syncwarp();
  tcgen05_before_sync();
  __syncthreads();
  // No CTA leaves before the others are done with its barriers.  What they
  // send it has arrived by then, as it waited for it; a CTA that gave up waiting
  // stays until stores in flight have landed.
  if (split > 1) {
    cluster_arrive_relaxed();
    cluster_wait();
    if (!ok) {
      const long long c0 = clock64();
      while (clock64() - c0 < 1000000LL) {
      }
    }
  }
  tcgen05_after_sync();
  if (w == kOutWarps + 1) tmem_dealloc(tmem, L::kTmemCols);
}

template <int kBN, int kBlock>
cudaError_t launch(const Fp4MatmulArgs& a, MatmulKernelArgs p, const ThinPlan& t, const LaunchCtx& ctx) {
  using L = Layout<kBN, kBlock>;
  CUtensorMap amap, bmap;
  cudaError_t e = make_fp8_tensor_map(&amap, a.a.data, a.a.rows, a.K / 2, kBN);
  if (e != cudaSuccess) return e;
  e = make_fp8_tensor_map(&bmap, a.b.data, a.b.rows, a.K / 2, kWeights);
  if (e != cudaSuccess) return e;
  constexpr int kPerCta = 113 * 1024;  // two CTAs share an SM's 228 KB, 1 KB of it reserved for each
  const int rest = 1024 + L::rest(t.split);
  int stages = (kPerCta - rest) / L::kStageBytes;
  if (stages > kMaxStages) stages = kMaxStages;
  const int smem = rest + stages * L::kStageBytes;
  const auto kernel = matmul_thin_kernel<kBN, kBlock>;
  static std::atomic<uint64_t> allowed{0};
  e = allow_smem(reinterpret_cast<const void*>(kernel), kPerCta, allowed);
  if (e != cudaSuccess) return e;
  p.tiles_a = (int)((a.a.rows + kBN - 1) / kBN);
  p.tiles_b = (int)((a.b.rows + kWeights - 1) / kWeights);
  const int64_t room = 2 * ctx.num_sms / t.split;
  int split = t.split;
  void* args[] = {&amap, &bmap, &p, &stages, &split};
  return launch_dependent(reinterpret_cast<const void*>(kernel),
                          dim3((unsigned)((t.tiles < room ? t.tiles : room) * split)), dim3(kThreads), smem, ctx.stream,
                          args, split);
}

template <int kBlock>
cudaError_t launch_columns(const Fp4MatmulArgs& a, const MatmulKernelArgs& p, const ThinPlan& t, const LaunchCtx& ctx) {
  if (t.bn == 16) return launch<16, kBlock>(a, p, t, ctx);
  if (t.bn == 32) return launch<32, kBlock>(a, p, t, ctx);
  return launch<64, kBlock>(a, p, t, ctx);
}

}  // namespace

ThinPlan thin_plan(const Fp4MatmulArgs& a, const LaunchCtx& ctx) {
  ThinPlan t;
  t.bn = a.a.rows <= 16 ? 16 : a.a.rows <= 32 ? 32 : 64;
  t.tiles = (a.a.rows + t.bn - 1) / t.bn * ((a.b.rows + kWeights - 1) / kWeights);
  // (8 rows, N 2048, K 8192: 5.2 us by eight CTAs a tile, 5.4 by up to four, 7.6 two, 9.8 one; 1 row, 5120 x 4096:
  // 5.2 by four, 5.3 two, 6.6 one; 64 rows, N 1024, K 8192: 7.4 by eight, 11.0 by fewer.)
  const int64_t stages = (a.K + kStageK - 1) / kStageK;
  t.split = 1;
  for (int s = 8; s >= 2 && t.split == 1; s /= 2)
    if (t.tiles * s <= 2 * ctx.num_sms && stages >= 2 * s) t.split = s;
  return t;
}

cudaError_t launch_matmul_thin(const Fp4MatmulArgs& a, MatmulKernelArgs p, const LaunchCtx& ctx) {
  const ThinPlan t = thin_plan(a, ctx);
  return a.block == 16 ? launch_columns<16>(a, p, t, ctx) : launch_columns<32>(a, p, t, ctx);
}

}  // namespace fp4
}  // namespace nvfp4
