// fp8_matmul_thin.cu -- the product of fp8_matmul.cu for few rows of A (a
// decoding step, a handful of rows per expert, a small matrix).
//
// The operands change places: a CTA's tile is 128 rows of B (the weights, on
// the tensor-memory lanes) by kBN = 16, 32 or 64 rows of A (the columns), so
// that few rows waste little of an MMA and every weight is read once per kBN
// rows.  The contracted dimension of a tile is split over a cluster of 1, 2,
// 4 or 8 CTAs where there are too few tiles to fill the machine: each CTA
// sums its share of the blocks, sends every column of its partial sums to
// the CTA of the cluster that owns the column (through distributed shared
// memory, counted on the owner's barrier), and the owner adds the shares in
// the order of their rank, so the result does not depend on timing.
//
// Bound by reading the weights: two CTAs per SM keep up to 200 KB of operand
// slices per SM in flight.  Warps 0-3 sum, warp 4 issues the copies, warp 5
// the MMAs (kBuffers accumulators, so the hand-overs overlap), warp 6 the
// scales.  64 rows to 16 experts of 4096 x 2048 weights: 22.6 us, 5.6 TB/s (82
// percent of the copy rate); one row through 5120 x 4096: 6.9 us.  (Kernel times
// here and below are of calls in a CUDA graph, on inputs that take turns and
// are larger than L2 together where the weights are.)
#include "fp8_tiles.cuh"

namespace nvfp4 {
namespace fp8 {
namespace {

constexpr int kSumWarps = 4;
constexpr int kThreads = 32 * (kSumWarps + 3);
constexpr int kWeights = 128;  // rows of B in a tile
constexpr int kStageW = kWeights * kBK;
constexpr int kScaleStages = 3, kScaleBatch = 4;  // blocks per scale stage
constexpr int kMaxStages = 8, kMaxBuffers = 8;

struct Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[kMaxBuffers], tempty[kMaxBuffers];
  uint64_t sfull[kScaleStages], sempty[kScaleStages];
  uint64_t got, taken;  // the cluster's partial sums: all are here / all have been added
  uint32_t tmem;
  uint32_t pad;
};

// Shared memory after the operand stages.
template <int kBN>
struct Layout {
  static constexpr int kStageBytes = kStageW + kBN * kBK;
  static constexpr int kBuffers = kBN == 64 ? 4 : 8;
  static constexpr int kTmemCols = kBN * kBuffers;
  static constexpr int kScaleFloats = kWeights + kBN;
  static constexpr int kScaleBytes = kScaleStages * kScaleBatch * kScaleFloats * 4;
  // Columns a CTA of a cluster owns (of few columns and many CTAs, the last CTAs own none).
  static __host__ __device__ int own(int split) { return split == 1 ? 0 : kBN / split < 4 ? 4 : kBN / split; }
  static __host__ __device__ int share_floats(int split) { return split * own(split) * kWeights; }
  static int rest(int experts, int split) {
    return kScaleBytes + 4 * share_floats(split) + (int)sizeof(Barriers) +
           4 * TileList<kBN, kWeights, 0>::ints(experts);
  }
};

template <int kBN, bool kRowScales>  // kRowScales: B has a scale per row (block_rows 1)
__global__ void __launch_bounds__(kThreads, 2)
matmul_thin_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                   const __grid_constant__ MatmulKernelArgs p, int stages, int split) {
  using L = Layout<kBN>;
  using Tiles = TileList<kBN, kWeights, 0>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* scales = reinterpret_cast<float*>(smem + stages * L::kStageBytes);
  float* shares = scales + L::kScaleBytes / 4;  // [rank of the sender][own columns / 4][row of B in the tile][4]
  const int own = L::own(split);
  Barriers* bar = reinterpret_cast<Barriers*>(shares + L::share_floats(split));
  int* first = reinterpret_cast<int*>(bar + 1);
  const int w = warp_index(), lane = threadIdx.x & 31;
  const int rank = split > 1 ? (int)cluster_rank() : 0;

  if (w == kSumWarps) {
    if (lane == 0) {
      for (int i = 0; i < stages; ++i) {
        mbar_init(&bar->full[i], 1);
        mbar_init(&bar->empty[i], 1);
      }
      for (int i = 0; i < L::kBuffers; ++i) {
        mbar_init(&bar->tfull[i], 1);
        mbar_init(&bar->tempty[i], kSumWarps);
      }
      for (int i = 0; i < kScaleStages; ++i) {
        mbar_init(&bar->sfull[i], 32);
        mbar_init(&bar->sempty[i], kSumWarps);
      }
      mbar_init(&bar->got, 1);
      mbar_init(&bar->taken, kSumWarps * split);
      fence_mbar_init();
      tma_prefetch_desc(&amap);
      tma_prefetch_desc(&bmap);
    }
  } else if (w == kSumWarps + 1) {
    tmem_alloc(&bar->tmem, L::kTmemCols);
  }
  __syncwarp();
  if (split > 1) cluster_arrive();  // (the barriers are set up)
  grid_begin();
  if (w == kSumWarps + 2) Tiles::fill(p, first);
  tcgen05_before_sync();
  __syncthreads();
  if (split > 1) cluster_wait();
  tcgen05_after_sync();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, bar->tmem, 0);
  const int tiles = first[member_count(p)];
  const int lg_split = __ffs(split) - 1;  // 1, 2, 4 or 8: shifts, for a division takes as long as the copy of a block
  const int t0 = blockIdx.x >> lg_split, step = gridDim.x >> lg_split;
  bool ok = true;
  // This CTA's share of a tile's blocks.
  auto share = [&](const Tile& tl, int& begin, int& end) {
    begin = (tl.nkb * rank) >> lg_split;
    end = (tl.nkb * (rank + 1)) >> lg_split;
  };

  if (w == kSumWarps) {
    uint32_t s = 0, phase = 1, sent = 0;
    for (int t = t0; t < tiles && ok; t += step) {
      const Tile tl = Tiles::at(p, first, t);
      int kb, end;
      share(tl, kb, end);
      int32_t x = (tl.kb0 + kb) * kBK;
      for (; kb < end; ++kb, x += kBK) {
        if (!mbar_wait(&bar->empty[s], phase)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(&bar->full[s], L::kStageBytes);
          const uint32_t dst = smem_u32(smem + s * L::kStageBytes), full = smem_u32(&bar->full[s]);
          tma_load(dst, &bmap, x, (int32_t)tl.b_row, full);
          tma_load(dst + kStageW, &amap, x, (int32_t)tl.a_row, full);
        }
        __syncwarp();
        ++sent;
        if (++s == (uint32_t)stages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) report_timeout(p.status);
    if (!ok)  // let the copies in flight land
      for (uint32_t i = sent < (uint32_t)stages ? 0 : sent - stages; i < sent; ++i)
        mbar_wait(&bar->full[i % stages], (i / stages) & 1);
  } else if (w == kSumWarps + 1) {
    constexpr uint32_t kIdesc = idesc_e4m3(kWeights, kBN);
    const uint64_t desc0 = operand_desc(smem_u32(smem));
    uint32_t s = 0, phase = 0, buf = 0, tphase = 1;
    for (int t = t0; t < tiles && ok; t += step) {
      const Tile tl = Tiles::at(p, first, t);
      int kb, end;
      share(tl, kb, end);
      for (; kb < end; ++kb) {
        if (!mbar_wait(&bar->full[s], phase) || !mbar_wait(&bar->tempty[buf], tphase)) {
          ok = false;
          break;
        }
        tcgen05_after_sync();
        if (elect_one()) {
          const uint64_t a = desc0 + s * (L::kStageBytes / 16), b = a + kStageW / 16;
#pragma unroll
          for (int k = 0; k < kBK / 32; ++k)
            umma_e4m3<1>(tmem + buf * kBN, a + 2 * k, b + 2 * k, kIdesc, k > 0);
          umma_commit(&bar->tfull[buf]);
          umma_commit(&bar->empty[s]);
        }
        __syncwarp();
        if (++s == (uint32_t)stages) {
          s = 0;
          phase ^= 1;
        }
        if (++buf == L::kBuffers) {
          buf = 0;
          tphase ^= 1;
        }
      }
    }
    if (!ok) report_timeout(p.status);
  } else if (w == kSumWarps + 2) {
    const int64_t kblocks = (p.a_cols + kBK - 1) / kBK, nblocks = (p.b_rows + 127) / 128;
    uint32_t it = 0;
    for (int t = t0; t < tiles && ok; t += step) {
      const Tile tl = Tiles::at(p, first, t);
      int kb, end;
      share(tl, kb, end);
      const int64_t member = p.wgrad || tl.nkb == 0 ? 0 : tl.member;
      const float* pa = p.sa + (int64_t)(tl.kb0 + kb) * p.a_rows + tl.a_row;
      const int64_t last_a = p.a_rows - 1 - tl.a_row;
      const float* pb;
      if constexpr (kRowScales)
        pb = p.sb + (member * kblocks + tl.kb0 + kb) * p.b_rows + tl.n0;
      else
        pb = p.sb + (member * nblocks + tl.n0 / 128) * kblocks + tl.kb0 + kb;
      for (; kb < end; kb += kScaleBatch, ++it) {
        const uint32_t s = it % kScaleStages;
        if (!mbar_wait(&bar->sempty[s], ((it / kScaleStages) & 1) ^ 1)) {
          ok = false;
          break;
        }
        uint32_t dst = smem_u32(scales + s * kScaleBatch * L::kScaleFloats) + 4 * lane;
        const int n = min(kScaleBatch, end - kb);
        for (int j = 0; j < n; ++j, dst += 4 * L::kScaleFloats) {
#pragma unroll
          for (int i = 0; i < (kBN + 31) / 32; ++i)
            if (lane + 32 * i < kBN) cp_async4(dst + 128 * i, pa + min((int64_t)(lane + 32 * i), last_a), true);
          pa += p.a_rows;
          if constexpr (kRowScales) {
#pragma unroll
            for (int i = 0; i < kWeights / 32; ++i)
              cp_async4(dst + 4 * kBN + 128 * i, pb + min(lane + 32 * i, tl.cols - 1), true);
            pb += p.b_rows;
          } else {
            if (lane == 0) cp_async4(dst + 4 * kBN, pb, true);
            ++pb;
          }
        }
        cp_async_arrive(&bar->sfull[s]);
      }
    }
    if (!ok) report_timeout(p.status);
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    const uint32_t lane_base = tmem + ((uint32_t)(32 * w) << 16);
    const uint32_t sc = smem_u32(scales);
    const int n_in_tile = 32 * w + lane;
    uint32_t batch = 0, buf = 0, tphase = 0, round = 0;
    auto store = [&](const Tile& tl, int c, float v) {
      if (c >= tl.rows || n_in_tile >= tl.cols) return;
      const int64_t at = (tl.out_row + c) * p.b_rows + tl.n0 + n_in_tile;
      if (p.out_bf16) {
        uint16_t h;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
        static_cast<uint16_t*>(p.out)[at] = h;
      } else {
        static_cast<float*>(p.out)[at] = v;
      }
    };
    for (int t = t0; t < tiles && ok; t += step) {
      const Tile tl = Tiles::at(p, first, t);
      int begin, end;
      share(tl, begin, end);
      float acc[kBN];
#pragma unroll
      for (int i = 0; i < kBN; ++i) acc[i] = 0.0f;
      uint32_t off = 0;
#pragma unroll 1
      for (int kb = begin; kb < end; ++kb) {
        const int in_batch = (kb - begin) & (kScaleBatch - 1);
        if (in_batch == 0) {
          const uint32_t ss = batch % kScaleStages;
          off = sc + ss * (kScaleBatch * L::kScaleFloats * 4);
          ok = mbar_wait(&bar->sfull[ss], (batch / kScaleStages) & 1);
          if (!ok) break;
        }
        float sw;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(sw) : "r"(off + 4 * kBN + (kRowScales ? 4 * n_in_tile : 0)));
        ok = mbar_wait(&bar->tfull[buf], tphase);
        if (!ok) break;
        __syncwarp();
        tcgen05_after_sync();
        constexpr int kChunk = kBN < 32 ? kBN : 32;
#pragma unroll
        for (int c = 0; c < kBN; c += kChunk) {
          uint32_t v[kChunk];
          tmem_read(lane_base + buf * kBN + c, v);
          if (c == kBN - kChunk) {
            // everything is read: the accumulator may be overwritten
            tcgen05_before_sync();
            if (lane == 0) mbar_arrive(&bar->tempty[buf]);
          }
#pragma unroll
          for (int i = 0; i < kChunk; i += 4) {
            float x[4];
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                         : "r"(off + 4 * (c + i)));
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[c + i + j] = __fmaf_rn(__fmul_rn(__uint_as_float(v[i + j]), x[j]), sw, acc[c + i + j]);
          }
        }
        off += 4 * L::kScaleFloats;
        if (kb + 1 == end || in_batch == kScaleBatch - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->sempty[batch % kScaleStages]);
          ++batch;
        }
        if (++buf == L::kBuffers) {
          buf = 0;
          tphase ^= 1;
        }
      }
      if (!ok) break;
      if (split == 1) {
#pragma unroll
        for (int i = 0; i < kBN; ++i) store(tl, i, acc[i]);
        continue;
      }
      // Column c belongs to rank c / own.  Columns travel in fours.
      const int lg = __ffs(own) - 1;
      ok = mbar_wait_cluster(&bar->taken, (round & 1) ^ 1, p.status);
      if (!ok) break;
      const int held = max(0, min(own, tl.rows - rank * own));  // columns of this CTA that exist
      if (w == 0 && lane == 0) mbar_arrive_expect_tx(&bar->got, split * kWeights * 4 * ((held + 3) & ~3));
      const uint32_t mine = smem_u32(shares) + 4 * (rank * own * kWeights + 4 * n_in_tile), got = smem_u32(&bar->got);
      // To the ranks from this one on, then to those before it, so that not all
      // send to one CTA at a time (200 rows to 1040 x 8192: 12.6 to 11.7 us).
#pragma unroll
      for (int before = 0; before < 2; ++before)
#pragma unroll
        for (int i = 0; i < kBN; i += 4) {
          if (i >= tl.rows) break;
          if (((i >> lg) < rank) == before)
            store_async(map_to_cta(mine + 4 * (i & (own - 1)) * kWeights, i >> lg), acc[i], acc[i + 1], acc[i + 2],
                        acc[i + 3], map_to_cta(got, i >> lg));
        }
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
        store(tl, at, sum.x);
        store(tl, at + 1, sum.y);
        store(tl, at + 2, sum.z);
        store(tl, at + 3, sum.w);
      }
      if (t + step < tiles) {
        __syncwarp();
        if (lane < split) mbar_arrive_cluster_release(map_to_cta(smem_u32(&bar->taken), lane));
      }
      ++round;
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
  if (w == kSumWarps + 1) tmem_dealloc(tmem, L::kTmemCols);
}

template <int kBN>
cudaError_t launch(const Fp8MatmulArgs& a, const MatmulKernelArgs& p, int64_t tiles, int split, const LaunchCtx& ctx) {
  using L = Layout<kBN>;
  CUtensorMap amap, bmap;
  cudaError_t e = make_fp8_tensor_map(&amap, a.a, a.a_rows, a.a_cols, kBN);
  if (e != cudaSuccess) return e;
  e = make_fp8_tensor_map(&bmap, a.b, a.wgrad ? a.b_rows : a.b_rows * a.experts, a.a_cols, kWeights);
  if (e != cudaSuccess) return e;
  constexpr int kPerCta = 113 * 1024;  // two CTAs share an SM's 228 KB, 1 KB of it reserved for each
  const int rest = 1024 + L::rest(a.experts, split);
  int stages = (kPerCta - rest) / L::kStageBytes;
  if (stages > kMaxStages) stages = kMaxStages;
  const int smem = rest + stages * L::kStageBytes;
  const auto kernel = a.b_block_rows == 1 ? matmul_thin_kernel<kBN, true> : matmul_thin_kernel<kBN, false>;
  static std::atomic<uint64_t> allowed[2];
  e = allow_smem(reinterpret_cast<const void*>(kernel), kPerCta, allowed[a.b_block_rows == 1]);
  if (e != cudaSuccess) return e;
  const int64_t room = 2 * ctx.num_sms / split;
  MatmulKernelArgs k = p;
  void* args[] = {&amap, &bmap, &k, &stages, &split};
  return launch_dependent(reinterpret_cast<const void*>(kernel), dim3((unsigned)((tiles < room ? tiles : room) * split)),
                    dim3(kThreads), smem, ctx.stream, args, split);
}

}  // namespace

ThinPlan thin_plan(const Fp8MatmulArgs& a, const LaunchCtx& ctx) {
  const int64_t members = a.offsets ? a.experts : 1;
  const int64_t rows = a.wgrad ? a.a_rows : (a.a_rows + members - 1) / members;
  ThinPlan t;
  t.bn = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  t.tiles = members * ((rows + t.bn - 1) / t.bn) * ((a.b_rows + kWeights - 1) / kWeights);
  // Eight CTAs, four or two share a tile's blocks where all of them fit beside
  // one another (two per SM) and each keeps two blocks or more.  5120 x 4096
  // weights, one row: 10.5 us alone, 6.8 us in fours (eights: two turns, 10.1 us);
  // 1024 x 4096, 16 rows: 8.4, 4.6 and 4.2 us.  Two gain less, so they want more
  // blocks: 10240 x 8192, 32 rows 19.2 us against 22.8, 12800 x 2048, 16 rows 8.2
  // either way.
  const int64_t k = a.wgrad ? (a.a_cols + members - 1) / members : a.a_cols;
  const int64_t kb = (k + kBK - 1) / kBK;
  t.split = 1;
  for (int s = 8; s >= 2 && t.split == 1; s /= 2)
    if (t.tiles * s <= 2 * ctx.num_sms && kb >= (s == 2 ? 32 : 16)) t.split = s;
  return t;
}

cudaError_t launch_matmul_thin(const Fp8MatmulArgs& a, const MatmulKernelArgs& p, const LaunchCtx& ctx) {
  const ThinPlan t = thin_plan(a, ctx);
  // No more tiles than this, whatever the offsets.
  const int64_t tn = (a.b_rows + kWeights - 1) / kWeights, tm = (a.a_rows + t.bn - 1) / t.bn;
  const int64_t most = tn * (a.wgrad ? tm * a.experts : tm + (a.offsets ? a.experts : 0));
  if (t.bn == 16) return launch<16>(a, p, most, t.split, ctx);
  if (t.bn == 32) return launch<32>(a, p, most, t.split, ctx);
  return launch<64>(a, p, most, t.split, ctx);
}

}  // namespace fp8
}  // namespace nvfp4
