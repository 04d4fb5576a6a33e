// fp4_matmul.cu -- the product of 4-bit operands:
//     c[m][n] = fa fb sum_k a[m][k] sa[m][k / b] b[n][k] sb[n][k / b]
// with b = 16 and E4M3 scales (NVFP4; fa, fb = amax / 2688) or b = 32 and
// powers of two (MXFP4; fa = fb = 1).  The tensor cores take codes and scales
// as they are (tcgen05 block_scale) and sum in FP32 in tensor memory.
//
// Persistent, warp-specialised, one pair of CTAs (two SMs) per 256 x 256
// tile: each CTA stages 128 rows of A and 128 rows of B per 256 elements by
// TMA, with the scales of its rows of A and of all rows of B, and one lane of the
// first CTA copies the scales into both tensor memories and issues the pair's
// MMAs (256 x 256 x 64).  Eight warps of each CTA write a finished tile (32 rows
// by 128 columns each) through shared memory by TMA while the next one is
// multiplied.  Tensor memory has 512 columns: two accumulators of 256 would
// leave none for scales, so they share 48 columns, which are read first and
// given back for the next tile at once.
//
// Swizzled scales are copied by TMA as they stand; compact ones are put in order
// by six warps, 128 rows of two stages each in turn.
//
// 8192 x 5120 x 8192 (NVFP4, BF16 out): 98 us, 7.0 PFLOP/s, the tensor pipe 81 % busy at
// the clock the power limit leaves (1.87 GHz in one launch).  An MMA of 64 elements
// takes 128 cycles, so a stage asks the L2 for 74 bytes a cycle and SM, and the copies
// alone (one MMA a stage) take 80 us, about as long as the MMAs alone at this clock:
// the two bound it together.  Without the scales' way into tensor memory it would
// be 95; each half of B's scales sent to both CTAs at once (multicast) changes nothing.
// 4096 x 4096 x 4096: swizzled scales 25.5 us, with an amax for each row of both 26.3 (75 when
// every warp worked the columns' factors out for itself), compact scales 32.
#include "fp4_tiles.cuh"

namespace nvfp4 {
namespace fp4 {
namespace {

constexpr int kStages = 5;
constexpr int kStageA = 128 * kStageRow, kCodes = 2 * kStageA;
constexpr int kFirstScale = 2, kPairScaleWarps = 6, kOutWarps = 8, kFirstOut = 8;
constexpr int kThreads = 32 * (kFirstOut + kOutWarps);
constexpr int kSecond = 208;  // first column of the second accumulator
constexpr int kScaleCols = kSecond + 256;  // then the scales
constexpr int kOutBox = 32 * 128;  // bytes of one output box: 32 rows of 128 bytes
constexpr int kBand = 8;           // row tiles of a band: tiles in flight share both operands' rows in L2

struct __align__(16) Barriers {
  uint64_t full[kStages], empty[kStages], tfull[2], tempty;
  uint32_t tmem;
  uint32_t pad;
  uint4 heard;  // (word of the second CTA's pieces; nobody reads it)
};

template <int kBlock>
struct Layout {
  static constexpr int kScales = Format<kBlock>::kScaleBytes;  // of 128 rows
  static constexpr int kStageBytes = kCodes + 3 * kScales;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kOutWarps * kOutBox + (int)sizeof(Barriers);
  static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
  static_assert(kStageBytes % 1024 == 0, "swizzled operands");
  static_assert(kScaleCols + 3 * Format<kBlock>::kCols <= 512, "tensor memory");
};

// Word to the first CTA that a piece of scales of the second is in its place.  A thread
// of the first CTA issues the copies that read it, so the hand-over is one between
// CTAs.  An arrival would have to release at cluster scope, for which a warp waits about a
// microsecond (4096 x 4096 x 4096 45 us, 8192 x 8192 x 8192 292; 60 and 420 if an idle
// warp does it for all).  The bytes of an asynchronous store are counted on the
// barrier with such a release, and the warp goes on: 32 and 191 us.  (An arrival of CTA
// scope, which promises nothing to the other CTA, takes 28.5 and 168.)
constexpr int kWord = 16;
__device__ __forceinline__ void tell_first(Barriers* bar, int slot) {
  store_async(map_to_cta(smem_u32(&bar->heard), 0), 0.0f, 0.0f, 0.0f, 0.0f, map_to_cta(smem_u32(&bar->full[slot]), 0));
}

// An item: a tile of 256 x 256, or its left or right half.
struct Item {
  int m0, n0, half;
};

template <int kBlock>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
matmul_pair_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                   const __grid_constant__ CUtensorMap samap, const __grid_constant__ CUtensorMap sbmap,
                   const __grid_constant__ CUtensorMap omap, const __grid_constant__ MatmulKernelArgs p) {
  using F = Format<kBlock>;
  using L = Layout<kBlock>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* out_stage = smem + kStages * L::kStageBytes;
  Barriers* bar = reinterpret_cast<Barriers*>(out_stage + kOutWarps * kOutBox);
  const int w = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  // compact scales of a stage, 128 rows at a time: A's, and the halves of B's
  const int pieces = (p.a.swizzled ? 0 : 1) + (p.b.swizzled ? 0 : 2);

  if (w == 0) {
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) {
        mbar_init(&bar->full[i], 1 + pieces);  // the copies (word of the second CTA's pieces among them); the first's pieces
        mbar_init(&bar->empty[i], 1);
      }
      mbar_init(&bar->tfull[0], 1);
      mbar_init(&bar->tfull[1], 1);
      mbar_init(&bar->tempty, 2 * kOutWarps);
      fence_mbar_init();
      tma_prefetch_desc(&amap);
      tma_prefetch_desc(&bmap);
    }
  } else if (w == 1) {
    tmem_alloc_pair(&bar->tmem, 512);
  }
  __syncwarp();
  cluster_arrive();  // (barriers and tensor memory are set up)
  grid_begin();
  tcgen05_before_sync();
  __syncthreads();
  cluster_wait();
  tcgen05_after_sync();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, bar->tmem, 0);
  // Tiles are dealt out in turns of one per pair.  Where the last turn would
  // leave half of the pairs idle or more, its tiles are halved (256 x 128).
  const int t0 = blockIdx.x >> 1, step = gridDim.x >> 1;
  const int whole = p.tiles_a * p.tiles_b, over = whole % step, uncut = 2 * over <= step ? whole - over : whole;
  const int items = uncut + 2 * (whole - uncut);
  auto at = [&](int i) {
    const int t = i < uncut ? i : uncut + (i - uncut) / 2;
    const int band = t / (kBand * p.tiles_b), in_band = t - band * kBand * p.tiles_b;
    const int height = min(kBand, p.tiles_a - band * kBand);
    const int column = in_band / height;
    return Item{(band * kBand + in_band - column * height) * 256,
                column * 256 + (i < uncut ? 0 : 128 * ((i - uncut) & 1)), i >= uncut};
  };
  const int nkb = (int)((p.K + kStageK - 1) / kStageK);
  const int full_stages = (int)(p.K / kStageK), last_steps = (int)((p.K % kStageK + 63) / 64);  // of 64 elements
  bool ok = true;

  if (w == 0) {
    uint32_t s = 0, phase = 1;
    for (int i = t0; i < items && ok; i += step) {
      const Item it = at(i);
      if (it.n0 >= p.b.rows) continue;  // the right half of a tile that has none
      const int32_t arow = it.m0 + 128 * rank;
      // each CTA holds half of B's rows: of a halved tile, 64 (and 64 that no MMA reads)
      const int32_t brow = it.n0 + (it.half ? 64 : 128) * rank;
      for (int kb = 0; kb < nkb; ++kb) {
        if (!mbar_wait(&bar->empty[s], phase)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          if (rank == 0)
            mbar_arrive_expect_tx(&bar->full[s], 2 * (kCodes + (p.a.swizzled ? L::kScales : 0) +
                                                      (p.b.swizzled ? 2 * L::kScales : 0)) + pieces * kWord);
          const uint32_t dst = smem_u32(smem + s * L::kStageBytes);
          const uint32_t full = map_to_cta(smem_u32(&bar->full[s]), 0);
          tma_load_pair(dst, &amap, kb * kStageRow, arow, full);
          tma_load_pair(dst + kStageA, &bmap, kb * kStageRow, brow, full);
          // (a row of 128 rows' tiles, in elements of 8 bytes)
          if (p.a.swizzled) tma_load_pair(dst + kCodes, &samap, kb * (L::kScales / 8), arow / 128, full);
          if (p.b.swizzled) tma_load_pair(dst + kCodes + L::kScales, &sbmap, kb * (L::kScales / 8), it.n0 / 128, full);
        }
        __syncwarp();
        if (++s == kStages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) {  // given up: the copies in flight land long before this ends
      report_timeout(p.status);
      const long long c0 = clock64();
      while (clock64() - c0 < 50000000LL) {
      }
    }
  } else if (w == 1 && rank == 0) {
    const uint64_t desc0 = operand_desc(smem_u32(smem));
    const uint64_t sdesc0 = scale_desc(smem_u32(smem) + kCodes);
    const uint32_t sa = tmem + kScaleCols, sb = sa + F::kCols;
    uint32_t s = 0, phase = 0, buf = 0, tphase = 1;
    for (int i = t0; i < items && ok; i += step) {
      const Item it = at(i);
      if (it.n0 >= p.b.rows) continue;
      const uint32_t idesc = it.half ? F::idesc(256, 128) : F::idesc(256, 256);
      if (!mbar_wait(&bar->tempty, tphase)) {
        ok = false;
        break;
      }
      tphase ^= 1;
      const uint32_t d = tmem + buf * kSecond;
      for (int kb = 0; kb < nkb; ++kb) {
        if (!(pieces ? mbar_wait_acquire(&bar->full[s], phase) : mbar_wait(&bar->full[s], phase))) {
          ok = false;
          break;
        }
        tcgen05_after_sync();
        const uint64_t a = desc0 + s * (L::kStageBytes / 16), b = a + kStageA / 16;
        const uint64_t ds = sdesc0 + s * (L::kStageBytes / 16);
        const uint32_t add = kb > 0;
        // A step's scales: four columns of A's, eight of B's (its second 128 rows behind the first).
        auto copy = [&](int j) {
          scales_to_tmem<2>(sa + 4 * j, ds + j * (kScaleTile / 16));
          scales_to_tmem<2>(sb + 8 * j, ds + (L::kScales + j * kScaleTile) / 16);
          scales_to_tmem<2>(sb + 8 * j + 4, ds + (2 * L::kScales + j * kScaleTile) / 16);
        };
        auto multiply = [&](int k) {
          umma_fp4<2, kBlock>(d, a + 2 * k, b + 2 * k, idesc | F::half(k), sa + F::col(k), sb + 2 * F::col(k), k > 0 ? 1 : add);
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
          if (kb + 1 == nkb) umma_commit_pair(&bar->tfull[buf]);
          umma_commit_pair(&bar->empty[s]);
        }
        __syncwarp();
        if (++s == kStages) {
          s = 0;
          phase ^= 1;
        }
      }
      buf ^= 1;
    }
    if (!ok) report_timeout(p.status);
  } else if (w >= kFirstScale && w < kFirstScale + kPairScaleWarps) {
    // A warp puts a piece of two stages in order, whose loads are in flight together: a
    // row's 16 bytes of one stage are half a sector (a stage at a time took 13 % longer).
    // At most three pairs of stages are dealt out at once: a warp that wrote stage i
    // waits for stage i + 5 next, or an earlier one; it knows that stage i - kStages is
    // over, so what it waits for is at most one phase of the barrier away.
    static_assert(kStages == 5, "three pairs");
    const int active = min(kPairScaleWarps, 3 * pieces);
    if (w - kFirstScale < active) {
      uint32_t s = 0, phase = 1;
      int turn = w - kFirstScale;  // pieces until the next of this warp
      const CompactScales<kBlock> of_a(p.a.scale, p.K, p.a.rows), of_b(p.b.scale, p.K, p.b.rows);
      for (int i = t0; i < items && ok; i += step) {
        const Item it = at(i);
        if (it.n0 >= p.b.rows) continue;
        for (int kb = 0; kb < nkb && ok; kb += 2) {
          const bool two = kb + 1 < nkb;
          const uint32_t slot[2] = {s, s + 1 == kStages ? 0 : s + 1};
          const uint32_t use[2] = {phase, s + 1 == kStages ? phase ^ 1 : phase};
          for (int j = 0; j < pieces; ++j) {
            if (turn-- != 0) continue;
            turn = active - 1;
            const int piece = j + (p.a.swizzled ? 1 : 0);
            const bool there = piece < 2 || !it.half;
            uint32_t v[2][4][F::kTiles];
            if (piece == 0)
              of_a.read_two(it.m0 + 128 * (int64_t)rank, kb, two, v);
            else if (there)
              of_b.read_two(it.n0 + 128 * (piece - 1), kb, two, v);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (h == 1 && !two) break;
              ok = ok && mbar_wait(&bar->empty[slot[h]], use[h]);
              if (!ok) break;
              if (there) of_a.write(smem_u32(smem + slot[h] * L::kStageBytes) + kCodes + piece * L::kScales, v[h]);
              fence_proxy_async_shared();
              __syncwarp();
              if (lane == 0) {
                if (rank == 0)
                  mbar_arrive(&bar->full[slot[h]]);
                else
                  tell_first(bar, slot[h]);
              }
            }
          }
          s = two ? slot[1] : slot[0], phase = two ? use[1] : use[0];
          if (++s == kStages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) report_timeout(p.status);
    }
  } else if (w >= kFirstOut) {
    const int q = w & 3, half = (w - kFirstOut) >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16) + half * 128;
    const uint32_t tempty = map_to_cta(smem_u32(&bar->tempty), 0);
    const uint32_t box = smem_u32(out_stage + (w - kFirstOut) * kOutBox);
    const int row0 = 128 * (int)rank + 32 * q;
    uint32_t buf = 0, tphase = 0;
    for (int i = t0; i < items && ok; i += step) {
      const Item it = at(i);
      if (it.n0 >= p.b.rows) continue;
      const int rows = (int)min((int64_t)256, p.a.rows - it.m0) - row0;  // that this warp has
      const int cols = (int)min((int64_t)(it.half ? 128 : 256), p.b.rows - it.n0) - 128 * half;
      const float fa = row_factor(p.a, p.a.amax_per_row ? it.m0 + row0 + lane : 0);
      const Factor all = factor(fa, p.b.amax_per_row ? 1.0f : row_factor(p.b, 0));
      // with an amax for each column: lane l has those of columns l, 32 + l, ... of the warp's 128
      float fb[4] = {};
      if (p.b.amax_per_row)
#pragma unroll
        for (int k = 0; k < 4; ++k) fb[k] = row_factor(p.b, it.n0 + 128 * half + 32 * k + lane);
      ok = mbar_wait(&bar->tfull[buf], tphase);
      if (!ok) break;
      __syncwarp();
      tcgen05_after_sync();
      // The accumulators share columns 208 .. 255: of the first one the last, of
      // the second one the first.  The warps that hold them read them before they
      // let the next tile begin; the others are through with the tile before.
      const bool holds = half != (int)buf, work = rows > 0 && cols > 0;
      auto release = [&]() {
        tcgen05_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty);
      };
      if (!holds || !work) release();
      const uint32_t src = lane_base + buf * kSecond;
      // 128 bytes of the rows, from column c of the warp's: by TMA, which leaves out
      // rows past the last; rows off 16-byte boundaries the warp writes itself.
      auto put = [&](int c, auto&& fill) {
        if (c >= cols) return;
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
        fill();
        if (p.out_map) {
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            tma_store(&omap, box, it.n0 + 128 * half + c, it.m0 + row0);
            bulk_commit();
          }
        } else {
          __syncwarp();
          const int n = min(32, rows);
#pragma unroll 1
          for (int r0 = 0; r0 < n; r0 += 8) {  // eight rows read, then written
            uint32_t x[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
              asm volatile("ld.shared.u32 %0, [%1];"
                           : "=r"(x[r])
                           : "r"(box + (r0 + r) * 128 + (((lane >> 2) ^ r) * 16) + (lane & 3) * 4));
            const int64_t to = (int64_t)(it.m0 + row0 + r0) * p.b.rows + it.n0 + 128 * half + c;
            if (p.out_bf16) {
              uint16_t* dst = static_cast<uint16_t*>(p.out) + to + 2 * lane;
              const bool lo = c + 2 * lane < cols, hi = c + 2 * lane + 1 < cols;
#pragma unroll
              for (int r = 0; r < 8; ++r, dst += p.b.rows) {
                if (lo && r0 + r < n) dst[0] = (uint16_t)x[r];
                if (hi && r0 + r < n) dst[1] = (uint16_t)(x[r] >> 16);
              }
            } else {
              uint32_t* dst = static_cast<uint32_t*>(p.out) + to + lane;
              const bool there = c + lane < cols;
#pragma unroll
              for (int r = 0; r < 8; ++r, dst += p.b.rows)
                if (there && r0 + r < n) *dst = x[r];
            }
          }
          __syncwarp();
        }
      };
      if (work) {
        // 64 columns at a time, the shared ones first
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int c = 64 * (half ? 1 - h : h);
          uint32_t v[64];
          tmem_read(src + c, v);
          if (h == 0 && holds) release();
          if (p.b.amax_per_row) {
            const float f0 = c == 0 ? fb[0] : fb[2], f1 = c == 0 ? fb[1] : fb[3];
            if (one_product(fa, f0, f1)) {
#pragma unroll
              for (int k = 0; k < 64; ++k)
                v[k] = __float_as_uint(__fmul_rn(__uint_as_float(v[k]),
                                                 __fmul_rn(fa, __shfl_sync(0xFFFFFFFFu, k < 32 ? f0 : f1, k & 31))));
            } else {
#pragma unroll
              for (int k = 0; k < 64; ++k)
                v[k] = __float_as_uint(factor(fa, __shfl_sync(0xFFFFFFFFu, k < 32 ? f0 : f1, k & 31))(__uint_as_float(v[k])));
            }
          } else {
#pragma unroll
            for (int k = 0; k < 64; ++k) v[k] = __float_as_uint(all(__uint_as_float(v[k])));
          }
          // 16-byte places of a row are swizzled by the row, as TMA expects them
          if (p.out_bf16) {
            put(c, [&]() {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                      : "=r"(o[k])
                      : "f"(__uint_as_float(v[8 * j + 2 * k + 1])), "f"(__uint_as_float(v[8 * j + 2 * k])));
                sts_v4(box + lane * 128 + ((j ^ (lane & 7)) * 16), o[0], o[1], o[2], o[3]);
              }
            });
          } else {
#pragma unroll
            for (int g = 0; g < 2; ++g)
              put(c + 32 * g, [&]() {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  sts_v4(box + lane * 128 + ((j ^ (lane & 7)) * 16), v[32 * g + 4 * j], v[32 * g + 4 * j + 1],
                         v[32 * g + 4 * j + 2], v[32 * g + 4 * j + 3]);
              });
          }
        }
      }
      buf ^= 1;
      tphase ^= buf ^ 1;
    }
    if (!ok) report_timeout(p.status);
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  tcgen05_before_sync();
  __syncthreads();
  cluster_sync();
  tcgen05_after_sync();
  if (w == 1) tmem_dealloc_pair(tmem, 512);
}

// Which of the two kernels a product runs on.  Up to 32 rows the thin one wins
// (8 / 24 rows, N 4096, K 4096: 4.9 / 5.4 us against 8.7 / 10.6; N 512, K 512: 2.6 /
// 3.1 against 4.5 / 6.0).  Above, it does where its tiles are few and long, so that
// eight CTAs share each (64 rows, N 1024, K 8192: 6.1 against 9.3 us; N 4096, K 4096:
// 7.3 / 7.3), and else the paired one (64 rows, N 2048, K 2048: 6.4 against 4.9; N 8192, K
// 8192: 12.1 / 11.9).  Past 64 rows the paired one, within 6 percent, always (96
// rows, N 512, K 8192: 12.4 against 10.4; N 10240, K 8192: 13.7 / 14.5).  Swept over 8
// to 1024 rows, N 512 to 10240, K 512 to 8192, in CUDA graphs.
bool thin_is_faster(const Fp4MatmulArgs& a, const LaunchCtx& ctx) {
  if (a.a.rows <= 32) return true;
  return a.a.rows <= kThinRows && a.K >= 4096 && thin_plan(a, ctx).split == 8;
}

template <int kBlock>
cudaError_t launch_pair(const Fp4MatmulArgs& a, MatmulKernelArgs p, const LaunchCtx& ctx) {
  using L = Layout<kBlock>;
  CUtensorMap amap, bmap, samap = {}, sbmap = {}, omap = {};
  cudaError_t e = make_fp8_tensor_map(&amap, a.a.data, a.a.rows, a.K / 2, 128);
  if (e == cudaSuccess) e = make_fp8_tensor_map(&bmap, a.b.data, a.b.rows, a.K / 2, 128);
  const int64_t scale_row = a.K / (4 * kBlock) * kScaleTile;  // bytes of 128 rows
  if (e == cudaSuccess && a.a.swizzled)
    e = make_scale_tensor_map(&samap, a.a.scale, a.a.rows / 128, scale_row, L::kScales, 1);
  if (e == cudaSuccess && a.b.swizzled)
    e = make_scale_tensor_map(&sbmap, a.b.scale, a.b.rows / 128, scale_row, L::kScales, 2);
  // TMA writes the output where its rows start on 16 bytes.
  p.out_map = a.b.rows * (a.out_bf16 ? 2 : 4) % 16 == 0;
  if (e == cudaSuccess && p.out_map) e = make_matmul_out_map(&omap, a.out, a.out_bf16, a.a.rows, a.b.rows);
  if (e != cudaSuccess) return e;
  p.tiles_a = (int)((a.a.rows + 255) / 256);
  p.tiles_b = (int)((a.b.rows + 255) / 256);
  const int64_t tiles = (int64_t)p.tiles_a * p.tiles_b;
  const unsigned pairs = (unsigned)(2 * tiles < ctx.num_sms / 2 ? 2 * tiles : ctx.num_sms / 2);  // (halves)
  const auto kernel = matmul_pair_kernel<kBlock>;
  static std::atomic<uint64_t> allowed{0};
  e = allow_smem(reinterpret_cast<const void*>(kernel), L::kSmemBytes, allowed);
  if (e != cudaSuccess) return e;
  void* args[] = {&amap, &bmap, &samap, &sbmap, &omap, &p};
  return launch_dependent(reinterpret_cast<const void*>(kernel), dim3(2 * pairs), dim3(kThreads), L::kSmemBytes,
                          ctx.stream, args);
}

}  // namespace
}  // namespace fp4

cudaError_t launch_fp4_matmul(const Fp4MatmulArgs& a, const LaunchCtx& ctx) {
  using namespace fp4;
  if (a.a.rows == 0 || a.b.rows == 0) return cudaSuccess;
  if (a.K == 0) return cudaMemsetAsync(a.out, 0, (size_t)a.a.rows * a.b.rows * (a.out_bf16 ? 2 : 4), ctx.stream);
  MatmulKernelArgs p = {};
  p.a = a.a;
  p.b = a.b;
  p.K = a.K;
  p.out = a.out;
  p.out_bf16 = a.out_bf16;
  p.status = ctx.status;
  if (thin_is_faster(a, ctx)) return launch_matmul_thin(a, p, ctx);
  return a.block == 16 ? launch_pair<16>(a, p, ctx) : launch_pair<32>(a, p, ctx);
}

}  // namespace nvfp4
