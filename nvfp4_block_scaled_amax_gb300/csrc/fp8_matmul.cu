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
// Persistent, warp-specialised, one pair of CTAs (two SMs) per 256 x 256
// tile: each CTA stages 128 rows of A and 128 rows of B per block by TMA, one
// lane of the first CTA issues the pair's MMAs (256 x 256 x 32) into one of
// two accumulators that fill tensor memory (256 columns each), and eight
// warps of each CTA read the finished accumulator of their 128 rows and add
// it, scaled, to their registers (128 per thread) while the next block is
// multiplied.  Output leaves through shared memory by TMA while the next
// tile is summed; one more warp works the tiles out ahead.
//
// Measured at 8192 x 5120 x 8192 (BF16 out, 128 x 128 blocks of B): 210 us, 3.3
// PFLOP/s, in bursts of some milliseconds; back to back for seconds 245 us, 2.8
// PFLOP/s, for the power limit lowers the clock.  At 4096 x 4864 x 16384 (FP32
// out) a scale per row of B takes 236 us, 128 x 128 blocks 200 (bursts, as every
// figure below).  The MMAs alone take 168 us, with their operand copies 185 us
// (256 x 128 MMAs: 240 us, so the tile is 256 wide although two accumulators
// then leave no third to run ahead).  What bounds it is the hand-over: an
// accumulator must be heard of, read, scaled and given back within the time
// of one block's MMAs (about 520 cycles), of which the scaled sums alone take
// 290.  The tensor pipe is 78 percent busy (60 with a scale per row of B).
#include "fp8_tiles.cuh"

namespace nvfp4 {
namespace fp8 {
namespace {

constexpr int kStages = 4;
constexpr int kStageA = 128 * kBK, kStageBytes = 2 * kStageA;
constexpr int kBufCols = 256;    // tensor-memory columns of an accumulator
constexpr int kChunk = 64;       // columns read at a time
constexpr int kScaleStages = 2;
constexpr int kScaleBatch = 8;   // blocks per scale stage: one hand-over for eight blocks
constexpr int kScaleFloats = 128 + 256;  // of A's 128 rows, of B's 256
constexpr int kSumWarps = 8;
constexpr int kOutBox = 32 * 128;   // bytes of one output box: 32 rows of 128 bytes
constexpr int kOutBoxes = 2;        // per warp: one is written while the other is stored
constexpr int kThreads = 32 * (4 + kSumWarps);
using Tiles = TileList<256, 256, 8>;

constexpr float kSmallestNormal = 0x1p-126f, kLargest = 0x1.fffffep127f;

constexpr int kTileSlots = 4;       // tiles worked out ahead

// A tile as one warp hands it to the others (see Tile).
struct __align__(16) TileSlot {
  int nkb, kb0, half, member;  // half: of a halved tile
  int a_row, b_row, n0, out_row;
  int rows, cols, pad[2];
};

struct __align__(16) Barriers {
  uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], sfull[kScaleStages], sempty[kScaleStages];
  uint64_t listed[kTileSlots], done[kTileSlots];
  TileSlot tiles[kTileSlots];
  uint32_t tmem;
  uint32_t pad[3];
};

constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kSumWarps * kOutBoxes * kOutBox +
                           kScaleStages * kScaleBatch * kScaleFloats * 4 + (int)sizeof(Barriers) + 4 * Tiles::ints(kMaxExperts);
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
static_assert(kScaleStages == 2, "the summing warps toggle between two scale stages");

template <bool kColScales>  // B has a scale per row (block_rows 1)
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
matmul_pair_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                   const __grid_constant__ CUtensorMap omap,
                   const __grid_constant__ MatmulKernelArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* out_stage = smem + kStages * kStageBytes;
  float* scales = reinterpret_cast<float*>(out_stage + kSumWarps * kOutBoxes * kOutBox);
  Barriers* bar = reinterpret_cast<Barriers*>(scales + kScaleStages * kScaleBatch * kScaleFloats);
  int* first = reinterpret_cast<int*>(bar + 1);
  const int w = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();

  if (w == 0) {
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) {
        mbar_init(&bar->full[i], 1);
        mbar_init(&bar->empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar->tfull[i], 1);
        mbar_init(&bar->tempty[i], 2 * kSumWarps);
      }
      for (int i = 0; i < kScaleStages; ++i) {
        mbar_init(&bar->sfull[i], kColScales ? 33 : 32);  // the lanes' own copies (and the bulk copies)
        mbar_init(&bar->sempty[i], kSumWarps);
      }
      for (int i = 0; i < kTileSlots; ++i) {
        mbar_init(&bar->listed[i], 1);
        mbar_init(&bar->done[i], kSumWarps + (rank == 0 ? 3 : 2));
      }
      fence_mbar_init();
      tma_prefetch_desc(&amap);
      tma_prefetch_desc(&bmap);
      if (p.out_map) tma_prefetch_desc(&omap);
    }
  } else if (w == 1) {
    tmem_alloc_pair(&bar->tmem, 512);
  }
  __syncwarp();
  cluster_arrive();  // (barriers and tensor memory are set up)
  grid_begin();
  if (w == 2) Tiles::fill(p, first);
  tcgen05_before_sync();
  __syncthreads();
  cluster_wait();
  tcgen05_after_sync();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, bar->tmem, 0);
  // Tiles are dealt out in turns of one per pair.  Where the last turn would
  // leave half of the pairs idle or more, its tiles are halved (256 x 128), one
  // half to a pair: such a turn takes about 0.6 of a whole one.
  const int t0 = blockIdx.x >> 1, step = gridDim.x >> 1;
  const int whole = first[member_count(p)], over = whole % step, uncut = 2 * over <= step ? whole - over : whole;
  const int tiles = uncut + 2 * (whole - uncut);
  const int items = t0 < tiles ? (tiles - 1 - t0) / step + 1 : 0;
  auto slot_of = [&](int i) { return bar->tiles + i % kTileSlots; };
  // Waits for tile i of this CTA; a warp that is through with it calls leave.
  auto listed = [&](int i) { return mbar_wait(&bar->listed[i % kTileSlots], (i / kTileSlots) & 1); };
  auto leave = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar->done[i % kTileSlots]);
  };

  if (w < 4) {
    // 128 threads here, 256 that sum, 168 registers each at launch.  Every
    // register that these warps can spare helps the sums (72 / 216: weight gradient
    // 153 us against 147, the product above 215.5 against 213.7); with a scale
    // per row of B they need more than 24.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kColScales ? 40 : 24));
    // These loops are the same in all lanes of their warp; one lane issues.
    if (w == 0) {
      // both operands' slices, counted on the first CTA's barrier
      uint32_t s = 0, phase = 1;
      bool ok = true;
      for (int i = 0; i < items && ok; ++i) {
        if (!(ok = listed(i))) break;
        const TileSlot* tl = slot_of(i);
        const int32_t arow = tl->a_row + 128 * rank;
        // each CTA holds half of B's rows: of a halved tile, 64 (and 64 that no MMA reads)
        const int32_t brow = tl->b_row + (tl->half ? 64 : 128) * rank;
        int32_t x = tl->kb0 * kBK;
        const int nkb = __shfl_sync(0xFFFFFFFFu, tl->nkb, 0);
        leave(i);
        for (int kb = 0; kb < nkb; ++kb, x += kBK) {
          if (!mbar_wait(&bar->empty[s], phase)) {
            ok = false;
            break;
          }
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(&bar->full[s], 2 * kStageBytes);
            const uint32_t dst = smem_u32(smem + s * kStageBytes);
            const uint32_t full = map_to_cta(smem_u32(&bar->full[s]), 0);
            tma_load_pair(dst, &amap, x, arow, full);
            tma_load_pair(dst + kStageA, &bmap, x, brow, full);
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
      uint32_t s = 0, phase = 0, buf = 0, tphase = 1;
      bool ok = true;
      for (int i = 0; i < items && ok; ++i) {
        if (!(ok = listed(i))) break;
        const int nkb = __shfl_sync(0xFFFFFFFFu, slot_of(i)->nkb, 0);
        const uint32_t idesc = __shfl_sync(0xFFFFFFFFu, slot_of(i)->half ? idesc_e4m3(256, 128) : idesc_e4m3(256, 256), 0);
        leave(i);
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&bar->full[s], phase) || !mbar_wait(&bar->tempty[buf], tphase)) {
            ok = false;
            break;
          }
          tcgen05_after_sync();
          if (elect_one()) {
            const uint64_t a = desc0 + s * (kStageBytes / 16), b = a + kStageA / 16;
            const uint32_t d = tmem + buf * kBufCols;
#pragma unroll
            for (int k = 0; k < kBK / 32; ++k)  // 32 bytes further inside the 128-byte swizzled rows
              umma_e4m3<2>(d, a + 2 * k, b + 2 * k, idesc, k > 0);
            umma_commit_pair(&bar->tfull[buf]);
            umma_commit_pair(&bar->empty[s]);
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            phase ^= 1;
          }
          buf ^= 1;
          tphase ^= buf ^ 1;
        }
      }
      if (!ok) report_timeout(p.status);
    } else if (w == 2) {
      // the block's scales: 128 of this CTA's rows of A, 256 (or 2) of B
      const int64_t kblocks = (p.a_cols + kBK - 1) / kBK, nblocks = (p.b_rows + 127) / 128;
      uint32_t it = 0;
      bool ok = true;
      // A scale per row of both: rows of memory, one bulk copy each where 16-byte
      // boundaries allow, instead of 12 copies of 4 bytes a lane (4096 x 4864 x
      // 16384: 235 us against 243).
      const bool a_bulk = p.a_rows % 4 == 0 && (reinterpret_cast<uintptr_t>(p.sa) & 15) == 0;
      const bool b_bulk = kColScales && p.b_rows % 4 == 0 && (reinterpret_cast<uintptr_t>(p.sb) & 15) == 0;
      for (int i = 0; i < items && ok; ++i) {
        if (!(ok = listed(i))) break;
        const TileSlot tl = *slot_of(i);
        leave(i);
        const bool bulk = kColScales && a_bulk && b_bulk && tl.a_row % 4 == 0;
        const uint32_t a_bytes = 4 * (uint32_t)max((int64_t)0, min((int64_t)128, p.a_rows - tl.a_row - 128 * rank));
        const uint32_t b_bytes = 4 * (uint32_t)tl.cols;
        if (bulk) fence_proxy_async_shared();  // another tile's may have come by plain copies
        const int64_t member = p.wgrad || tl.nkb == 0 ? 0 : tl.member;
        const float* pa = p.sa + (int64_t)tl.kb0 * p.a_rows + tl.a_row;
        const float* pb;
        int oa[4], ob[8], nb;  // offsets of this lane's scales; how many of B's exist
#pragma unroll
        for (int i = 0; i < 4; ++i)
          oa[i] = (int)min((int64_t)(128 * rank + lane + 32 * i), p.a_rows - 1 - tl.a_row);
        if constexpr (kColScales) {
          pb = p.sb + (member * kblocks + tl.kb0) * p.b_rows + tl.n0;
          nb = tl.cols;
#pragma unroll
          for (int i = 0; i < 8; ++i) ob[i] = min(lane + 32 * i, nb - 1);
        } else {
          pb = p.sb + (member * nblocks + tl.n0 / 128) * kblocks + tl.kb0;
          nb = (int)min((int64_t)2, nblocks - tl.n0 / 128);
          ob[0] = lane < nb ? lane * (int)kblocks : 0;
        }
        for (int kb = 0; kb < tl.nkb; kb += kScaleBatch, ++it) {
          const uint32_t s = it % kScaleStages;
          if (!mbar_wait(&bar->sempty[s], ((it / kScaleStages) & 1) ^ 1)) {
            ok = false;
            break;
          }
          uint32_t dst = smem_u32(scales + s * kScaleBatch * kScaleFloats) + 4 * lane;
          const int n = min(kScaleBatch, tl.nkb - kb);
          if (bulk) {
            if (lane == 0) {
              mbar_arrive_expect_tx(&bar->sfull[s], n * (a_bytes + b_bytes));
              const float *qa = pa + 128 * rank, *qb = pb;
              for (int j = 0; j < n; ++j) {
                const uint32_t to = dst + 4 * kScaleFloats * j;
                if (a_bytes) bulk_load(to, qa, a_bytes, &bar->sfull[s]);
                bulk_load(to + 512, qb, b_bytes, &bar->sfull[s]);
                qa += p.a_rows;
                qb += p.b_rows;
              }
            }
            __syncwarp();
            pa += n * p.a_rows;
            pb += n * p.b_rows;
            cp_async_arrive(&bar->sfull[s]);
            continue;
          }
          if (kColScales && lane == 0) mbar_arrive(&bar->sfull[s]);
          for (int j = 0; j < n; ++j, dst += 4 * kScaleFloats) {
#pragma unroll
            for (int i = 0; i < 4; ++i) cp_async4(dst + 128 * i, pa + oa[i], true);
            pa += p.a_rows;
            if constexpr (kColScales) {
#pragma unroll
              for (int i = 0; i < 8; ++i) cp_async4(dst + 512 + 128 * i, pb + ob[i], lane + 32 * i < nb);
              pb += p.b_rows;
            } else {
              if (lane < 2) cp_async4(dst + 512, pb + ob[0], lane < nb);
              ++pb;
            }
          }
          cp_async_arrive(&bar->sfull[s]);
        }
      }
      if (!ok) report_timeout(p.status);
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (w == 3) {
      // The tiles, ahead of the other warps: working one out takes about 1000
      // cycles, which in every warp's own loop cost 16384 x 4096 x 2048 in eight
      // members, FP32 out, 165 us against 153.
      for (int i = 0; i < items; ++i) {
        const int t = t0 + i * step;
        Tile tl = Tiles::at(p, first, t < uncut ? t : uncut + (t - uncut) / 2);
        if (t >= uncut) {
          const int right = 128 * ((t - uncut) & 1);
          tl.n0 += right;
          tl.b_row += right;
          tl.cols = max(0, min(128, tl.cols - right));
          if (tl.cols == 0) tl.nkb = 0;
        }
        bool free = false;  // within the time of a tile, which may pass the limit of one wait
        for (int64_t n = 0; n <= p.a_cols >> 26 && !free; ++n)
          free = mbar_wait(&bar->done[i % kTileSlots], ((i / kTileSlots) & 1) ^ 1);
        if (!free) {
          report_timeout(p.status);
          break;
        }
        if (lane == 0) {
          *slot_of(i) = {tl.nkb, tl.kb0, t >= uncut, tl.member, (int)tl.a_row, (int)tl.b_row, (int)tl.n0,
                         (int)tl.out_row, tl.rows, tl.cols, {0, 0}};
          mbar_arrive(&bar->listed[i % kTileSlots]);
        }
        __syncwarp();
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kColScales ? 232 : 240));
    const int q = w & 3, half = (w - 4) >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16) + half * 128;
    const uint32_t tempty0 = map_to_cta(smem_u32(&bar->tempty[0]), 0);
    const uint32_t box = smem_u32(out_stage + (w - 4) * kOutBoxes * kOutBox);
    uint32_t boxes = 0;
    const uint32_t sc = smem_u32(scales);
    const uint32_t sc_row = sc + 4 * (32 * q + (kColScales ? lane >> 2 : lane));
    const uint32_t sc_col = 4 * (128 + (kColScales ? 128 * half + 2 * (lane & 3) : half)) -
                            4 * (32 * q + (kColScales ? lane >> 2 : lane));  // from sc_row
    // The accumulator the next block is in: its barriers and its columns, the
    // other one 8 bytes and 256 columns further or back.
    uint32_t tfull = smem_u32(&bar->tfull[0]), tempty = tempty0, src = lane_base, tphase = 0;
    uint32_t stage = 0, sphase = 0;
    bool ok = true;
    for (int item = 0; item < items && ok; ++item) {
      if (!(ok = listed(item))) break;
      const int nkb = slot_of(item)->nkb;
      uint64_t sum[64];  // pairs of columns
#pragma unroll
      for (int i = 0; i < 64; ++i) sum[i] = 0;
      const bool idle = slot_of(item)->half && half;  // a halved tile has the first half's columns only
      for (int kb = 0; kb < nkb; kb += kScaleBatch) {
        ok = mbar_wait_at(smem_u32(&bar->sfull[stage]), sphase);
        if (!ok) break;
        if (idle) {
          for (int n = min(kScaleBatch, nkb - kb); n > 0 && ok; --n) {
            ok = mbar_wait_at(tfull, tphase);
            if (ok && lane == 0) mbar_arrive_cluster(tempty);
            tphase ^= (tfull >> 3) & 1;
            tfull ^= 8;
            tempty ^= 8;
            src ^= kBufCols;
          }
        } else {
          uint32_t scale = sc_row + stage * (kScaleBatch * kScaleFloats * 4);
          // Kept as small as it can be: instructions beside the sums cost more
          // here than their issue slots (two dozen more made the kernel half as slow
          // again, the hand-over of the scales outside and shorter waits 3 to 8
          // percent faster), as if the loop just fitted an instruction store.
#pragma unroll 1
          for (int n = min(kScaleBatch, nkb - kb); n > 0; --n, scale += 4 * kScaleFloats) {
            float sa[kColScales ? 4 : 1], sb = 0.0f, both = 0.0f;
            if constexpr (kColScales) {
              // four rows of the lane: lane / 4 + 8 i
#pragma unroll
              for (int i = 0; i < 4; ++i) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(sa[i]) : "r"(scale + 32 * i));
            } else {
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(sa[0]) : "r"(scale));
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(sb) : "r"(scale + sc_col));
              both = __fmul_rn(sa[0], sb);
            }
            ok = mbar_wait_at(tfull, tphase);
            if (!ok) break;
            __syncwarp();
            tcgen05_after_sync();
            // One factor for both scales, as long as it is a normal number.  A row
            // where it is not takes them one after the other, the larger first: a
            // block's sum (0, or 2^-18 to 2^25) times both may be a normal number
            // all the same, and then no step leaves their range.  The larger one is
            // multiplied into tensor memory, which keeps this loop small (the same
            // on the registers: 8192 x 5120 x 8192 210.9 us, here 209.7, without
            // the test 208.3).
            if (!kColScales && __any_sync(0xFFFFFFFFu, __float_as_uint(both) - 0x00800000u >= 0x7F000000u)) {
              const float m = fabsf(both);
              const bool own = sa[0] != 0.0f && sb != 0.0f && (m < kSmallestNormal || m > kLargest);
              const float ahead = own ? fmaxf(sa[0], sb) : 1.0f;
              both = own ? fminf(sa[0], sb) : both;
              if (__any_sync(0xFFFFFFFFu, own)) {
#pragma unroll 1
                for (int c = 0; c < 128; c += 16) {
                  uint32_t v[16];
                  tmem_read(src + c, v);
#pragma unroll
                  for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__fmul_rn(__uint_as_float(v[i]), ahead));
                  tmem_write(src + c, v);
                }
              }
            }
#pragma unroll
            for (int c = 0; c < 128; c += kChunk) {
              // once everything is read, the accumulator may be overwritten
              auto release = [&]() {
                if (c != 128 - kChunk) return;
                tcgen05_before_sync();
                if (lane == 0) mbar_arrive_cluster(tempty);
              };
              if constexpr (kColScales) {
                // A column's scale serves the lane's four rows.  Two steps an
                // element are bound by instruction issue, which packed arithmetic
                // halves (4096 x 4864 x 16384: 290 us against 332 with scalar).
                uint32_t u[32], v[32];
                float sb[8][2];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                               : "=f"(sb[j][0]), "=f"(sb[j][1])
                               : "r"(scale + sc_col + 4 * (c + 8 * j)));
                tmem_read_16x256(src + c, u, v);
                release();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const uint64_t s2 = pack2(sb[j][0], sb[j][1]);
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const uint32_t* x = i < 2 ? u + 4 * j + 2 * i : v + 4 * j + 2 * i - 4;
                    uint64_t& to = sum[(c / 8 + j) * 4 + i];
                    to = fma2(mul2(pack2(__uint_as_float(x[0]), __uint_as_float(x[1])), s2), pack2(sa[i], sa[i]), to);
                  }
                }
              } else {
                uint32_t v[kChunk];
                tmem_read(src + c, v);
                release();
#pragma unroll
                for (int i = 0; i < kChunk / 2; ++i)
                  sum[c / 2 + i] = fma2(pack2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])),
                                        pack2(both, both), sum[c / 2 + i]);
              }
            }
            tphase ^= (tfull >> 3) & 1;  // the second of the two is done: the next phase
            tfull ^= 8;
            tempty ^= 8;
            src ^= kBufCols;
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->sempty[stage]);
        stage ^= 1;
        sphase ^= stage ^ 1;
      }
      if (!ok) break;
      const TileSlot tl = *slot_of(item);
      leave(item);
      float acc[128];
#pragma unroll
      for (int i = 0; i < 64; ++i) unpack2(sum[i], acc[2 * i], acc[2 * i + 1]);
      // The 32 rows of this warp go out through shared memory, 128 bytes of
      // each row at a time, stored by TMA while the next tile is summed.  Rows
      // past a member's end, and rows whose pitch TMA cannot take, are written
      // by the warp itself, a row at a time.
      const int row0 = 128 * (int)rank + 32 * q, c0 = 128 * half;
      if (idle || row0 >= tl.rows || c0 >= tl.cols) continue;
      const bool by_tma = p.out_map && row0 + 32 <= tl.rows;
      auto put = [&](int c, auto&& fill) {  // 128 bytes of the rows, from column c of the tile
        if (c >= tl.cols) return;
        const uint32_t src = box + (boxes % kOutBoxes) * kOutBox;
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kOutBoxes - 1) : "memory");
        __syncwarp();
        fill(src);
        ++boxes;
        if (by_tma) {
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) tma_store(&omap, src, tl.n0 + c, tl.out_row + row0);
        } else {
          __syncwarp();
          const int rows = min(32, tl.rows - row0);
          for (int r = 0; r < rows; ++r) {
            uint32_t x;
            asm volatile("ld.shared.u32 %0, [%1];"
                         : "=r"(x)
                         : "r"(src + r * 128 + (((lane >> 2) ^ (r & 7)) * 16) + (lane & 3) * 4)
                         : "memory");
            const int64_t at = (int64_t)(tl.out_row + row0 + r) * p.b_rows + tl.n0 + c;
            if (p.out_bf16) {
              uint16_t* dst = static_cast<uint16_t*>(p.out) + at + 2 * lane;
              if (c + 2 * lane < tl.cols) dst[0] = (uint16_t)x;
              if (c + 2 * lane + 1 < tl.cols) dst[1] = (uint16_t)(x >> 16);
            } else if (c + lane < tl.cols) {
              static_cast<uint32_t*>(p.out)[at + lane] = x;
            }
          }
        }
        if (lane == 0) bulk_commit();  // a group of its own (empty if the warp wrote)
      };
      auto bf16x2 = [](float lo, float hi) {
        uint32_t h;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
        return h;
      };
      // 16-byte places of a row are swizzled by the row, as TMA expects them.
      if constexpr (kColScales) {
        const int r0 = lane >> 2, e = lane & 3;  // the lane's rows r0 + 8 i (r0 & 7 = r0), its two columns of eight
        if (p.out_bf16) {
#pragma unroll
          for (int g = 0; g < 2; ++g)
            put(c0 + 64 * g, [&](uint32_t src) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  sts_u32(src + (r0 + 8 * i) * 128 + ((j ^ r0) * 16) + 4 * e,
                          bf16x2(acc[(8 * g + j) * 8 + 2 * i], acc[(8 * g + j) * 8 + 2 * i + 1]));
            });
        } else {
#pragma unroll
          for (int g = 0; g < 4; ++g)
            put(c0 + 32 * g, [&](uint32_t src) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  sts_v2(src + (r0 + 8 * i) * 128 + (((2 * j + (e >> 1)) ^ r0) * 16) + 8 * (e & 1),
                         __float_as_uint(acc[(4 * g + j) * 8 + 2 * i]), __float_as_uint(acc[(4 * g + j) * 8 + 2 * i + 1]));
            });
        }
      } else if (p.out_bf16) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
          put(c0 + 64 * g, [&](uint32_t src) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float* f = acc + 64 * g + 8 * j;
              sts_v4(src + lane * 128 + ((j ^ (lane & 7)) * 16), bf16x2(f[0], f[1]), bf16x2(f[2], f[3]),
                     bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
            }
          });
      } else {
#pragma unroll
        for (int g = 0; g < 4; ++g)
          put(c0 + 32 * g, [&](uint32_t src) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float* f = acc + 32 * g + 4 * j;
              sts_v4(src + lane * 128 + ((j ^ (lane & 7)) * 16), __float_as_uint(f[0]), __float_as_uint(f[1]),
                     __float_as_uint(f[2]), __float_as_uint(f[3]));
            }
          });
      }
    }
    if (!ok) report_timeout(p.status);
    if (lane == 0) bulk_wait_all();
  }
  tcgen05_before_sync();
  __syncthreads();
  cluster_sync();
  tcgen05_after_sync();
  if (w == 1) tmem_dealloc_pair(tmem, 512);
}

// Which of the two kernels a product runs on.  Up to 32 rows (96 per expert)
// the thin kernel's tiles fit and it is ahead (5120 x 4096 weights, 1 / 16 rows:
// 6.9 / 7.1 us against 22.7 / 19.2; 1100 rows to 16 experts of 4096 x 2048: 38.1
// against 39.0).  Above, the estimated times decide, in us, fitted to both kernels
// at 64 to 1024 rows, N 512 to 8192, K 512 to 8192: a start, then the blocks that
// each CTA or pair sums one after another.  For instance, thin against pair at
// 128 rows and 128 x 128 blocks: N 1024, K 4096 8.2 / 12.1; N 5120, K 4096 17.2 /
// 13.8; N 8192, K 512 7.5 / 5.6.  Of 128 such products (64 to 1024 rows, both
// forms of scales) the rule picks the faster kernel every time.  (All in CUDA
// graphs, several inputs in turn.)
bool thin_is_faster(const Fp8MatmulArgs& a, const LaunchCtx& ctx) {
  const int64_t members = a.offsets ? a.experts : 1;
  const int64_t rows = a.wgrad ? a.a_rows : (a.a_rows + members - 1) / members;
  if (rows <= (members > 1 ? 96 : 32)) return true;
  const int64_t k = a.wgrad ? (a.a_cols + members - 1) / members : a.a_cols;
  const double kb = (double)((k + kBK - 1) / kBK);
  const int64_t pair_tiles = members * ((rows + 255) / 256) * ((a.b_rows + 255) / 256);
  const int64_t pairs = ctx.num_sms / 2, over = pair_tiles % pairs;
  const double last = over == 0 ? 0.0 : 2 * over <= pairs ? 0.65 : 1.0;  // of a turn: halved tiles
  const double pair = 4.5 + (pair_tiles / pairs + last) * kb * (a.b_block_rows == 1 ? 0.50 : 0.38) +
                      (a.b_rows * (a.out_bf16 ? 2 : 4) % 16 ? 2.5 : 0.0);  // rows written by the warps
  const ThinPlan t = thin_plan(a, ctx);
  const int64_t ctas = t.tiles * t.split, turns = (ctas + 2 * ctx.num_sms - 1) / (2 * ctx.num_sms);
  const double block = ctas > ctx.num_sms ? 0.6 : 0.45;  // two CTAs of an SM slow each other
  const double thin = 4.5 + (t.split > 1 ? 2.0 : 0.0) + turns * kb / t.split * block;
  return thin < pair;
}

}  // namespace
}  // namespace fp8

cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, const LaunchCtx& ctx) {
  using namespace fp8;
  if (a.a_rows == 0 || a.b_rows == 0) return cudaSuccess;
  const int64_t out_rows = a.wgrad ? a.a_rows * a.experts : a.a_rows;
  if (a.a_cols == 0)
    return cudaMemsetAsync(a.out, 0, (size_t)out_rows * a.b_rows * (a.out_bf16 ? 2 : 4), ctx.stream);
  MatmulKernelArgs p = {};
  p.sa = a.sa;
  p.sb = a.sb;
  p.a_rows = a.a_rows;
  p.a_cols = a.a_cols;
  p.b_rows = a.b_rows;
  p.experts = a.experts;
  p.wgrad = a.wgrad;
  p.offsets = a.offsets;
  p.out = a.out;
  p.out_bf16 = a.out_bf16;
  p.status = ctx.status;
  if (thin_is_faster(a, ctx)) return launch_matmul_thin(a, p, ctx);
  CUtensorMap amap, bmap, omap = {};
  cudaError_t e = make_fp8_tensor_map(&amap, a.a, a.a_rows, a.a_cols, 128);
  if (e != cudaSuccess) return e;
  e = make_fp8_tensor_map(&bmap, a.b, a.wgrad ? a.b_rows : a.b_rows * a.experts, a.a_cols, 128);
  if (e != cudaSuccess) return e;
  // TMA writes the output where its rows start on 16 bytes.
  p.out_map = a.b_rows * (a.out_bf16 ? 2 : 4) % 16 == 0;
  if (p.out_map && (e = make_matmul_out_map(&omap, a.out, a.out_bf16, out_rows, a.b_rows)) != cudaSuccess) return e;
  // No more tiles than this, whatever the offsets.
  const int64_t tn = (a.b_rows + 255) / 256, tm = (a.a_rows + 255) / 256;
  const int64_t tiles = tn * (a.wgrad ? tm * a.experts : tm + (a.offsets ? a.experts : 0));
  const unsigned pairs = (unsigned)(2 * tiles < ctx.num_sms / 2 ? 2 * tiles : ctx.num_sms / 2);  // (halves)
  const auto kernel = a.b_block_rows == 1 ? matmul_pair_kernel<true> : matmul_pair_kernel<false>;
  static std::atomic<uint64_t> allowed[2];
  e = allow_smem(reinterpret_cast<const void*>(kernel), kSmemBytes, allowed[a.b_block_rows == 1]);
  if (e != cudaSuccess) return e;
  void* args[] = {&amap, &bmap, &omap, &p};
  return launch_dependent(reinterpret_cast<const void*>(kernel), dim3(2 * pairs), dim3(kThreads), kSmemBytes, ctx.stream, args);
}

}  // namespace nvfp4
