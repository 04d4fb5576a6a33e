// expert_mlp.cu -- a layer of gated experts over 4-bit weights for a few
// tokens:
//     y[t] = sum_j gates[t][j] Wd[e] (silu(Wg[e] x[t]) * (Wu[e] x[t])),   e = ids[t][j].
//
// With a few rows an expert the time is that of reading its weights once, and
// unpacking them to multiply in 16 bits costs more instructions than the SMs can
// issue meanwhile (about two a weight; 64 tokens, 4 of 32 experts of 4096 x 1536: 135
// us, where reading takes 51).  So the tensor cores take the weights as they are
// (tcgen05 block_scale), and the activations become 4 bits too: as the sum of
// kTerms 4-bit operands.
//
// Terms.  A block (16 or 32 elements, as the weights') has one scale s, at which
// its largest element is at most 6 (NVFP4: the next E4M3 number above a sixth of it,
// MXFP4: the next power of two), and eight rows of E2M1 codes, counting in s, s / 4, s /
// 32, s / 256, ...: a code of the first is off by at most s, which is 4 of the next
// unit; from then on codes are off by at most half a unit, which is 4 of the next
// again.  Eight terms leave s 2^-21, which is 2^-23.4 (NVFP4) or 2^-22.5 (MXFP4) of the
// block's largest element, about what the FP32 sums lose: a BF16 element keeps all of
// its own bits down to 2^-14 of its block's largest.  (Six left 2^-17.4 and took 2 to
// 3 % less time.)  Every step but the choice of codes is exact in FP32, and the rows of a token are
// added with their ratios after the product.  They are rows beside the others: N = 8
// tokens, where few rows leave an MMA's columns empty anyway.
// E4M3 scales span 17 powers of two; they count in units of their row, so that a
// row's small blocks lose nothing until 2^-39 of its largest.  The unit comes from
// the row's largest element, which of a hidden row is not known before all of its
// tiles are: NVFP4 keeps the hidden rows in FP32 and cuts them in a launch of their
// own.  (A unit from a bound, |g|, |u| <= amax sum|x|, would spare the launch but
// hold h to 2^-39 of a number that may be any multiple of it.)  MXFP4's powers
// of two need no unit, and its hidden rows are cut where they are made.
//
// Four launches (NVFP4 five): slots sorted by expert and x into terms; gate and up
// products with SiLU; (NVFP4) the hidden rows into terms; down product, weighted by
// the gates; the slots of a token added in order.  The products are fp4_matmul_thin.cu's:
// 128 weight rows on the tensor-memory lanes (64 gate and 64 up rows) by kTok
// tokens' terms, the contracted dimension of a tile split over a cluster where
// there are few tiles; partial results travel with their terms already added.
//
// Measured: 13 tokens, 4 of 16 experts of 2720 x 1184 (MXFP4) 27.8 us, where reading
// the weights takes 15.5; 64 tokens, 4 of 32 experts of 4096 x 1536 (NVFP4) 77 us of
// 51 (72 with six terms and hidden rows that were cut tile by tile).  Weights and scales
// come at 5.9 TB/s while they come; the rest are steps that wait for one another:
// about 7 us until x's terms are there (the first three stages of weights of every
// CTA are read meanwhile), the hidden rows' way from one product to the next, and
// 4 for the join.  Not kept, as the time stayed or grew: the next weights, or the
// next product's, or the next tile's scales fetched into L2 ahead; two stages of
// scales a warp.
#include "expert_mlp.cuh"

namespace nvfp4 {
namespace fp4 {
namespace {

// What the launches hand to each other, in the workspace.
struct Rows {
  uint8_t* codes;   // [slots * kTerms][width / 2]: sorted slot, term
  uint8_t* scales;  // [segments][scale tiles of the width][512]: rows of a segment as in Format's tiles
  float* unit;      // [slots] NVFP4: what a scale of 1 stands for in term 0
};
struct Plan {
  int32_t* counts;       // segments, sorted slots
  int4* table;           // [segments] expert, first sorted slot, slots
  int32_t* slot_of_row;  // [slots] slot of a sorted one
  int32_t* scale_row;    // [slots] where a sorted one's scales begin: segment * kScaleRows + row
};

// ---------------------------------------------------------------------------
// Slots by expert, and x into terms
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 256, kPrepWarps = kPrepThreads / 32;
constexpr int kPrepPart = 128 * kPrepWarps;  // elements of a CTA
constexpr int kScaleRows = 128;              // of a segment's scale tiles

struct PrepArgs {
  const uint16_t* x;
  const int32_t* ids;
  int slots, topk, experts, width, tok;
  Rows x_rows;
  float* h_unit;
  Plan plan;
};

// Slots by expert, by all threads of a CTA: how many chose each expert before e
// (row0[e], and how many segments they make, seg0[e]; e up to `experts`).  ids:
// those outside the range become -1.  Ends with a barrier.
__device__ __forceinline__ void group_slots(const int32_t* from, int slots, int experts, int tok, int* ids, int* row0,
                                            int* seg0, int threads) {
  const int tid = threadIdx.x, lane = tid & 31;
  for (int e = tid; e <= experts; e += threads) row0[e] = 0;
  for (int s = tid; s < slots; s += threads) {
    const int e = __ldcg(&from[s]);
    ids[s] = e >= 0 && e < experts ? e : -1;
  }
  __syncthreads();
  for (int s = tid; s < slots; s += threads)
    if (ids[s] >= 0) atomicAdd(&row0[ids[s]], 1);
  __syncthreads();
  if (tid < 32) {
    int rows = 0, segs = 0;
    for (int base = 0; base < experts; base += 32) {
      const int e = base + lane, n = e < experts ? row0[e] : 0, s = (n + tok - 1) / tok;
      int rn = n, rs = s;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int un = __shfl_up_sync(0xFFFFFFFFu, rn, d), us = __shfl_up_sync(0xFFFFFFFFu, rs, d);
        if (lane >= d) rn += un, rs += us;
      }
      if (e < experts) row0[e] = rows + rn - n, seg0[e] = segs + rs - s;
      rows += __shfl_sync(0xFFFFFFFFu, rn, 31);
      segs += __shfl_sync(0xFFFFFFFFu, rs, 31);
    }
    if (lane == 0) row0[experts] = rows, seg0[experts] = segs;
  }
  __syncthreads();
}

template <int kBlock>
__global__ void __launch_bounds__(kPrepThreads) prepare_kernel(const __grid_constant__ PrepArgs p) {
  extern __shared__ int lists[];
  int* ids = lists;                      // [slots]
  int* row0 = ids + p.slots;             // [experts + 1] first sorted slot
  int* seg0 = row0 + p.experts + 1;      // [experts + 1] first segment
  __shared__ float largest[kPrepWarps];
  __shared__ int2 place[kMaxTopk];  // of a choice: its sorted slot (-1: dropped), and the row of its first scales
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int parts = (p.width + kPrepPart - 1) / kPrepPart;
  const int token = blockIdx.x / parts, part = blockIdx.x % parts;
  // (first the wait: the next kernel reads what precedes this one ahead of its own)
  grid_dependency_wait();
  grid_launch_dependents();
  // The row's largest finite element.
  const uint16_t* row = p.x + (int64_t)token * p.width;
  float m = 0.0f;
#pragma unroll 2
  for (int k = 8 * tid; k < p.width; k += 8 * kPrepThreads) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + k);
    const float v[8] = {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y),
                        bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w)};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = fabsf(v[i]);
      if (a <= kFltMax) m = fmaxf(m, a);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  if (lane == 0) largest[w] = m;
  group_slots(p.ids, p.slots, p.experts, p.tok, ids, row0, seg0, kPrepThreads);
  m = largest[0];
#pragma unroll
  for (int i = 1; i < kPrepWarps; ++i) m = fmaxf(m, largest[i]);
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    for (int e = tid; e < p.experts; e += kPrepThreads)
      for (int r = row0[e], i = seg0[e]; r < row0[e + 1]; r += p.tok, ++i)
        p.plan.table[i] = make_int4(e, r, min(p.tok, row0[e + 1] - r), 0);
    if (tid == 0) p.plan.counts[0] = seg0[p.experts], p.plan.counts[1] = row0[p.experts];
  }
  // This CTA's share of the token's choices: how many earlier slots chose the same expert.
  for (int j = blockIdx.y + w * gridDim.y; j < p.topk; j += kPrepWarps * gridDim.y) {
    const int s = token * p.topk + j, e = ids[s];  // (a dropped choice counts others that were dropped)
    int before = 0;
    for (int i = lane; i < s; i += 32) before += ids[i] == e;
    before = __reduce_add_sync(0xFFFFFFFFu, before);
    if (lane == 0) {
      const int seg = before / p.tok;
      place[j] = e < 0 ? make_int2(-1, 0) : make_int2(row0[e] + before, (seg0[e] + seg) * kScaleRows + (before - seg * p.tok) * kTerms);
    }
  }
  // Terms of 128 elements a warp, the last ones padded to a step of 64 with zeros.
  const float unit = kBlock == 16 ? unit_of(m) : 1.0f;
  const int64_t k = (int64_t)part * kPrepPart + 128 * w + 4 * lane;
  const int64_t tiles = (p.width + 4 * kBlock - 1) / (4 * kBlock), row_bytes = p.width / 2;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (k < p.width) {
    const uint2 u = *reinterpret_cast<const uint2*>(row + k);
    v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
  }
  uint16_t codes[kTerms];
  const uint32_t scale = to_terms<kBlock>(v, unit, [&](int i, uint16_t c) { codes[i] = c; });
  __syncthreads();
  // They go to the rows of those choices.
  for (int j = blockIdx.y; j < p.topk; j += gridDim.y) {
    const int r = place[j].x, n0 = place[j].y % kScaleRows, seg = place[j].y / kScaleRows;
    if (r < 0) continue;
    if (part == 0 && tid == 0) {
      p.plan.slot_of_row[r] = token * p.topk + j;
      p.plan.scale_row[r] = place[j].y;
      p.x_rows.unit[r] = unit;
      if (kBlock == 32) p.h_unit[r] = 1.0f;
    }
    if (k < p.width)
#pragma unroll
      for (int i = 0; i < kTerms; ++i)
        *reinterpret_cast<uint16_t*>(p.x_rows.codes + ((int64_t)r * kTerms + i) * row_bytes + k / 2) = codes[i];
    if (k < (p.width + 63) / 64 * 64)
      put_scale<kBlock>(p.x_rows.scales + seg * tiles * kScaleTile, n0, k, scale);
  }
}

// NVFP4: the hidden rows into terms, a CTA kPrepPart elements of one.
struct CutArgs {
  const float* hidden;  // [sorted slot][width]
  int width;
  Rows rows;
  Plan plan;
};

__global__ void __launch_bounds__(kPrepThreads) cut_hidden_kernel(const __grid_constant__ CutArgs p) {
  __shared__ float largest[kPrepWarps];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int parts = (p.width + kPrepPart - 1) / kPrepPart;
  const int r = blockIdx.x / parts, part = blockIdx.x % parts;
  // (first the wait: the next kernel reads what precedes this one ahead of its own)
  grid_dependency_wait();
  grid_launch_dependents();
  if (r >= __ldcg(&p.plan.counts[1])) return;
  const float* row = p.hidden + (int64_t)r * p.width;
  const int64_t k = (int64_t)part * kPrepPart + 128 * w + 4 * lane;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (k < p.width) {
    const float4 u = __ldcg(reinterpret_cast<const float4*>(row + k));
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  }
  float m = 0.0f;  // the row's largest finite element
#pragma unroll 2
  for (int i = 4 * tid; i < p.width; i += 4 * kPrepThreads) {
    const float4 u = __ldcg(reinterpret_cast<const float4*>(row + i));
    m = fmaxf(fmaxf(m, finite_magnitude(u.x)), fmaxf(finite_magnitude(u.y), fmaxf(finite_magnitude(u.z), finite_magnitude(u.w))));
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  if (lane == 0) largest[w] = m;
  __syncthreads();
  m = largest[0];
#pragma unroll
  for (int i = 1; i < kPrepWarps; ++i) m = fmaxf(m, largest[i]);
  const float unit = unit_of(m);
  if (part == 0 && tid == 0) p.rows.unit[r] = unit;
  const int64_t tiles = (p.width + 63) / 64, row_bytes = p.width / 2;
  const int at = __ldcg(&p.plan.scale_row[r]);
  const uint32_t scale = to_terms<16>(v, unit, [&](int i, uint16_t codes) {
    if (k < p.width) *reinterpret_cast<uint16_t*>(p.rows.codes + ((int64_t)r * kTerms + i) * row_bytes + k / 2) = codes;
  });
  if (k < tiles * 64)  // (the last ones padded to a step of 64 with zeros)
    put_scale<16>(p.rows.scales + at / kScaleRows * tiles * kScaleTile, at % kScaleRows, k, scale);
}

// ---------------------------------------------------------------------------
// The products
// ---------------------------------------------------------------------------
constexpr int kOutWarps = 4;
constexpr int kThreads = 32 * (kOutWarps + 2 + kScaleWarps);
constexpr int kWeights = 128;  // weight rows of a tile
constexpr int kMaxStages = 8;

struct MlpKernelArgs {
  const uint8_t* scale;  // of the weights, compact
  const float* amax;
  int amax_per_expert;
  int experts, rows, width;  // weight rows of an expert, contracted dimension
  int inner;                 // up: gate rows of an expert
  const int32_t* ids;        // up
  int slots;
  Plan plan;
  Rows in;                   // the activations' terms
  float* hidden;             // up, NVFP4: the hidden rows, [sorted slot][inner]
  Rows out;                  // up, MXFP4: the hidden rows' terms
  const float* gates;        // down
  float* parts;              // down: [slots][rows]
  int tiles;                 // of an expert's weights
  unsigned* status;
};

struct Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2];
  uint64_t got, taken;  // the cluster's partial results: all are here / all have been added
  uint32_t tmem;
  uint32_t pad;
};

template <int kTok, int kBlock>
struct Layout {
  using F = Format<kBlock>;
  static constexpr int kBN = kTok * kTerms;
  static constexpr int kWCodes = kWeights * kStageRow;
  static constexpr int kCodes = kWCodes + kBN * kStageRow;
  static constexpr int kStageBytes = kCodes + 2 * F::kScaleBytes;
  static constexpr int kCols = 2 * kBN + 2 * F::kCols;
  static constexpr int kTmemCols = kCols <= 64 ? 64 : kCols <= 128 ? 128 : 256;
  static_assert(kBN % 16 == 0 && kCols <= 256 && kStageBytes % 1024 == 0, "tensor memory of two CTAs; swizzled operands");
  static constexpr int kResultBytes = kTok * kWeights * 4;  // a tile's results
  static __host__ __device__ int own(int split) { return (kTok + split - 1) / split; }  // tokens a CTA of a cluster joins
  static __host__ __device__ int share_bytes(int split) {
    return split == 1 ? 0 : split * own(split) * kWeights * 4;
  }
  static int rest(int split, int slots, int experts) {
    return kResultBytes + share_bytes(split) + (int)sizeof(Barriers) + 4 * (2 * (experts + 1) + slots);
  }
};

template <bool kDown, int kTok, int kBlock>
__global__ void __launch_bounds__(kThreads, 2)
expert_product_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                      const __grid_constant__ MlpKernelArgs p, int stages, int split) {
  using L = Layout<kTok, kBlock>;
  using F = Format<kBlock>;
  constexpr int kBN = L::kBN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* results = reinterpret_cast<float*>(smem + stages * L::kStageBytes);  // [token][row]
  float* shares = results + L::kResultBytes / 4;                              // [rank][own token][row]
  Barriers* bar = reinterpret_cast<Barriers*>(shares + L::share_bytes(split) / 4);
  int* row0 = reinterpret_cast<int*>(bar + 1);  // up: as group_slots gives them
  int* seg0 = row0 + p.experts + 1;
  int* ids = seg0 + p.experts + 1;
  const int own = L::own(split);
  const int w = warp_index(), lane = threadIdx.x & 31;
  const int rank = split > 1 ? (int)cluster_rank() : 0;

  if (w == kOutWarps) {
    if (lane == 0) {
      for (int i = 0; i < stages; ++i) {
        mbar_init(&bar->full[i], 2);
        mbar_init(&bar->empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar->tfull[i], 1);
        mbar_init(&bar->tempty[i], kOutWarps);
      }
      mbar_init(&bar->got, 1);
      mbar_init(&bar->taken, kOutWarps * split);
      fence_mbar_init();
      tma_prefetch_desc(&wmap);
      tma_prefetch_desc(&xmap);
    }
  } else if (w == kOutWarps + 1) {
    tmem_alloc(&bar->tmem, L::kTmemCols);
  }
  __syncwarp();
  if (split > 1) cluster_arrive();  // (the barriers are set up)
  // Ahead of the wait for the kernel before: what that one does not write, as it
  // waited for its own predecessor before it let this one begin.
  int segs;
  if constexpr (kDown)
    segs = __ldcg(p.plan.counts);  // (two kernels back or more; from L2, as this memory served earlier calls)
  else
    group_slots(p.ids, p.slots, p.experts, kTok, ids, row0, seg0, kThreads), segs = seg0[p.experts];
  tcgen05_before_sync();
  __syncthreads();
  if (split > 1) cluster_wait();
  tcgen05_after_sync();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, bar->tmem, 0);
  const int lg_split = __ffs(split) - 1;
  const int t0 = blockIdx.x >> lg_split, step = gridDim.x >> lg_split;
  const int tiles = __shfl_sync(0xFFFFFFFFu, segs, 0) * p.tiles;
  const int nkb = (p.width + kStageK - 1) / kStageK;
  const int full_stages = p.width / kStageK, last_steps = (p.width % kStageK + 63) / 64;  // of 64 elements
  const int kb0 = (nkb * rank) >> lg_split, kb1 = (nkb * (rank + 1)) >> lg_split;
  bool ok = true;
  // A segment: its expert, first sorted slot and slots.
  auto segment_of = [&](int i) -> int4 {
    if constexpr (kDown) return __ldcg(&p.plan.table[i]);
    int lo = 0, hi = p.experts;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (seg0[mid] <= i) lo = mid; else hi = mid;
    }
    const int r = row0[lo] + (i - seg0[lo]) * kTok;
    return make_int4(lo, r, min(kTok, row0[lo + 1] - r), 0);
  };
  // First row of a tile of an expert, in the stack of all experts' weights.
  constexpr int kTileRows = kDown ? kWeights : kWeights / 2;
  auto first_row = [&](int expert, int tile) { return expert * p.rows + tile * kTileRows; };
  // (The copying warp and those of the weights' scales wait when the ring is full.
  // No warp lets the next kernel begin ahead of its wait: the down product reads the
  // plan ahead of its own.)
  if (w < kOutWarps || w == kOutWarps + 1) {
    grid_dependency_wait();
    grid_launch_dependents();
  }

  if (w == kOutWarps) {
    const int scale_tiles = (p.width + 4 * kBlock - 1) / (4 * kBlock);
    // A tile's places, worked out once for all of its stages: that takes as long as a stage's copies.
    struct Place {
      int row, x_row;
      const uint8_t* x_scales;
    };
    auto place_of = [&](int t) {
      const int i = t / p.tiles, tile = t - i * p.tiles;
      const int4 seg = segment_of(i);
      return Place{first_row(seg.x, tile), seg.y * kTerms,
                   p.in.scales + (int64_t)i * scale_tiles * kScaleTile};
    };
    auto scale_bytes = [&](int kb) { return (uint32_t)min(F::kTiles, scale_tiles - kb * F::kTiles) * kScaleTile; };
    auto weights = [&](const Place& at, int kb, uint32_t s) {
      if (elect_one()) {
        const uint32_t dst = smem_u32(smem + s * L::kStageBytes), full = smem_u32(&bar->full[s]);
        mbar_arrive_expect_tx(&bar->full[s], L::kCodes + scale_bytes(kb));
        tma_load(dst, &wmap, kb * kStageRow, at.row, full);
        if (!kDown) tma_load(dst + L::kWCodes / 2, &wmap, kb * kStageRow, at.row + p.inner, full);
      }
      __syncwarp();
    };
    auto activations = [&](const Place& at, int kb, uint32_t s) {
      if (elect_one()) {
        const uint32_t dst = smem_u32(smem + s * L::kStageBytes), full = smem_u32(&bar->full[s]);
        tma_load(dst + L::kWCodes, &xmap, kb * kStageRow, at.x_row, full);
        bulk_load(dst + L::kCodes + F::kScaleBytes, at.x_scales + kb * F::kScaleBytes, scale_bytes(kb),
                  &bar->full[s]);
      }
      __syncwarp();
    };
    // The first stages' weights ahead of the kernel before, whose results the activations are.
    int early = 0;
    for (int t = t0; t < tiles && early < stages; t += step) {
      const Place at = place_of(t);
      for (int kb = kb0; kb < kb1 && early < stages; ++kb, ++early) weights(at, kb, early);
    }
    grid_dependency_wait();
    grid_launch_dependents();
    uint32_t s = 0, phase = 1;
    int sent = 0;
    for (int t = t0; t < tiles && ok; t += step) {
      const Place at = place_of(t);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (sent >= early) {
          if (!mbar_wait(&bar->empty[s], phase)) {
            ok = false;
            break;
          }
          weights(at, kb, s);
        }
        activations(at, kb, s);
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
      for (int i = sent < stages ? 0 : sent - stages; i < sent; ++i) mbar_wait(&bar->full[i % stages], (i / stages) & 1);
    }
  } else if (w == kOutWarps + 1) {
    constexpr uint32_t kIdesc = F::idesc(kWeights, kBN);
    const uint64_t desc0 = operand_desc(smem_u32(smem));
    const uint64_t sdesc0 = scale_desc(smem_u32(smem) + L::kCodes);
    const uint32_t sw = tmem + 2 * kBN, sx = sw + F::kCols;
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
        const uint64_t a = desc0 + s * (L::kStageBytes / 16), b = a + L::kWCodes / 16;
        const uint64_t ds = sdesc0 + s * (L::kStageBytes / 16);
        const uint32_t add = kb > kb0;
        auto copy = [&](int j) {
          scales_to_tmem<1>(sw + 4 * j, ds + j * (kScaleTile / 16));
          scales_to_tmem<1>(sx + 4 * j, ds + (F::kScaleBytes + j * kScaleTile) / 16);
        };
        auto multiply = [&](int k) {
          umma_fp4<1, kBlock>(tmem + buf * kBN, a + 2 * k, b + 2 * k, kIdesc | F::half(k), sw + F::col(k), sx + F::col(k),
                              k > 0 ? 1 : add);
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
    bool waited = false;
    stale_lines_gone();
    if (mine < active) {
      uint32_t s = 0, phase = 1, it = 0;
      const CompactScales<kBlock> scales(p.scale, p.width, (int64_t)p.experts * p.rows);
      for (int t = t0; t < tiles && ok; t += step) {
        const int r0 = first_row(segment_of(t / p.tiles).x, t % p.tiles);
        for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
          if ((it & (active - 1)) == (uint32_t)mine) {
            uint32_t v[4][F::kTiles];
            const int64_t gap = kDown ? 0 : p.inner - kWeights / 2;
            scales.read(r0, kWeights, kb, v, gap);
            if (!waited && it >= (uint32_t)stages) {
              grid_dependency_wait();
              grid_launch_dependents();
              waited = true;
            }
            ok = mbar_wait(&bar->empty[s], phase);
            if (ok) {
              scales.write(smem_u32(smem + s * L::kStageBytes) + L::kCodes, v);
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
    if (!waited) {
      grid_dependency_wait();
      grid_launch_dependents();
    }
  } else {
    const uint32_t lane_base = tmem + ((uint32_t)(32 * w) << 16);
    const int r = 32 * w + lane;
    uint32_t buf = 0, tphase = 0, round = 0;
    for (int t = t0; t < tiles && ok; t += step) {
      const int tile = t % p.tiles, segment = t / p.tiles;
      const int4 seg = segment_of(segment);
      const float factor = kBlock == 16 ? __fdiv_rn(p.amax[p.amax_per_expert ? seg.x : 0], 2688.0f) : 1.0f;
      // this CTA's tokens of the segment, all or its share
      const int first = split == 1 ? 0 : rank * own, mine = max(0, min(split == 1 ? kTok : own, seg.z - first));
      // what lane n needs to know of token first + n, ahead of the sums
      float unit = 0.0f, gate_of = 0.0f;  // of its terms; down: its gate
      int slot = 0;
      if (lane < mine) {
        const int row = seg.y + first + lane;
        unit = __fmul_rn(p.in.unit[row], factor);
        if constexpr (kDown) {
          slot = p.plan.slot_of_row[row];
          gate_of = p.gates[slot];
        }
      }
      ok = mbar_wait(&bar->tfull[buf], tphase);
      if (ok && split > 1) ok = mbar_wait_cluster(&bar->taken, (round & 1) ^ 1, p.status);
      if (!(ok = together(ok))) break;
      tcgen05_after_sync();
      if (split > 1 && w == 0 && lane == 0) mbar_arrive_expect_tx(&bar->got, split * kWeights * 4 * mine);
      // A token's terms added, the smallest first.
#pragma unroll 1
      for (int n = 0; n < seg.z; n += 2) {
        uint32_t v[16];
        tmem_read(lane_base + buf * kBN + n * kTerms, v);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float sum = add_terms(v + kTerms * h);
          const int token = n + h;
          if (token >= seg.z) break;
          if (split == 1) {
            results[token * kWeights + r] = sum;
          } else {
            const int to = token / own;
            store_async(map_to_cta(smem_u32(shares + (rank * own + token - to * own) * kWeights + r), to), sum,
                        map_to_cta(smem_u32(&bar->got), to));
          }
        }
      }
      tcgen05_before_sync();  // everything is read
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->tempty[buf]);
      if (split > 1) {
        ok = together(mbar_wait_cluster(&bar->got, round & 1, p.status));
        if (!ok) break;
        for (int n = 0; n < mine; ++n) {
          float sum = 0.0f;
          for (int i = 0; i < split; ++i) sum = __fadd_rn(sum, shares[(i * own + n) * kWeights + r]);
          results[n * kWeights + r] = sum;
        }
        __syncwarp();
        if (t + step < tiles && lane < split)
          mbar_arrive_cluster_release(map_to_cta(smem_u32(&bar->taken), lane));
        ++round;
      }
      // results[n]: the sums of token first + n of the segment
      if constexpr (kDown) {
        const int o = kWeights * tile + r;
        for (int n = 0; n < mine; ++n) {
          const float v = __fmul_rn(results[n * kWeights + r], __shfl_sync(0xFFFFFFFFu, unit, n));
          const float weighted = __fmul_rn(v, __shfl_sync(0xFFFFFFFFu, gate_of, n));
          const int64_t to = (int64_t)__shfl_sync(0xFFFFFFFFu, slot, n) * p.rows + o;
          if (o < p.rows) p.parts[to] = weighted;
        }
      } else {
        together(true);  // gate and up sums come from different warps
        // 16 lanes take a token's 64 hidden values, four each
        const int64_t f = kTileRows * (int64_t)tile + 4 * (lane & 15);
        const int64_t out_tiles = (p.inner + 4 * kBlock - 1) / (4 * kBlock);
        for (int n = 2 * w + (lane >> 4); n - (lane >> 4) < mine; n += 2 * kOutWarps) {
          const bool there = n < mine;
          const int row = seg.y + first + n;
          const float x_unit = __shfl_sync(0xFFFFFFFFu, unit, n & 31);
          float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          if (there && f < p.inner) {
            const float4 a = *reinterpret_cast<const float4*>(results + n * kWeights + 4 * (lane & 15));
            const float4 b = *reinterpret_cast<const float4*>(results + n * kWeights + 64 + 4 * (lane & 15));
            const float gate[4] = {a.x, a.y, a.z, a.w}, up[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float z = __fmul_rn(gate[i], x_unit);
              v[i] = __fmul_rn(__fdiv_rn(z, __fadd_rn(1.0f, expf(-z))), __fmul_rn(up[i], x_unit));
            }
          }
          if constexpr (kBlock == 16) {
            if (there && f < p.inner)
              *reinterpret_cast<float4*>(p.hidden + (int64_t)row * p.inner + f) = make_float4(v[0], v[1], v[2], v[3]);
          } else {
            uint8_t* codes_at = p.out.codes + (int64_t)row * kTerms * (p.inner / 2) + f / 2;
            const uint32_t scale = to_terms<kBlock>(v, 1.0f, [&](int i, uint16_t codes) {
              if (there && f < p.inner) *reinterpret_cast<uint16_t*>(codes_at + (int64_t)i * (p.inner / 2)) = codes;
            });
            if (there)
              put_scale<kBlock>(p.out.scales + segment * out_tiles * kScaleTile, (first + n) * kTerms, f, scale);
          }
        }
        together(true);  // the results may be overwritten
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

// y[t] = the sum of a token's weighted results in the order of its choices.
__global__ void __launch_bounds__(256) join_slots_kernel(const float* parts, const int32_t* ids, int topk,
                                                         int experts, int rows, int tokens, uint16_t* y) {
  grid_begin();
  const int per = rows / 4;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < tokens * per; i += gridDim.x * 256) {
    const int token = i / per, at = 4 * (i % per);
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int j0 = 0; j0 < topk; j0 += 4) {
      float4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (j0 + j >= topk) continue;
        const int slot = token * topk + j0 + j, e = ids[slot];
        if (e >= 0 && e < experts) v[j] = __ldcg(reinterpret_cast<const float4*>(parts + (int64_t)slot * rows + at));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        sum = make_float4(__fadd_rn(sum.x, v[j].x), __fadd_rn(sum.y, v[j].y), __fadd_rn(sum.z, v[j].z),
                          __fadd_rn(sum.w, v[j].w));
    }
    uint32_t lo, hi;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(sum.y), "f"(sum.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(sum.w), "f"(sum.z));
    *reinterpret_cast<uint2*>(y + (int64_t)token * rows + at) = make_uint2(lo, hi);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// Tokens of a segment: more cost columns that few experts fill, fewer read the
// weights of a popular expert again.  Fourteen are the most whose columns fit twice into
// half of the tensor memory, beside the scales.  Eight where experts have four on average
// or fewer (13 tokens, 4 of 16 experts of 2720 x 1184: 27.8 us against 31.0 with
// fourteen); with eight on average there is hardly a difference (64 tokens, 4 of 32
// experts of 4096 x 1536: 77.6 with eight, 77.0).
int tokens_per_segment(int64_t tokens, int64_t slots, int64_t experts) {
  return tokens <= 2 ? 2 : tokens <= 8 || slots <= 4 * experts ? 8 : 14;
}
int64_t most_segments(const ExpertMlpArgs& a) {
  const int64_t slots = a.tokens * a.topk, used = slots < a.experts ? slots : a.experts;
  return used + slots / tokens_per_segment(a.tokens, slots, a.experts);
}

// The workspace, cut into its parts.
struct Workspace {
  Rows x, h;
  float* hidden;
  Plan plan;
  float* parts;
  size_t bytes;
};
Workspace cut(const ExpertMlpArgs& a) {
  Workspace ws = {};
  uint8_t* at = static_cast<uint8_t*>(a.workspace);
  size_t used = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* p = at + used;
    used += (size_t)((bytes + 127) / 128 * 128);
    return p;
  };
  const int64_t slots = a.tokens * a.topk, segs = most_segments(a), per = 4 * a.block;
  ws.x.codes = take(slots * kTerms * (a.hidden / 2));
  ws.x.scales = take(segs * ((a.hidden + per - 1) / per) * kScaleTile);
  ws.x.unit = reinterpret_cast<float*>(take(4 * slots));
  ws.h.codes = take(slots * kTerms * (a.inner / 2));
  ws.h.scales = take(segs * ((a.inner + per - 1) / per) * kScaleTile);
  ws.h.unit = reinterpret_cast<float*>(take(4 * slots));
  ws.hidden = reinterpret_cast<float*>(take(a.block == 16 ? 4 * slots * a.inner : 0));
  ws.plan.counts = reinterpret_cast<int32_t*>(take(8));
  ws.plan.table = reinterpret_cast<int4*>(take(16 * segs));
  ws.plan.slot_of_row = reinterpret_cast<int32_t*>(take(4 * slots));
  ws.plan.scale_row = reinterpret_cast<int32_t*>(take(4 * slots));
  ws.parts = reinterpret_cast<float*>(take(4 * slots * a.hidden));
  ws.bytes = used;
  return ws;
}

template <bool kDown, int kTok, int kBlock>
cudaError_t launch_product(const Fp4Side& weights, MlpKernelArgs p, int64_t slots, int64_t segments, const LaunchCtx& ctx) {
  using L = Layout<kTok, kBlock>;
  CUtensorMap wmap, xmap;
  const int64_t all = (int64_t)p.experts * p.rows;
  cudaError_t e = make_fp8_tensor_map(&wmap, weights.data, all, p.width / 2, kDown ? kWeights : kWeights / 2);
  if (e != cudaSuccess) return e;
  e = make_fp8_tensor_map(&xmap, p.in.codes, slots * kTerms, p.width / 2, L::kBN);
  if (e != cudaSuccess) return e;
  p.scale = weights.scale;
  p.amax = weights.amax;
  p.amax_per_expert = weights.amax_per_row;
  p.tiles = kDown ? (p.rows + kWeights - 1) / kWeights : (p.inner + kWeights / 2 - 1) / (kWeights / 2);
  p.status = ctx.status;
  const int64_t tiles = segments * p.tiles, stages_k = (p.width + kStageK - 1) / kStageK;
  // A tile's stages are shared by up to four CTAs where they fit beside one another, two
  // stages each at least (6 tokens, one of 2 experts of 8192 x 1024: 21.6 us, unshared 25.5, by
  // up to eight 22.7; 8 tokens, one expert of 4096 x 2048: 19.9, 20.8 and 20.8).
  int split = 1;
  for (int s = 4; s >= 2 && split == 1; s /= 2)
    if (tiles * s <= 2 * ctx.num_sms && stages_k >= 2 * s) split = s;
  constexpr int kPerCta = 113 * 1024;  // two CTAs share an SM's 228 KB, 1 KB of it reserved for each
  const int rest = 1024 + L::rest(split, p.slots, p.experts);
  int stages = (kPerCta - rest) / L::kStageBytes;
  if (stages > kMaxStages) stages = kMaxStages;
  const int smem = rest + stages * L::kStageBytes;
  const auto kernel = expert_product_kernel<kDown, kTok, kBlock>;
  static std::atomic<uint64_t> allowed{0};
  e = allow_smem(reinterpret_cast<const void*>(kernel), kPerCta, allowed);
  if (e != cudaSuccess) return e;
  const int64_t room = 2 * ctx.num_sms / split;
  void* args[] = {&wmap, &xmap, &p, &stages, &split};
  return launch_dependent(reinterpret_cast<const void*>(kernel), dim3((unsigned)((tiles < room ? tiles : room) * split)),
                          dim3(kThreads), smem, ctx.stream, args, split);
}

template <int kTok, int kBlock>
cudaError_t launch_products(const ExpertMlpArgs& a, const Workspace& ws, const LaunchCtx& ctx) {
  const int64_t slots = a.tokens * a.topk, used = slots < a.experts ? slots : a.experts;
  MlpKernelArgs p = {};
  p.experts = a.experts;
  p.plan = ws.plan;
  p.gates = a.gates;
  p.parts = ws.parts;
  p.inner = (int)a.inner;
  p.ids = a.ids;
  p.slots = (int)slots;
  MlpKernelArgs up = p, down = p;
  up.rows = (int)(2 * a.inner), up.width = (int)a.hidden, up.in = ws.x, up.out = ws.h, up.hidden = ws.hidden;
  down.rows = (int)a.hidden, down.width = (int)a.inner, down.in = ws.h;
  cudaError_t e = launch_product<false, kTok, kBlock>(a.up, up, slots, used, ctx);
  if (e == cudaSuccess && kBlock == 16) {
    CutArgs c = {ws.hidden, (int)a.inner, ws.h, ws.plan};
    void* args[] = {&c};
    e = launch_dependent(reinterpret_cast<const void*>(cut_hidden_kernel),
                         dim3((unsigned)(slots * ((a.inner + kPrepPart - 1) / kPrepPart))), dim3(kPrepThreads), 0, ctx.stream,
                         args);
  }
  return e != cudaSuccess ? e : launch_product<true, kTok, kBlock>(a.down, down, slots, used, ctx);
}

template <int kBlock>
cudaError_t launch_layer(const ExpertMlpArgs& a, const LaunchCtx& ctx) {
  const Workspace ws = cut(a);
  PrepArgs p = {};
  p.x = static_cast<const uint16_t*>(a.x);
  p.ids = a.ids;
  p.slots = (int)(a.tokens * a.topk);
  p.topk = a.topk;
  p.experts = a.experts;
  p.width = (int)a.hidden;
  p.tok = tokens_per_segment(a.tokens, p.slots, a.experts);
  p.x_rows = ws.x;
  p.h_unit = ws.h.unit;
  p.plan = ws.plan;
  void* args[] = {&p};
  // Few tokens' choices are dealt to more CTAs, as far as two fit on an SM (one token, 32 of 64 experts of
  // 2048 x 512: 27.6 us, by one CTA for all of a token's 34.0; 13 tokens, 4 of 16 experts of 2720 x 1184: 27.8
  // and 28.0; with a CTA for each choice of 64 tokens, 4 of 32 experts of 4096 x 1536, 77.6 instead of 77.0).
  const unsigned groups = (unsigned)(a.tokens * ((a.hidden + kPrepPart - 1) / kPrepPart));
  int64_t shares = 2 * ctx.num_sms / groups;
  shares = shares < 1 ? 1 : shares < a.topk ? shares : a.topk;
  cudaError_t e = launch_dependent(reinterpret_cast<const void*>(prepare_kernel<kBlock>), dim3(groups, (unsigned)shares),
                                   dim3(kPrepThreads), 4 * (p.slots + 2 * p.experts + 2), ctx.stream, args);
  if (e != cudaSuccess) return e;
  e = p.tok == 2 ? launch_products<2, kBlock>(a, ws, ctx)
      : p.tok == 8 ? launch_products<8, kBlock>(a, ws, ctx)
                   : launch_products<14, kBlock>(a, ws, ctx);
  if (e != cudaSuccess) return e;
  int rows = (int)a.hidden, tokens = (int)a.tokens, topk = a.topk, experts = a.experts;
  const float* slots = ws.parts;
  const int32_t* ids = a.ids;
  void* y = a.y;
  const int64_t want = ((int64_t)tokens * rows / 4 + 255) / 256;
  void* join[] = {&slots, &ids, &topk, &experts, &rows, &tokens, &y};
  return launch_dependent(reinterpret_cast<const void*>(join_slots_kernel),
                          dim3((unsigned)(want < 8 * ctx.num_sms ? want : 8 * ctx.num_sms)), dim3(256), 0, ctx.stream, join);
}

}  // namespace
}  // namespace fp4

size_t expert_mlp_workspace(const ExpertMlpArgs& a) {
  const size_t any = fp4::cut(a).bytes, few = fp4::few_tokens_workspace(a);
  return any > few ? any : few;
}

cudaError_t launch_expert_mlp(const ExpertMlpArgs& a, const LaunchCtx& ctx) {
  if (a.tokens == 0 || a.hidden == 0) return cudaSuccess;
  if (a.inner == 0) return cudaMemsetAsync(a.y, 0, (size_t)a.tokens * a.hidden * 2, ctx.stream);
  if (fp4::few_tokens(a, ctx)) return fp4::launch_few_tokens(a, ctx);
  return a.block == 16 ? fp4::launch_layer<16>(a, ctx) : fp4::launch_layer<32>(a, ctx);
}

}  // namespace nvfp4
