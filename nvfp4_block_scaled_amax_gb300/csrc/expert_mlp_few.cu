// expert_mlp_few.cu -- the layer of expert_mlp.cu for one or two tokens and up to
// eight choices in all (and x's terms in shared memory, see few_tokens), in two
// launches: what the launches there take to begin is most of the time of so little
// work (one token to two of eight experts of 4096 x 2048: 19.9 us there and 15.8
// here, of which reading the weights takes 4.2; the rest is the start of two launches, the cut of x and of the hidden values
// into terms, and the clusters' joins, one after the other).
//
// The first kernel cuts x into terms itself, each CTA its share of the
// contracted dimension, while the first weights are on their way; both tokens
// are columns for every expert, whoever chose it.  It leaves the hidden rows in
// FP32, with the largest value of each tile of 64, and the second one cuts them
// the same way, a stage at a time, as the row's largest value is known by then.  It
// sums over all chosen experts of a row tile in one cluster, an accumulator
// each, and so has y in hand.
#include "expert_mlp.cuh"

namespace nvfp4 {
namespace fp4 {
namespace {

constexpr int kTok = 2, kBN = 16;
static_assert(kTok * kTerms <= kBN, "rows of the terms");
constexpr int kMaxChoices = 8;  // and experts at most
constexpr int kOutWarps = 4;
constexpr int kThreads = 32 * (kOutWarps + 2 + kScaleWarps);
constexpr int kTermWarps = kOutWarps + kScaleWarps;
constexpr int kWeights = 128;
constexpr int kMaxStages = 8, kMaxResident = 12;  // stages of the ring; of x's terms

struct FewArgs {
  const uint16_t* x;     // up
  const int32_t* ids;    // [tokens][topk]
  const float* gates;
  int tokens, topk, experts;
  const uint8_t* scale;  // of the weights, compact
  const float* amax;
  int amax_per_expert;
  int rows, width, inner;
  int tiles;             // of an expert's weights
  float* hidden;         // [experts chosen][kTok][inner]
  float* largest;        // [experts chosen][kTok][h_tiles]: the largest finite magnitudes of 64 each
  int h_tiles;
  uint16_t* y;           // down
  unsigned* status;
};

// The experts that were chosen, in the order of their first choice.
struct Chosen {
  int n;
  uint32_t by;  // bit kTok i + token: the token chose expert i
  int expert[kMaxChoices];
};

struct Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2];
  uint64_t terms;        // up: x's terms are there
  uint64_t got, taken;   // the cluster's partial results
  uint32_t tmem;
  float largest[kTermWarps][kTok];      // up: of x
  float unit[kTok * kMaxChoices];       // down: of the hidden rows' terms
  Chosen chosen;
};

// One warp finds them: lane s has choice s.
__device__ __forceinline__ void find_chosen(const FewArgs& p, Chosen& to) {
  const int lane = threadIdx.x & 31;
  int e = lane < p.tokens * p.topk ? __ldcg(&p.ids[lane]) : -1;
  if (e >= p.experts) e = -1;
  const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
  const int leader = __ffs(same) - 1;
  const uint32_t firsts = __ballot_sync(0xFFFFFFFFu, e >= 0 && lane == leader);
  const int i = __popc(firsts & ((1u << leader) - 1));
  const uint32_t by = __reduce_or_sync(0xFFFFFFFFu, e >= 0 ? 1u << (kTok * i + lane / p.topk) : 0u);
  if (e >= 0 && lane == leader) to.expert[i] = e;
  if (lane == 0) to.n = __popc(firsts), to.by = by;
}

template <bool kDown, int kBlock>
struct Layout {
  using F = Format<kBlock>;
  static constexpr int kWCodes = kWeights * kStageRow, kXCodes = kBN * kStageRow;
  static constexpr int kXBytes = kXCodes + F::kScaleBytes;
  // a stage of the ring: weights and their scales, and (down) the hidden terms with theirs
  static constexpr int kStageBytes = kWCodes + F::kScaleBytes + (kDown ? kXBytes : 0);
  static constexpr int kBuffers = kDown ? 1 : 2;
  static constexpr int kDCols = kDown ? kBN * kMaxChoices : kBN;  // of an accumulator
  static constexpr int kCols = kBuffers * kDCols + 2 * F::kCols;
  static constexpr int kTmemCols = kCols <= 64 ? 64 : 256;
  static_assert(kCols <= 256 && kStageBytes % 1024 == 0 && kXBytes % 1024 == 0, "tensor memory; swizzled operands");
  static int rest(int split, int resident) {
    return resident * kXBytes + kTok * kWeights * 4 + split * kWeights * 4 + (int)sizeof(Barriers);
  }
};

// x's largest finite element: warp `me` of kTermWarps, its part.
__device__ __forceinline__ void look_at_x(const FewArgs& p, int me, Barriers& bar) {
  const int lane = threadIdx.x & 31;
  for (int token = 0; token < p.tokens; ++token) {
    const uint4* row = reinterpret_cast<const uint4*>(p.x + (int64_t)token * p.width);
    float m = 0.0f;
#pragma unroll 2
    for (int k = 32 * me + lane; k < p.width / 8; k += 32 * kTermWarps) {
      const uint4 u = row[k];
      const float v[8] = {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y),
                          bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w)};
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_magnitude(v[i]));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    if (lane == 0) bar.largest[me][token] = m;
  }
}

// 128 elements of a token (four a lane, from k on, the lane's first) into a
// stage's terms: rows of 128 bytes, 16-byte places swizzled by the row, and behind
// them (`scales`) the blocks' scales.
template <int kBlock>
__device__ __forceinline__ void cut_part(float (&v)[4], float unit, int token, int k, uint8_t* codes_at, uint8_t* scales) {
  const int in_stage = k % kStageK, b = in_stage / 2;
  const uint32_t scale = to_terms<kBlock>(v, unit, [&](int i, uint16_t codes) {
    const int n = token * kTerms + i;
    *reinterpret_cast<uint16_t*>(codes_at + n * kStageRow + (((b >> 4) ^ (n & 7)) * 16) + (b & 15)) = codes;
  });
  put_scale<kBlock>(scales, token * kTerms, in_stage, scale);
}

// ---------------------------------------------------------------------------
template <bool kDown, int kBlock>
__global__ void __launch_bounds__(kThreads, 2)
few_tokens_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ FewArgs p, int stages, int split,
                  int resident) {
  using L = Layout<kDown, kBlock>;
  using F = Format<kBlock>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* x_terms = smem + stages * L::kStageBytes;  // up: [stage of this CTA's share] as kXBytes
  float* results = reinterpret_cast<float*>(x_terms + resident * L::kXBytes);  // [token][row]
  float* shares = results + kTok * kWeights;                                   // [rank][row] of the CTA's token
  Barriers* bar = reinterpret_cast<Barriers*>(shares + split * kWeights);
  const int w = warp_index(), lane = threadIdx.x & 31;
  const int rank = split > 1 ? (int)cluster_rank() : 0;

  if (w == kOutWarps) {
    if (lane == 0) {
      for (int i = 0; i < stages; ++i) {
        mbar_init(&bar->full[i], kDown ? 2 + 2 * p.tokens : 2);  // the copies, the weights' scales (and the terms)
        mbar_init(&bar->empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar->tfull[i], 1);
        mbar_init(&bar->tempty[i], kOutWarps);
      }
      mbar_init(&bar->terms, kTermWarps);
      mbar_init(&bar->got, 1);
      mbar_init(&bar->taken, kOutWarps * split);
      fence_mbar_init();
      tma_prefetch_desc(&wmap);
    }
  } else if (w == kOutWarps + 1) {
    tmem_alloc(&bar->tmem, L::kTmemCols);
  }
  __syncwarp();
  if (split > 1) cluster_arrive();  // (the barriers are set up)
  // The second kernel begins when all CTAs of the first are past their wait, and
  // reads what neither writes ahead of its own.
  if (!kDown) {
    grid_dependency_wait();
    grid_launch_dependents();
  }
  if (w == 0) find_chosen(p, bar->chosen);
  if (!kDown && w != kOutWarps && w != kOutWarps + 1) look_at_x(p, w < kOutWarps ? w : w - 2, *bar);
  tcgen05_before_sync();
  __syncthreads();
  if (split > 1) cluster_wait();
  tcgen05_after_sync();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, bar->tmem, 0);
  const int lg_split = __ffs(split) - 1;
  const int t0 = blockIdx.x >> lg_split, step = gridDim.x >> lg_split;
  const int nkb = (p.width + kStageK - 1) / kStageK;
  const int full_stages = p.width / kStageK, last_steps = (p.width % kStageK + 63) / 64;  // of 64 elements
  // up: a tile for each chosen expert's 64 gate and 64 up rows, its stages shared by the cluster; down: a
  // tile for 128 rows, the stages of all chosen experts shared
  const Chosen& chosen = bar->chosen;
  const int n_experts = __shfl_sync(0xFFFFFFFFu, chosen.n, 0);
  const int tiles = kDown ? p.tiles : n_experts * p.tiles, per_tile = kDown ? n_experts * nkb : nkb;
  const int i0 = (per_tile * rank) >> lg_split, i1 = (per_tile * (rank + 1)) >> lg_split;
  constexpr int kTileRows = kDown ? kWeights : kWeights / 2;
  bool ok = true;

  // x into terms: the CTA's share of the stages, by the warps that neither copy nor multiply.
  float unit[kTok] = {1.0f, 1.0f};
  auto cut_x = [&](int me) {  // me: 0 .. kTermWarps - 1
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      float m = bar->largest[0][i];
#pragma unroll
      for (int j = 1; j < kTermWarps; ++j) m = fmaxf(m, bar->largest[j][i]);
      unit[i] = kBlock == 16 ? unit_of(m) : 1.0f;
    }
    // 128 elements of a token at a time, up to the last step of 64 padded with zeros
    const int parts = 2 * (i1 - i0);
    for (int q = me; q < parts * p.tokens; q += kTermWarps) {
      const int token = q / parts, k = i0 * kStageK + 128 * (q % parts) + 4 * lane;
      if (k - 4 * lane >= p.width) continue;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (k < p.width) {
        const uint2 u = *reinterpret_cast<const uint2*>(p.x + (int64_t)token * p.width + k);
        v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
      }
      uint8_t* stage = x_terms + (k / kStageK - i0) * L::kXBytes;
      cut_part<kBlock>(v, token == 0 ? unit[0] : unit[1], token, k, stage, stage + L::kXCodes);
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar->terms);
  };

  if (w == kOutWarps) {
    // Stage i of tile t: its expert (of those chosen) and its place along the contracted dimension.
    auto expert_of = [&](int t, int i) { return kDown ? i / nkb : t / p.tiles; };
    auto weights = [&](int t, int i, uint32_t s) {
      const int e = expert_of(t, i), kb = kDown ? i - e * nkb : i, tile = kDown ? t : t - e * p.tiles;
      const int row = chosen.expert[e] * p.rows + tile * kTileRows;
      if (elect_one()) {
        const uint32_t dst = smem_u32(smem + s * L::kStageBytes), full = smem_u32(&bar->full[s]);
        mbar_arrive_expect_tx(&bar->full[s], L::kWCodes);
        tma_load(dst, &wmap, kb * kStageRow, row, full);
        if (!kDown) tma_load(dst + L::kWCodes / 2, &wmap, kb * kStageRow, row + p.inner, full);
      }
      __syncwarp();
    };
    int early = 0;
    if constexpr (kDown) {
      for (int t = t0; t < tiles && early < stages; t += step)
        for (int i = i0; i < i1 && early < stages; ++i, ++early) weights(t, i, early);
      grid_dependency_wait();
      grid_launch_dependents();
    }
    uint32_t s = 0, phase = 1;
    int sent = 0;
    for (int t = t0; t < tiles && ok; t += step)
      for (int i = i0; i < i1; ++i) {
        if (sent >= early) {
          if (!mbar_wait(&bar->empty[s], phase)) {
            ok = false;
            break;
          }
          weights(t, i, s);
        }
        ++sent;
        if (++s == (uint32_t)stages) {
          s = 0;
          phase ^= 1;
        }
      }
    if (!ok) {
      report_timeout(p.status);
      // let the copies in flight land
      for (int i = sent < stages ? 0 : sent - stages; i < sent; ++i) mbar_wait(&bar->full[i % stages], (i / stages) & 1);
    }
  } else if (w == kOutWarps + 1) {
    if (kDown) grid_dependency_wait(), grid_launch_dependents();
    constexpr uint32_t kIdesc = F::idesc(kWeights, kBN);
    const uint64_t desc0 = operand_desc(smem_u32(smem)), xdesc0 = operand_desc(smem_u32(x_terms));
    // (the ring's scales: the weights', then the hidden terms'; of x's terms behind their codes)
    const uint64_t sdesc0 = scale_desc(smem_u32(smem) + L::kWCodes + (kDown ? L::kXCodes : 0));
    const uint64_t xsdesc0 = scale_desc(smem_u32(x_terms) + L::kXCodes);
    const uint32_t sw = tmem + L::kBuffers * L::kDCols, sx = sw + F::kCols;
    uint32_t s = 0, phase = 0, buf = 0, tphase = 1;
    if (!kDown) ok = mbar_wait(&bar->terms, 0);
    for (int t = t0; t < tiles && ok; t += step) {
      if (!mbar_wait(&bar->tempty[buf], tphase)) {
        ok = false;
        break;
      }
      for (int i = i0; i < i1; ++i) {
        if (!mbar_wait(&bar->full[s], phase)) {
          ok = false;
          break;
        }
        tcgen05_after_sync();
        const int e = kDown ? i / nkb : 0, kb = i - e * nkb;
        const uint64_t a = desc0 + s * (L::kStageBytes / 16);
        const uint64_t b = kDown ? a + L::kWCodes / 16 : xdesc0 + (i - i0) * (L::kXBytes / 16);
        const uint64_t ds = sdesc0 + s * (L::kStageBytes / 16);
        const uint64_t dx = kDown ? ds + F::kScaleBytes / 16 : xsdesc0 + (i - i0) * (L::kXBytes / 16);
        const uint32_t d = tmem + buf * L::kDCols + e * kBN;
        const uint32_t add = i > i0 && kb > 0;
        auto copy = [&](int j) {
          scales_to_tmem<1>(sw + 4 * j, ds + j * (kScaleTile / 16));
          scales_to_tmem<1>(sx + 4 * j, dx + j * (kScaleTile / 16));
        };
        auto multiply = [&](int k) {
          umma_fp4<1, kBlock>(d, a + 2 * k, b + 2 * k, kIdesc | F::half(k), sw + F::col(k), sx + F::col(k), k > 0 ? 1 : add);
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
          if (i + 1 == i1) umma_commit(&bar->tfull[buf]);
        }
        __syncwarp();
        if (++s == (uint32_t)stages) {
          s = 0;
          phase ^= 1;
        }
      }
      if (i0 == i1 && lane == 0) mbar_arrive(&bar->tfull[buf]);  // (fewer stages than CTAs: nothing to add)
      if (++buf == L::kBuffers) {
        buf = 0;
        tphase ^= 1;
      }
    }
    if (!ok) report_timeout(p.status);
  } else if (w > kOutWarps + 1) {
    bool waited = !kDown;
    if (kDown) stale_lines_gone();
    const int mine = w - kOutWarps - 2, active = active_scale_warps(stages);
    if (!kDown) cut_x(kOutWarps + mine);
    if (mine < active) {
      uint32_t s = 0, phase = 1, it = 0;
      const CompactScales<kBlock> scales(p.scale, p.width, (int64_t)p.experts * p.rows);
      for (int t = t0; t < tiles && ok; t += step)
        for (int i = i0; i < i1 && ok; ++i, ++it) {
          if ((it & (active - 1)) == (uint32_t)mine) {
            const int e = kDown ? i / nkb : t / p.tiles, kb = kDown ? i - e * nkb : i, tile = kDown ? t : t - e * p.tiles;
            uint32_t v[4][F::kTiles];
            const int64_t row = (int64_t)chosen.expert[e] * p.rows + tile * kTileRows, gap = kDown ? 0 : p.inner - kWeights / 2;
            if (!waited && it >= (uint32_t)stages) {
              grid_dependency_wait();
              grid_launch_dependents();
              waited = true;
            }
            scales.read(row, kWeights, kb, v, gap);
            ok = mbar_wait(&bar->empty[s], phase);
            if (ok) {
              scales.write(smem_u32(smem + s * L::kStageBytes) + L::kWCodes + (kDown ? L::kXCodes : 0), v);
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
      if (!ok) report_timeout(p.status);
    }
    if (!waited) {
      grid_dependency_wait();
      grid_launch_dependents();
    }
  } else {
    if (kDown) grid_dependency_wait(), grid_launch_dependents();
    else cut_x(w);
    // down: the share's hidden rows into terms, parts of 128 elements dealt out to these warps: stage q / per_stage
    // of the ring, of its expert the token and the half of the stage.  (A warp is one stage, or two of a token's,
    // ahead of itself, which a ring of two allows.)
    const int per_stage = 2 * p.tokens;
    uint32_t used = 0;  // stages of the ring before this tile's
    auto hidden_at = [&](int q, int& row, int& k) {
      const int i = i0 + q / per_stage, e = i / nkb, at = q % per_stage;
      row = kTok * e + (at >> 1), k = (i - e * nkb) * kStageK + 128 * (at & 1) + 4 * lane;
    };
    auto read_hidden = [&](int q, float (&v)[4]) {
      int row, k;
      hidden_at(q, row, k);
      float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (q < per_stage * (i1 - i0) && k < p.width && (chosen.by >> row & 1))
        u = __ldcg(reinterpret_cast<const float4*>(p.hidden + (int64_t)row * p.width + k));
      v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    };
    auto cut_hidden = [&]() {
      float next[4];
      read_hidden(w, next);
      for (int q = w; q < per_stage * (i1 - i0); q += kOutWarps) {
        float v[4] = {next[0], next[1], next[2], next[3]};
        read_hidden(q + kOutWarps, next);
        const uint32_t use = used + q / per_stage, slot = use % stages;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bar->empty[slot], ((use / stages) & 1) ^ 1))) return false;
        int row, k;
        hidden_at(q, row, k);
        uint8_t* to = smem + slot * L::kStageBytes + L::kWCodes;
        if (k - 4 * lane < p.width)
          cut_part<kBlock>(v, kBlock == 16 ? bar->unit[row] : 1.0f, row % kTok, k, to, to + L::kXCodes + F::kScaleBytes);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->full[slot]);
      }
      used += i1 - i0;
      return true;
    };
    if (kDown && kBlock == 16) {
      for (int row = w; row < kTok * n_experts; row += kOutWarps) {
        float m = 0.0f;
        if (chosen.by >> row & 1)
          for (int i = lane; i < p.h_tiles; i += 32) m = fmaxf(m, __ldcg(p.largest + row * p.h_tiles + i));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        if (lane == 0) bar->unit[row] = unit_of(m);
      }
      together(true);
    }
    const uint32_t lane_base = tmem + ((uint32_t)(32 * w) << 16);
    const int r = 32 * w + lane;
    uint32_t buf = 0, tphase = 0, round = 0;
    // down: what a token's sum over expert i's hidden values counts for: lane kTok i + token
    float weight = 0.0f;
    if (kDown && lane < kTok * n_experts && (chosen.by >> lane & 1)) {
      const int e = chosen.expert[lane / kTok], token = lane % kTok;
      float gate = 0.0f;
      for (int j = 0; j < p.topk; ++j)
        if (p.ids[token * p.topk + j] == e) gate = __fadd_rn(gate, p.gates[token * p.topk + j]);
      const float factor = kBlock == 16 ? __fdiv_rn(p.amax[p.amax_per_expert ? e : 0], 2688.0f) : 1.0f;
      weight = __fmul_rn(__fmul_rn(kBlock == 16 ? bar->unit[lane] : 1.0f, factor), gate);
    }
    for (int t = t0; t < tiles && ok; t += step) {
      const int e0 = kDown ? 0 : t / p.tiles, tile = kDown ? t : t - e0 * p.tiles;
      // the tokens that this CTA finishes: all, or the one with its rank
      const int first = split == 1 ? 0 : rank, end = min(p.tokens, split == 1 ? kTok : rank + 1);
      if (kDown) ok = cut_hidden();
      ok = ok && mbar_wait(&bar->tfull[buf], tphase);
      if (ok && split > 1) ok = mbar_wait_cluster(&bar->taken, (round & 1) ^ 1, p.status);
      if (!(ok = together(ok))) break;
      tcgen05_after_sync();
      if (split > 1 && w == 0 && lane == 0)
        mbar_arrive_expect_tx(&bar->got, end > first ? split * kWeights * 4 : 0);
      float out[kTok] = {0.0f, 0.0f};
      const int ea = kDown ? i0 / nkb : 0, eb = i0 == i1 ? ea : kDown ? (i1 - 1) / nkb + 1 : 1;
      for (int e = ea; e < eb; ++e) {
        uint32_t v[16];
        tmem_read(lane_base + buf * L::kDCols + e * kBN, v);
#pragma unroll
        for (int token = 0; token < kTok; ++token) {
          const float sums = add_terms(v + kTerms * token);
          if constexpr (kDown) {
            const float by = __shfl_sync(0xFFFFFFFFu, weight, kTok * e + token);
            if (chosen.by >> (kTok * e + token) & 1) out[token] = __fadd_rn(out[token], __fmul_rn(sums, by));
          } else {
            out[token] = sums;
          }
        }
      }
      tcgen05_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->tempty[buf]);
      if (split > 1) {
#pragma unroll
        for (int token = 0; token < kTok; ++token)
          if (token < p.tokens)
            store_async(map_to_cta(smem_u32(shares + rank * kWeights + r), token), out[token],
                        map_to_cta(smem_u32(&bar->got), token));
        ok = together(mbar_wait_cluster(&bar->got, round & 1, p.status));
        if (!ok) break;
        if (end > first) {
          float all = 0.0f;
          for (int i = 0; i < split; ++i) all = __fadd_rn(all, shares[i * kWeights + r]);
          out[0] = all;
        }
        __syncwarp();
        if (t + step < tiles && lane < split) mbar_arrive_cluster_release(map_to_cta(smem_u32(&bar->taken), lane));
        ++round;
      }
      // out[i]: token first + i
      if constexpr (kDown) {
        const int o = kWeights * tile + r;
        for (int token = first; token < end; ++token) {
          uint16_t h;
          asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(token == first ? out[0] : out[1]));
          if (o < p.rows) p.y[(int64_t)token * p.rows + o] = h;
        }
      } else {
        results[r] = out[0];
        if (split == 1) results[kWeights + r] = out[1];
        together(true);  // gate and up sums come from different warps
        // 16 lanes take a token's 64 hidden values, four each
        const int token = first + (lane >> 4), f = kTileRows * tile + 4 * (lane & 15);
        const float factor = kBlock == 16 ? __fdiv_rn(p.amax[p.amax_per_expert ? chosen.expert[e0] : 0], 2688.0f) : 1.0f;
        if (w == 0 && end > first) {
          const bool there = token < end && (chosen.by >> (kTok * e0 + token) & 1);
          const float x_unit = __fmul_rn(token == 0 ? unit[0] : unit[1], factor);
          float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, m = 0.0f;
          if (there && f < p.inner) {
            const float4 a = *reinterpret_cast<const float4*>(results + (token - first) * kWeights + 4 * (lane & 15));
            const float4 b = *reinterpret_cast<const float4*>(results + (token - first) * kWeights + 64 + 4 * (lane & 15));
            const float gate[4] = {a.x, a.y, a.z, a.w}, up[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float z = __fmul_rn(gate[i], x_unit);
              v[i] = __fmul_rn(__fdiv_rn(z, __fadd_rn(1.0f, expf(-z))), __fmul_rn(up[i], x_unit));
              m = fmaxf(m, finite_magnitude(v[i]));
            }
            *reinterpret_cast<float4*>(p.hidden + (int64_t)(kTok * e0 + token) * p.inner + f) =
                make_float4(v[0], v[1], v[2], v[3]);
          }
#pragma unroll
          for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
          if (there && (lane & 15) == 0) p.largest[(kTok * e0 + token) * p.h_tiles + tile] = m;
        }
        together(true);  // the results may be overwritten
      }
      if (++buf == L::kBuffers) {
        buf = 0;
        tphase ^= 1;
      }
    }
    if (!ok) report_timeout(p.status);
  }
  __syncwarp();
  tcgen05_before_sync();
  __syncthreads();
  // (as in expert_mlp.cu)
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

// ---------------------------------------------------------------------------
int64_t stages_of(int64_t width) { return (width + kStageK - 1) / kStageK; }
int64_t most_experts(const ExpertMlpArgs& a) {
  const int64_t slots = a.tokens * a.topk;
  return slots < a.experts ? slots : a.experts;
}
int64_t hidden_tiles(const ExpertMlpArgs& a) { return (a.inner + kWeights / 2 - 1) / (kWeights / 2); }
// CTAs of a cluster that share a tile's stages: as many as fit beside one another, up to four, two stages each
// at least (one token, two of 8 experts of 4096 x 2048: 15.8 us, by up to eight too, two 17.6, unshared 20.0).
int split_of(int64_t tiles, int64_t stages, const LaunchCtx& ctx) {
  for (int s = 4; s >= 2; s /= 2)
    if (tiles * s <= 2 * ctx.num_sms && stages >= 2 * s) return s;
  return 1;
}
int up_split(const ExpertMlpArgs& a, const LaunchCtx& ctx) {
  return split_of(most_experts(a) * hidden_tiles(a), stages_of(a.hidden), ctx);
}

struct Workspace {
  float *hidden, *largest;
  size_t bytes;
};
Workspace cut(const ExpertMlpArgs& a) {
  Workspace ws = {};
  const int64_t rows = kTok * most_experts(a);
  uint8_t* at = static_cast<uint8_t*>(a.workspace);
  auto take = [&](int64_t bytes) {
    uint8_t* p = at + ws.bytes;
    ws.bytes += (size_t)((bytes + 127) / 128 * 128);
    return reinterpret_cast<float*>(p);
  };
  ws.hidden = take(4 * rows * a.inner);
  ws.largest = take(4 * rows * hidden_tiles(a));
  return ws;
}

template <bool kDown, int kBlock>
cudaError_t launch_product(const ExpertMlpArgs& a, FewArgs p, const LaunchCtx& ctx) {
  using L = Layout<kDown, kBlock>;
  const Fp4Side& weights = kDown ? a.down : a.up;
  p.rows = (int)(kDown ? a.hidden : 2 * a.inner);
  p.width = (int)(kDown ? a.inner : a.hidden);
  p.inner = (int)a.inner;
  p.scale = weights.scale;
  p.amax = weights.amax;
  p.amax_per_expert = weights.amax_per_row;
  p.h_tiles = (int)hidden_tiles(a);
  p.tiles = kDown ? (p.rows + kWeights - 1) / kWeights : p.h_tiles;
  CUtensorMap wmap;
  cudaError_t e = make_fp8_tensor_map(&wmap, weights.data, (int64_t)p.experts * p.rows, p.width / 2,
                                      kDown ? kWeights : kWeights / 2);
  if (e != cudaSuccess) return e;
  const int64_t tiles = kDown ? p.tiles : most_experts(a) * p.tiles;
  int split = kDown ? split_of(tiles, most_experts(a) * stages_of(p.width), ctx) : up_split(a, ctx);
  int resident = kDown ? 0 : (int)((stages_of(p.width) + split - 1) / split);
  constexpr int kPerCta = 113 * 1024;  // two CTAs share an SM's 228 KB, 1 KB of it reserved for each
  const int rest = 1024 + L::rest(split, resident);
  int stages = (kPerCta - rest) / L::kStageBytes;
  if (stages > kMaxStages) stages = kMaxStages;
  const auto kernel = few_tokens_kernel<kDown, kBlock>;
  static std::atomic<uint64_t> allowed{0};
  e = allow_smem(reinterpret_cast<const void*>(kernel), kPerCta, allowed);
  if (e != cudaSuccess) return e;
  const int64_t room = 2 * ctx.num_sms / split;
  void* args[] = {&wmap, &p, &stages, &split, &resident};
  return launch_dependent(reinterpret_cast<const void*>(kernel), dim3((unsigned)((tiles < room ? tiles : room) * split)),
                          dim3(kThreads), rest + stages * L::kStageBytes, ctx.stream, args, split);
}

}  // namespace

bool few_tokens(const ExpertMlpArgs& a, const LaunchCtx& ctx) {
  if (a.tokens > kTok || a.tokens * a.topk > kMaxChoices) return false;
  const int split = up_split(a, ctx);
  // x's terms stay in shared memory, beside three stages of weights at least; where a CTA's share is
  // longer (many tiles, none of them shared) it would leave fewer, and the layer has work enough for
  // the launches of expert_mlp.cu.
  return (stages_of(a.hidden) + split - 1) / split <= kMaxResident;
}

size_t few_tokens_workspace(const ExpertMlpArgs& a) {
  return a.tokens <= kTok && a.tokens * a.topk <= kMaxChoices ? cut(a).bytes : 0;
}

cudaError_t launch_few_tokens(const ExpertMlpArgs& a, const LaunchCtx& ctx) {
  const Workspace ws = cut(a);
  FewArgs p = {};
  p.x = static_cast<const uint16_t*>(a.x);
  p.ids = a.ids;
  p.gates = a.gates;
  p.tokens = (int)a.tokens;
  p.topk = a.topk;
  p.experts = a.experts;
  p.hidden = ws.hidden;
  p.largest = ws.largest;
  p.y = static_cast<uint16_t*>(a.y);
  p.status = ctx.status;
  const cudaError_t e = a.block == 16 ? launch_product<false, 16>(a, p, ctx) : launch_product<false, 32>(a, p, ctx);
  if (e != cudaSuccess) return e;
  return a.block == 16 ? launch_product<true, 16>(a, p, ctx) : launch_product<true, 32>(a, p, ctx);
}

}  // namespace fp4
}  // namespace nvfp4
