// tokens.cu -- tokens sorted by expert and back.
//
// A token t has topk slots s = t * topk + j, each with an expert e_s.  The
// sort places the slots in stable order of their expert: with count_e the
// slots of expert e and offset_e the sum of the earlier experts' counts, each
// rounded up to `align`,
//     row(s) = offset_{e_s} + #{s' < s : e_{s'} = e_s}.
// The gather copies each token to the rows of its slots; the combine adds the
// rows of a token with its weights, y_t = sum_j w_tj rows[row(t, j)], and its
// gradient is drows[r] = w_s dy_t and dw_tj = <dy_t, rows[row(t, j)]>.
// Integer counting only, and every sum in a fixed order: results do not
// depend on timing.
#include "common.cuh"
#include "dependent.h"
#include "tokens.h"

namespace nvfp4 {
namespace {

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortChunk = 2048;  // slots of one CTA, as long as there are no more chunks than SMs

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a, int64_t chunk) {
  extern __shared__ int cnt[];
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) cnt[e] = 0;
  grid_begin();
  __syncthreads();
  const int64_t begin = blockIdx.x * chunk, end = min(begin + chunk, a.slots);
#pragma unroll 4
  for (int64_t s = begin + threadIdx.x; s < end; s += kSortThreads) {
    const int e = a.ids[s];
    if ((unsigned)e < (unsigned)a.experts) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads)
    a.scratch[(int64_t)blockIdx.x * a.experts + e] = cnt[e];
}

// One CTA per chunk.  Each warp counts its own run of the chunk's slots with
// match_any (so the order inside an expert is the slots' order), the counts
// become first rows, and a second walk hands the rows out.  Latency is all
// that counts, so every step between the walks is spread over the CTA: 2048
// slots to 64 experts 6.6 us (one warp adding the first rows up and the CTA
// filling one member's padding after another: 15.8), 131,072 to 256 16.7.
//
// kCopy (few slots): the sort and the gather in one launch.  Every CTA sorts
// all slots for itself, which costs less than a second launch would, the
// first one writes the maps, and each copies its share of the rows, a warp
// per piece of 2 KB.
constexpr int kCopyPiece = 2048;
constexpr int kCopyRows = 6144;  // at most, one integer of shared memory each

template <bool kCopy>
__global__ void __launch_bounds__(kSortThreads)
sort_place_kernel(SortArgs a, int64_t chunk, const uint8_t* x, uint8_t* out, int64_t row_bytes, int topk) {
  extern __shared__ int smem[];
  int* wcnt = smem;                            // [warps][experts]: counts, then the next row of warp and expert
  int* total = smem + kSortWarps * a.experts;  // [experts]
  int* base = total + a.experts;               // [experts]: rows in the earlier chunks, then the chunk's first row
  int* first = base + a.experts;               // [experts + 1]: offsets
  int* map = first + a.experts + 1;            // kCopy: [rows], slot of each row
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nchunks = kCopy ? 1 : gridDim.x, self = kCopy ? 0 : blockIdx.x;
  const bool writes = !kCopy || blockIdx.x == 0;
  for (int i = threadIdx.x; i < (kSortWarps + 2) * a.experts; i += kSortThreads) wcnt[i] = 0;  // and total, base
  if (kCopy)
    for (int i = threadIdx.x; i < a.rows; i += kSortThreads) map[i] = -1;
  grid_begin();
  __syncthreads();
  const int64_t seg = chunk / kSortWarps;
  const int64_t begin = self * chunk + w * seg;
  const int64_t end = min(begin + seg, a.slots);
  int* mine = wcnt + w * a.experts;
  // The first ids of the lane are read at once and kept for both walks.
  constexpr int kHeld = 4;
  int held[kHeld];
  auto expert_at = [&](int64_t s) {
    const int e = s < end ? a.ids[s] : -1;
    return (unsigned)e < (unsigned)a.experts ? e : -1;
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k) held[k] = expert_at(begin + 32 * k + lane);
  auto walk = [&](auto&& visit) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (begin + 32 * k < end) visit(begin + 32 * k + lane, held[k]);
    for (int64_t s0 = begin + 32 * kHeld; s0 < end; s0 += 32) visit(s0 + lane, expert_at(s0 + lane));
  };
  walk([&](int64_t, int e) {
    const unsigned peers = __match_any_sync(0xFFFFFFFFu, e);
    if (e >= 0 && lane == __ffs(peers) - 1) mine[e] += __popc(peers);
    __syncwarp();
  });
  if (nchunks > 1)  // a lane per expert: its rows in the earlier chunks and in all of them, chunks dealt out to the warps
    for (int e = lane; e < a.experts; e += 32) {
      int before = 0, all = 0;
#pragma unroll 4
      for (int c = w; c < nchunks; c += kSortWarps) {
        const int v = a.scratch[(int64_t)c * a.experts + e];
        before += c < self ? v : 0;
        all += v;
      }
      if (before) atomicAdd(&base[e], before);  // (integers: any order gives the same)
      if (all) atomicAdd(&total[e], all);
    }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) {
    int c[kSortWarps], all = 0;
#pragma unroll
    for (int i = 0; i < kSortWarps; ++i) c[i] = wcnt[i * a.experts + e];
#pragma unroll
    for (int i = 0; i < kSortWarps; ++i) {
      wcnt[i * a.experts + e] = all;
      all += c[i];
    }
    if (nchunks == 1) total[e] = all;
  }
  __syncthreads();
  if (w == 0) {
    int run = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
      const int e = e0 + lane;
      // (unsigned: the sum before the division may pass 2^31, the member's rows do not)
      const int padded = e < a.experts ? (int)(((unsigned)total[e] + a.align - 1) / a.align * a.align) : 0;
      int incl = padded;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += v;
      }
      if (e < a.experts) {
        first[e] = run + incl - padded;
        base[e] += first[e];
      }
      run += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (lane == 0) first[a.experts] = run;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kSortWarps * a.experts; i += kSortThreads) wcnt[i] += base[i % a.experts];
  __syncthreads();
  walk([&](int64_t s, int e) {
    const unsigned peers = __match_any_sync(0xFFFFFFFFu, e);
    const int row = e >= 0 ? mine[e] + __popc(peers & ((1u << lane) - 1u)) : -1;
    __syncwarp();
    if (e >= 0 && lane == __ffs(peers) - 1) mine[e] += __popc(peers);
    __syncwarp();
    if (s < end) {
      if (writes) {
        a.row_of_slot[s] = row;
        if (row >= 0) a.slot_of_row[row] = (int32_t)s;
      }
      if (kCopy && row >= 0) map[row] = (int)s;
    }
  });
  if (writes) {
    // rows without a slot: the end of every member and the end of the capacity
    // (a warp per member where that is a few rows, or the CTA)
    const int group = a.align <= kSortThreads ? 32 : kSortThreads, groups = kSortThreads / group;
    for (int e = self * groups + threadIdx.x / group; e < a.experts; e += nchunks * groups)
      // (64 bits: a member may end just below 2^31, a lane's first row and its next one past it)
      for (int64_t r = (int64_t)first[e] + total[e] + threadIdx.x % group; r < first[e + 1]; r += group)
        a.slot_of_row[r] = -1;
    for (int64_t r = first[a.experts] + (int64_t)self * kSortThreads + threadIdx.x; r < a.rows;
         r += (int64_t)nchunks * kSortThreads)
      a.slot_of_row[r] = -1;
    if (self == 0)
      for (int e = threadIdx.x; e <= a.experts; e += kSortThreads) a.offsets[e] = first[e];
  }
  if constexpr (kCopy) {
    __syncthreads();
    const int pieces = (int)((row_bytes + kCopyPiece - 1) / kCopyPiece);
    for (int64_t u = (int64_t)blockIdx.x * kSortWarps + w; u < a.rows * pieces; u += (int64_t)gridDim.x * kSortWarps) {
      const int64_t r = u / pieces, off = (u - r * pieces) * kCopyPiece;
      const int slot = map[r], n = (int)min((int64_t)kCopyPiece, row_bytes - off);
      const uint8_t* src = x + (slot >= 0 ? slot / topk : 0) * row_bytes + off;
      uint8_t* dst = out + r * row_bytes + off;
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = (lane + 32 * i) * 16;
        v[i] = make_uint4(0, 0, 0, 0);
        if (slot >= 0 && at < n) v[i] = *reinterpret_cast<const uint4*>(src + at);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((lane + 32 * i) * 16 < n) *reinterpret_cast<uint4*>(dst + (lane + 32 * i) * 16) = v[i];
    }
  }
}

// ---------------------------------------------------------------------------
// Gather: a warp takes 2 KB of a token into registers and stores them to the
// rows of its kept slots, so a token is read once however many rows it goes
// to; then the warps zero the rows without a slot.  Memory-bound, mostly by
// stores.  A warp per piece: 16384 x 4096 BF16 to 36,800 rows in 104 us, 6.8
// TB/s; the same warps in a grid that stays (8 per SM) 121 us; through shared
// memory, bulk copies of 2 to 8 KB in and out, 134 us.
constexpr int kGatherWarps = 4;
constexpr int kPiece = 2048;   // bytes of a token a warp moves at a time
constexpr int kZeroRows = 8;   // rows a warp looks at in one go

__global__ void __launch_bounds__(32 * kGatherWarps)
gather_kernel(const uint8_t* x, uint8_t* out, TokenArgs a, int64_t row_bytes) {
  grid_begin();
  const int lane = threadIdx.x & 31;
  const int64_t slots = a.tokens * a.topk;
  const int pieces = (int)((row_bytes + kPiece - 1) / kPiece);
  const int64_t warp = (int64_t)blockIdx.x * kGatherWarps + (threadIdx.x >> 5);
  const int64_t warps = (int64_t)gridDim.x * kGatherWarps;
  for (int64_t u = warp; u < a.tokens * pieces; u += warps) {
    const int64_t t = u / pieces, off = (u - t * pieces) * kPiece;
    const int n = (int)min((int64_t)kPiece, row_bytes - off);
    const uint4* src = reinterpret_cast<const uint4*>(x + t * row_bytes + off) + lane;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((lane + 32 * i) * 16 < n) v[i] = __ldcs(src + 32 * i);
    for (int j0 = 0; j0 < a.topk; j0 += 32) {
      const int mine = j0 + lane < a.topk ? a.row_of_slot[t * a.topk + j0 + lane] : -1;
      for (int j = 0; j < min(32, a.topk - j0); ++j) {
        const int row = __shfl_sync(0xFFFFFFFFu, mine, j);
        if (row < 0 || row >= a.rows) continue;
        uint4* dst = reinterpret_cast<uint4*>(out + row * row_bytes + off) + lane;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((lane + 32 * i) * 16 < n) __stcs(dst + 32 * i, v[i]);
      }
    }
  }
  for (int64_t r0 = warp * kZeroRows; r0 < a.rows; r0 += warps * kZeroRows) {
    // (a lane without a row of its own counts as none, whatever the number of slots: 0 is no valid slot of 0 tokens)
    const bool there = lane < kZeroRows && r0 + lane < a.rows;
    const int slot = there ? a.slot_of_row[r0 + lane] : 0;
    unsigned empty = __ballot_sync(0xFFFFFFFFu, there && (slot < 0 || slot >= slots));
    for (; empty; empty &= empty - 1) {
      uint4* dst = reinterpret_cast<uint4*>(out + (r0 + __ffs(empty) - 1) * row_bytes);
      for (int64_t i = lane; i < row_bytes / 16; i += 32) __stcs(dst + i, make_uint4(0, 0, 0, 0));
    }
  }
}

constexpr int kRowThreads = 128;

template <bool kBf16>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[kBf16 ? 8 : 4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kBf16) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    } else {
      f[i] = __uint_as_float(w[i]);
    }
  }
}
template <bool kBf16>
__device__ __forceinline__ uint4 pack(const float (&f)[kBf16 ? 8 : 4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kBf16)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    else
      w[i] = __float_as_uint(f[i]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One CTA per token: y = sum_j w_j rows[row_j], j ascending, in FP32, rounded
// once.  A slot without a row is skipped, so what its row might hold (or
// what its weight is) does not matter.  Four rows are read before the first
// is added; memory-bound.
template <bool kBf16>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(const uint4* rows, uint4* y, TokenArgs a, int vecs) {
  constexpr int kN = kBf16 ? 8 : 4;
  __shared__ int64_t start[64];  // of each kept row, in vectors
  __shared__ float weight[64];
  grid_begin();
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    // the kept slots, in order
    __syncthreads();
    int kept = 0;
    for (int j0 = 0; j0 < a.topk; j0 += 32) {  // every warp looks, so that every thread knows how many
      const int j = j0 + (threadIdx.x & 31);
      const int r = j < a.topk ? a.row_of_slot[t * a.topk + j] : -1;
      const bool there = r >= 0 && r < a.rows;
      const unsigned m = __ballot_sync(0xFFFFFFFFu, there);
      if (there && threadIdx.x < 32) {
        const int at = kept + __popc(m & ((1u << threadIdx.x) - 1u));
        start[at] = (int64_t)r * vecs;
        weight[at] = a.weights ? a.weights[t * a.topk + j] : 1.0f;
      }
      kept += __popc(m);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < vecs; i += kRowThreads) {
      float acc[kN] = {};
      for (int j0 = 0; j0 < kept; j0 += 4) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j0 + j < kept) v[j] = __ldcs(rows + start[j0 + j] + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j0 + j >= kept) break;
          const float w = weight[j0 + j];
          float f[kN];
          unpack<kBf16>(v[j], f);
#pragma unroll
          for (int c = 0; c < kN; ++c) acc[c] = __fmaf_rn(w, f[c], acc[c]);
        }
      }
      __stcs(y + t * vecs + i, pack<kBf16>(acc));
    }
  }
}

// One CTA per token, one pass: dy_t is read once per four of its rows, each
// row gets w dy, and the dot products are summed per thread, then over the
// warp by halving distances, then over the warps in order.  CTAs past the
// tokens zero the rows that have no slot.
template <bool kBf16>
__global__ void __launch_bounds__(kRowThreads) combine_grad_kernel(const uint4* dy, const uint4* rows, uint4* drows,
                                                                   float* dweights, TokenArgs a, int vecs) {
  constexpr int kN = kBf16 ? 8 : 4;
  __shared__ float part[kRowThreads / 32][4];
  grid_begin();
  if (blockIdx.x >= a.tokens) {
    const int64_t r0 = (blockIdx.x - a.tokens) * 32;
    const bool there = r0 + (threadIdx.x & 31) < a.rows;  // (a lane past the rows has none to zero)
    const int mine = there ? a.slot_of_row[r0 + (threadIdx.x & 31)] : 0;
    unsigned empty = __ballot_sync(0xFFFFFFFFu, there && (mine < 0 || mine >= a.tokens * a.topk));
    for (; empty; empty &= empty - 1) {
      uint4* dst = drows + (r0 + __ffs(empty) - 1) * vecs;
      for (int i = threadIdx.x; i < vecs; i += kRowThreads) __stcs(dst + i, make_uint4(0, 0, 0, 0));
    }
    return;
  }
  const int64_t t = blockIdx.x;
  const int32_t* at = a.row_of_slot + t * a.topk;
  for (int j0 = 0; j0 < a.topk; j0 += 4) {
    int r[4];
    float w[4], dot[4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r[j] = j0 + j < a.topk ? at[j0 + j] : -1;
      if (r[j] >= a.rows) r[j] = -1;
      w[j] = a.weights && j0 + j < a.topk ? a.weights[t * a.topk + j0 + j] : 1.0f;
    }
    for (int i = threadIdx.x; i < vecs; i += kRowThreads) {
      float g[kN];
      uint4 v[4];
      unpack<kBf16>(dy[t * vecs + i], g);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (r[j] >= 0) v[j] = __ldcs(rows + (int64_t)r[j] * vecs + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (r[j] < 0) continue;
        float f[kN], d[kN];
        unpack<kBf16>(v[j], f);
#pragma unroll
        for (int c = 0; c < kN; ++c) {
          dot[j] = __fmaf_rn(g[c], f[c], dot[j]);
          d[c] = __fmul_rn(w[j], g[c]);
        }
        __stcs(drows + (int64_t)r[j] * vecs + i, pack<kBf16>(d));
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) dot[j] = __fadd_rn(dot[j], __shfl_xor_sync(0xFFFFFFFFu, dot[j], d));
      if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < 4 && j0 + (int)threadIdx.x < a.topk && dweights != nullptr) {
      float sum = part[0][threadIdx.x];
      for (int i = 1; i < kRowThreads / 32; ++i) sum = __fadd_rn(sum, part[i][threadIdx.x]);
      dweights[t * a.topk + j0 + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

int64_t chunk_of(int64_t slots, int sms) {
  const int64_t c = (slots + sms - 1) / sms;
  const int64_t unit = 32 * kSortWarps;  // whole warps' runs
  return c <= kSortChunk ? kSortChunk : (c + unit - 1) / unit * unit;
}

}  // namespace

int sort_chunks(int64_t slots, const LaunchCtx& ctx) {
  const int64_t c = chunk_of(slots, ctx.num_sms);
  const int64_t n = (slots + c - 1) / c;
  return n < 1 ? 1 : (int)n;
}

// Enough for any number of SMs: chunks hold at least kSortChunk slots.
int64_t sort_scratch_ints(int64_t slots, int experts) {
  const int64_t n = (slots + kSortChunk - 1) / kSortChunk;
  return n <= 1 ? 0 : n * experts;
}

namespace {
int sort_smem(int experts, int64_t map) { return (int)sizeof(int) * ((kSortWarps + 3) * experts + 1 + (int)map); }
}  // namespace

cudaError_t launch_sort_tokens(const SortArgs& args, const LaunchCtx& ctx) {
  SortArgs a = args;
  int64_t chunk = chunk_of(a.slots, ctx.num_sms), row_bytes = 0;
  const int n = sort_chunks(a.slots, ctx);
  const int smem = sort_smem(a.experts, 0);
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(&sort_place_kernel<false>), sort_smem(kMaxExperts, 0), allowed);
  if (e != cudaSuccess) return e;
  const uint8_t* x = nullptr;
  uint8_t* out = nullptr;
  int topk = 1;
  void* p[] = {&a, &chunk, &x, &out, &row_bytes, &topk};
  if (n > 1 && (e = launch_dependent(reinterpret_cast<const void*>(&sort_count_kernel), dim3(n), dim3(kSortThreads),
                               sizeof(int) * a.experts, ctx.stream, p)) != cudaSuccess)  // (its two arguments come first)
    return e;
  return launch_dependent(reinterpret_cast<const void*>(&sort_place_kernel<false>), dim3(n), dim3(kSortThreads), smem,
                    ctx.stream, p);
}

cudaError_t launch_dispatch_tokens(const SortArgs& s, const void* x, void* out, const TokenArgs& t,
                                   const LaunchCtx& ctx) {
  // Few slots and rows: one launch (1024 tokens of 4096 BF16, top 2, 8 experts: 6.6
  // us against 7.9 in two; of 1024, 32 experts, members of 128: 7.6 against 10.2;
  // 8 tokens: 3.3 us).  The warps hold the ids of 2048 slots between the two walks.
  const int64_t row_bytes = t.width * (t.bf16 ? 2 : 4);
  if (s.slots > kSortChunk || s.rows > kCopyRows || row_bytes == 0) {
    const cudaError_t e = launch_sort_tokens(s, ctx);
    return e != cudaSuccess ? e : launch_gather_tokens(x, out, t, ctx);
  }
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e =
      allow_smem(reinterpret_cast<const void*>(&sort_place_kernel<true>), sort_smem(kMaxExperts, kCopyRows), allowed);
  if (e != cudaSuccess) return e;
  const int64_t units = s.rows * ((row_bytes + kCopyPiece - 1) / kCopyPiece);
  const int64_t want = (units + kSortWarps - 1) / kSortWarps;
  const unsigned grid = (unsigned)(want < 1 ? 1 : want < ctx.num_sms ? want : ctx.num_sms);
  SortArgs sort = s;
  int64_t chunk = (s.slots + 32 * kSortWarps - 1) / (32 * kSortWarps) * (32 * kSortWarps), bytes = row_bytes;
  const uint8_t* src = static_cast<const uint8_t*>(x);
  uint8_t* dst = static_cast<uint8_t*>(out);
  int topk = t.topk;
  void* p[] = {&sort, &chunk, &src, &dst, &bytes, &topk};
  return launch_dependent(reinterpret_cast<const void*>(&sort_place_kernel<true>), dim3(grid), dim3(kSortThreads),
                    sort_smem(s.experts, s.rows), ctx.stream, p);
}

cudaError_t launch_gather_tokens(const void* x, void* out, const TokenArgs& args, const LaunchCtx& ctx) {
  TokenArgs a = args;
  if (a.rows == 0 || a.width == 0) return cudaSuccess;
  int64_t row_bytes = a.width * (a.bf16 ? 2 : 4);
  const uint8_t* xv = static_cast<const uint8_t*>(x);
  uint8_t* ov = static_cast<uint8_t*>(out);
  // every warp has a piece to copy, or rows to look at
  const int64_t items = a.tokens * ((row_bytes + kPiece - 1) / kPiece), looks = (a.rows + kZeroRows - 1) / kZeroRows;
  const int64_t want = ((items > looks ? items : looks) + kGatherWarps - 1) / kGatherWarps;
  void* p[] = {&xv, &ov, &a, &row_bytes};
  return launch_dependent(reinterpret_cast<const void*>(&gather_kernel),
                          dim3((unsigned)(want < (1 << 30) ? want : (1 << 30))), dim3(32 * kGatherWarps), 0, ctx.stream, p);
}

cudaError_t launch_combine_tokens(const void* rows, void* y, const TokenArgs& args, const LaunchCtx& ctx) {
  TokenArgs a = args;
  if (a.tokens == 0 || a.width == 0) return cudaSuccess;
  int vecs = (int)(a.width * (a.bf16 ? 2 : 4) / 16);
  const unsigned grid = (unsigned)(a.tokens < (1 << 30) ? a.tokens : (1 << 30));
  void* p[] = {&rows, &y, &a, &vecs};
  return launch_dependent(a.bf16 ? reinterpret_cast<const void*>(&combine_kernel<true>)
                           : reinterpret_cast<const void*>(&combine_kernel<false>),
                    dim3(grid), dim3(kRowThreads), 0, ctx.stream, p);
}

cudaError_t launch_combine_tokens_grad(const void* dy, const void* rows, void* drows, float* dweights,
                                       const TokenArgs& args, const LaunchCtx& ctx) {
  TokenArgs a = args;
  int vecs = (int)(a.width * (a.bf16 ? 2 : 4) / 16);
  const int64_t grid = a.tokens + (vecs > 0 ? (a.rows + 31) / 32 : 0);
  if (grid == 0) return cudaSuccess;
  void* p[] = {&dy, &rows, &drows, &dweights, &a, &vecs};
  return launch_dependent(a.bf16 ? reinterpret_cast<const void*>(&combine_grad_kernel<true>)
                           : reinterpret_cast<const void*>(&combine_grad_kernel<false>),
                    dim3((unsigned)grid), dim3(kRowThreads), 0, ctx.stream, p);
}

}  // namespace nvfp4
