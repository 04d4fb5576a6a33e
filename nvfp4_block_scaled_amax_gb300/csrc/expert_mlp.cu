// expert_mlp.cu -- a layer of gated experts over 4-bit weights for a few
// tokens:
//     y[t] = sum_j gates[t][j] Wd[e] (silu(Wg[e] x[t]) * (Wu[e] x[t])),   e = ids[t][j],
// in two kernels of one body: the first gives the hidden values of every slot
// (t, j), the second multiplies them by Wd and adds a token's slots.
//
// With a few rows an expert the time is that of reading its weights once, so
// the weights stay 4 bits until they are in registers: each lane streams 16
// bytes (32 weights) of two weight rows at a time, four such loads ahead, and
// makes FP16 operands of them for mma.sync (16 weight rows x 8 tokens x 16):
// an E2M1 code times an E4M3 scale has six significant bits, so the NVFP4
// product is exact in FP16; MXFP4 codes are multiplied as they are, and the sum
// over a block is scaled in FP32, since powers of two may leave FP16's range.
// (tcgen05 has no product of 4-bit weights and 16-bit activations; the tensor
// cores are not what bounds this.)
//
// Activations are held in shared memory as FP16 scaled by a power of two for
// each row and each warp's share of the contracted dimension, so that their
// largest is in [2^14, 2^15): BF16 activations keep every bit down to 2^-31 of
// the largest, hidden values (FP32 between the kernels) are rounded to 11 bits,
// eight times finer than BF16's 8.  Sums, SiLU and the sum over slots are FP32.
//
// A CTA of 16 warps serves an even share of the items, an item being 16 weight
// rows of one expert for up to 8 kNT of its rows ("segment": an expert and
// such a group of rows).  ks warps share an item's contracted dimension and
// join their sums through shared memory in the order of the warps.  The second
// kernel writes each slot's weighted result; the CTA that completes a row tile
// for the last segment adds the tokens' slots in order, so the result does not
// depend on timing.
#include <cuda_fp16.h>

#include "common.cuh"
#include "dependent.h"
#include "fp4.h"
#include "tokens.h"

namespace nvfp4 {
namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kChunk = 128;   // weights of a row that four lanes take at a time
constexpr int kDepth = 4;     // such loads in flight
constexpr int kRedPitch = 20;  // floats of 16 rows in the joining buffer: the four lanes of a row meet other banks

struct KernelArgs {
  const uint16_t* x;      // first kernel: [tokens][width], BF16
  float* hidden;          // [slots][inner]: out of the first kernel, into the second
  const int32_t* ids;
  const float* gates;
  const uint8_t* data;    // [experts][rows][width / 2]
  const uint8_t* scale;
  const float* amax;
  int amax_per_expert;
  int slots, topk, experts;
  int width;              // contracted dimension
  int rows;               // weight rows of an expert
  int ks;                 // warps that share an item
  float* parts;           // second kernel: [slots][rows], weighted
  int* done;              // [row tiles] segments completed
  int num_tiles;          // row tiles of the second kernel
  uint16_t* y;            // [tokens][rows]
  int tokens;
};

__device__ __forceinline__ uint4 load_weights(const uint8_t* p, bool there) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (there)
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
  return v;
}
// Eight E2M1 codes -> four pairs in FP16.
__device__ __forceinline__ void to_f16(uint32_t q, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 q0, q1, q2, q3;\n mov.b32 {q0, q1, q2, q3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, q0;\n cvt.rn.f16x2.e2m1x2 %1, q1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, q2;\n cvt.rn.f16x2.e2m1x2 %3, q3;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(q));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ float power_of_two(uint32_t byte) {  // 2^(byte - 127), 255: NaN
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}
// Four words of four neighbouring lanes transposed: lane t's word i becomes word t of lane i.
__device__ __forceinline__ void transpose4(uint4& v, int t) {
  uint32_t a = t & 1 ? v.x : v.y, b = t & 1 ? v.z : v.w;  // to the neighbour
  a = __shfl_xor_sync(0xFFFFFFFFu, a, 1);
  b = __shfl_xor_sync(0xFFFFFFFFu, b, 1);
  if (t & 1) v.x = a, v.z = b; else v.y = a, v.w = b;
  a = t & 2 ? v.x : v.z, b = t & 2 ? v.y : v.w;
  a = __shfl_xor_sync(0xFFFFFFFFu, a, 2);
  b = __shfl_xor_sync(0xFFFFFFFFu, b, 2);
  if (t & 2) v.x = a, v.y = b; else v.z = a, v.w = b;
}

// Shared memory: activations [chunk][row][256 bytes], the joining buffers, and
// the slots sorted by expert.
template <int kNT>
struct Layout {
  static constexpr int kRows = 8 * kNT;  // rows of a segment
  static constexpr int kRedFloats = kRows * kRedPitch;  // of a warp
  static constexpr __host__ __device__ int chunks(int width) { return (width + kChunk - 1) / kChunk; }
  static constexpr __host__ __device__ int x_bytes(int width) { return chunks(width) * kRows * 2 * kChunk; }
  static constexpr int kRedBytes = 2 * kWarps * kRedFloats * 4;
  static constexpr int kScaleBytes = kWarps * kRows * 4;
  static constexpr __host__ __device__ int list_bytes(int slots, int experts) {
    return 4 * (2 * (experts + 1) + experts) + 4 * slots + 2 * ((slots + 1) & ~1) * 2;
  }
  static constexpr int bytes(int width, int slots, int experts, int tiles) {
    return x_bytes(width) + kRedBytes + kScaleBytes + list_bytes(slots, experts) + 4 * (tiles + 2);
  }
};

template <bool kDown, int kBlock, int kNT>
__global__ void __launch_bounds__(kThreads, 1) expert_mlp_kernel(const __grid_constant__ KernelArgs p) {
  using L = Layout<kNT>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int C = L::chunks(p.width);
  float* red = reinterpret_cast<float*>(smem + L::x_bytes(p.width));
  float* xinv = red + L::kRedBytes / 4;                 // [ks][rows of the segment]
  int* row0 = reinterpret_cast<int*>(xinv + kWarps * L::kRows);  // [experts + 1] first sorted slot
  int* seg0 = row0 + p.experts + 1;                     // [experts + 1] first segment
  int* count = seg0 + p.experts + 1;                    // [experts]
  int* ids = count + p.experts;                         // [slots]
  int* closed = ids + p.slots;                          // [tiles + 2]: how many, and which (second kernel)
  uint16_t* sorted = reinterpret_cast<uint16_t*>(closed + p.num_tiles + 2);  // [slots]
  uint16_t* place = sorted + ((p.slots + 1) & ~1);      // [slots] place within the expert
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t xs = smem_u32(smem);

  // The second kernel starts when all CTAs of the first are past this point, and
  // those are past everything before the first: what neither kernel writes may
  // be read ahead of its own wait.
  if (!kDown) {
    grid_dependency_wait();
    grid_launch_dependents();
  }

  // Slots by expert, in ascending order.
  for (int e = tid; e < p.experts; e += kThreads) count[e] = 0;
  for (int s = tid; s < p.slots; s += kThreads) {
    const int e = p.ids[s];
    ids[s] = e >= 0 && e < p.experts ? e : -1;
  }
  if (tid == 0) closed[0] = 0;
  __syncthreads();
  if (w == 0) {
    for (int base = 0; base < p.slots; base += 32) {
      const int s = base + lane, e = s < p.slots ? ids[s] : -1;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
      const int before = __popc(same & ((1u << lane) - 1));
      const int at = e >= 0 ? count[e] : 0;
      __syncwarp();
      if (e >= 0) {
        place[s] = (uint16_t)(at + before);
        if (before == 0) count[e] = at + __popc(same);
      }
      __syncwarp();
    }
    int rows = 0, segs = 0;
    for (int base = 0; base < p.experts; base += 32) {
      const int e = base + lane, n = e < p.experts ? count[e] : 0, m = (n + L::kRows - 1) / L::kRows;
      int rn = n, rm = m;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int un = __shfl_up_sync(0xFFFFFFFFu, rn, d), um = __shfl_up_sync(0xFFFFFFFFu, rm, d);
        if (lane >= d) rn += un, rm += um;
      }
      if (e < p.experts) row0[e] = rows + rn - n, seg0[e] = segs + rm - m;
      rows += __shfl_sync(0xFFFFFFFFu, rn, 31);
      segs += __shfl_sync(0xFFFFFFFFu, rm, 31);
    }
    if (lane == 0) row0[p.experts] = rows, seg0[p.experts] = segs;
  }
  __syncthreads();
  for (int s = tid; s < p.slots; s += kThreads)
    if (ids[s] >= 0) sorted[row0[ids[s]] + place[s]] = (uint16_t)s;
  const int segs = seg0[p.experts];
  const int tiles = p.rows / 16;  // items of a segment (first kernel: 8 gate rows and their up rows)
  const int64_t total = (int64_t)segs * tiles;
  const int i0 = (int)(total * blockIdx.x / gridDim.x), i1 = (int)(total * (blockIdx.x + 1) / gridDim.x);
  __syncthreads();

  // Expert of a segment.
  auto expert_of = [&](int seg) {
    int lo = 0, hi = p.experts;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (seg0[mid] <= seg) lo = mid; else hi = mid;
    }
    return lo;  // (the last of several with this first segment is the one that has it)
  };
  const int workers = kWarps / p.ks, worker = w / p.ks, k = w % p.ks;
  const int c0 = C * k / p.ks, c1 = C * (k + 1) / p.ks;
  // The worker's items: every `workers`-th of each segment's share of i0 .. i1.
  struct Cursor {
    int item, end, seg;  // end: of the segment's share
  };
  auto settle = [&](Cursor& c) {  // to the next segment while the share is used up; false at the end
    while (c.item >= c.end) {
      if (c.end >= i1) return false;
      c.item = c.end + worker;
      ++c.seg;
      c.end = min(i1, (c.seg + 1) * tiles);
    }
    return true;
  };
  const int first_seg = i0 / max(tiles, 1);
  Cursor ahead = {i0 + worker, min(i1, (first_seg + 1) * tiles), first_seg};
  if (i0 >= i1) ahead.end = i1;
  bool more = i0 < i1 && settle(ahead);
  int ac = c0;                     // the chunk to load next
  const uint8_t *wp[2], *sp[2];    // its weights and scales in the lane's two rows
  const int64_t pitch = p.width / 2, spitch = p.width / kBlock;
  auto aim = [&]() {
    if (!more) return;
    const int e = expert_of(ahead.seg), tile = ahead.item - ahead.seg * tiles;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t r = (int64_t)e * p.rows + (kDown ? 16 * tile + 8 * i : 8 * tile + i * (p.rows / 2)) + g;
      wp[i] = p.data + r * pitch + 16 * t + 64 * c0;
      sp[i] = p.scale + r * spitch + (kBlock == 16 ? 2 : 1) * (t + 4 * c0);
    }
    ac = c0;
  };
  uint4 ring[kDepth][2];
  uint32_t ring_s[kDepth][2];
  auto load = [&](uint4 (&q)[2], uint32_t (&s)[2]) {
    if (!more) return;
    const bool there = ac * kChunk + 32 * t < p.width;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      q[i] = load_weights(wp[i], there);
      if constexpr (kBlock == 16)
        s[i] = there ? __ldg(reinterpret_cast<const uint16_t*>(sp[i])) : 0u;
      else
        s[i] = there ? __ldg(sp[i]) : 0u;
      wp[i] += 64;
      sp[i] += kBlock == 16 ? 8 : 4;
    }
    if (++ac == c1) {
      ahead.item += workers;
      more = settle(ahead);
      aim();
    }
  };
  aim();
#pragma unroll
  for (int d = 0; d < kDepth; ++d) load(ring[d], ring_s[d]);

  if (kDown) {
    grid_dependency_wait();
    grid_launch_dependents();
  } else if (blockIdx.x == 0) {
    for (int i = tid; i < p.num_tiles; i += kThreads) p.done[i] = 0;
  }

  Cursor cur = {i1, i0, first_seg - 1};  // "before" the first segment
  int c = c1, ntok = 0, nt = 0, e = 0, first_row = 0, parity = 0;
  float factor = 1.0f;
  float acc[kNT][4];

  // The segment's activations into shared memory: a warp's share of a row at a time.
  auto load_x = [&]() {
    for (int q = w; q < ntok * p.ks; q += kWarps) {
      const int n = q / p.ks, part = q % p.ks;
      const int b0 = C * part / p.ks * (kChunk / 8), b1 = C * (part + 1) / p.ks * (kChunk / 8);  // pieces of 8 elements
      const int slot = sorted[first_row + n];
      float v[8];
      auto fetch = [&](int b) {
        if (8 * b >= p.width) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        } else if constexpr (kDown) {
          const float4* src = reinterpret_cast<const float4*>(p.hidden + (int64_t)slot * p.width + 8 * b);
          const float4 lo = __ldcg(src), hi = __ldcg(src + 1);
          v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
        } else {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)(slot / p.topk) * p.width + 8 * b));
          v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
          v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
        }
      };
      float m = 0.0f;
      for (int b = b0 + lane; b < b1; b += 32) {
        fetch(b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = fabsf(v[i]);
          m = a <= kFltMax ? fmaxf(m, a) : m;  // (an infinity or a NaN stays one whatever the others' scale)
        }
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
      // 2^s with s = 14 - floor(log2 m), at most 126 (m may be subnormal)
      const int up = m == 0.0f ? 0 : min(14 - ((int)(__float_as_uint(m) >> 23) - 127), 126);
      const float scale = __uint_as_float((uint32_t)(127 + up) << 23);
      if (lane == 0) xinv[part * L::kRows + n] = __uint_as_float((uint32_t)(127 - up) << 23);
      for (int b = b0 + lane; b < b1; b += 32) {
        fetch(b);
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm("cvt.rn.f16x2.f32 %0, %1, %2;"
              : "=r"(h[i])
              : "f"(__fmul_rn(v[2 * i + 1], scale)), "f"(__fmul_rn(v[2 * i], scale)));
        // Pieces in the order in which lanes 4 n .. 4 n + 3 read them together; odd rows half a line further.
        const int piece = b & 15;
        const int at = (kBlock == 16 ? (piece & 3) * 4 + (piece >> 2) : piece) ^ ((n & 1) * 4);
        sts_v4(xs + ((b >> 4) * L::kRows + n) * (2 * kChunk) + 16 * at, h[0], h[1], h[2], h[3]);
      }
    }
  };

  // The worker's sums of an item, joined; then what becomes of them.
  auto finish = [&]() {
    float* mine = red + (parity * kWarps + w) * L::kRedFloats;
#pragma unroll
    for (int i = 0; i < kNT; ++i)
      if (i < nt) {
        const int n = 8 * i + 2 * t;
        const float f0 = xinv[k * L::kRows + n], f1 = xinv[k * L::kRows + n + 1];
        mine[n * kRedPitch + g] = __fmul_rn(acc[i][0], f0);
        mine[(n + 1) * kRedPitch + g] = __fmul_rn(acc[i][1], f1);
        mine[n * kRedPitch + g + 8] = __fmul_rn(acc[i][2], f0);
        mine[(n + 1) * kRedPitch + g + 8] = __fmul_rn(acc[i][3], f1);
      }
    if (p.ks == 1)
      __syncwarp();
    else  // (at most eight workers then)
      asm volatile("bar.sync %0, %1;" ::"r"(1 + worker), "r"(32 * p.ks) : "memory");
    const float* all = red + (parity * kWarps + worker * p.ks) * L::kRedFloats;
    const int tile = cur.item - cur.seg * tiles;
    constexpr int kOut = kDown ? 16 : 8;
    for (int o = k * 32 + lane; o < ntok * kOut; o += 32 * p.ks) {
      const int n = o / kOut, r = o % kOut, slot = sorted[first_row + n];
      float a = 0.0f, b = 0.0f;
      for (int i = 0; i < p.ks; ++i) {
        a = __fadd_rn(a, all[i * L::kRedFloats + n * kRedPitch + r]);
        if (!kDown) b = __fadd_rn(b, all[i * L::kRedFloats + n * kRedPitch + r + 8]);
      }
      a = __fmul_rn(a, factor);
      if constexpr (kDown) {
        p.parts[(int64_t)slot * p.rows + 16 * tile + r] = __fmul_rn(a, p.gates[slot]);
      } else {
        b = __fmul_rn(b, factor);
        p.hidden[(int64_t)slot * (p.rows / 2) + 8 * tile + r] =
            __fmul_rn(__fdiv_rn(a, __fadd_rn(1.0f, expf(-a))), b);
      }
    }
    parity ^= 1;
  };

  // One chunk: its weights from the ring, 8 (kNT) MMAs.
  auto multiply = [&](uint4 (&q)[2], const uint32_t (&s)[2]) {
    const uint32_t xc = xs + (c * L::kRows + g) * (2 * kChunk);
    if constexpr (kBlock == 16) {
      uint32_t sc[2];  // two E4M3 scales as FP16
#pragma unroll
      for (int i = 0; i < 2; ++i) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(sc[i]) : "h"((uint16_t)s[i]));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t a[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          to_f16(j == 0 ? q[i].x : j == 1 ? q[i].y : j == 2 ? q[i].z : q[i].w, a[i]);
          const uint32_t both = __byte_perm(sc[i], sc[i], j < 2 ? 0x1010 : 0x3232);
#pragma unroll
          for (int h = 0; h < 4; ++h) a[i][h] = mul_f16x2(a[i][h], both);
        }
#pragma unroll
        for (int n = 0; n < kNT; ++n)
          if (n < nt) {
            const uint4 b = lds_v4(xc + n * 8 * (2 * kChunk) + 16 * ((4 * j + t) ^ ((g & 1) * 4)));
            mma_f16(acc[n], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
            mma_f16(acc[n], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
          }
      }
    } else {
      uint32_t sw[2];  // the chunk's four scales of each row
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        transpose4(q[i], t);
        sw[i] = s[i] << (8 * t);
        sw[i] |= __shfl_xor_sync(0xFFFFFFFFu, sw[i], 1);
        sw[i] |= __shfl_xor_sync(0xFFFFFFFFu, sw[i], 2);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t a[2][4];
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          to_f16(j == 0 ? q[i].x : j == 1 ? q[i].y : j == 2 ? q[i].z : q[i].w, a[i]);
          f[i] = power_of_two((sw[i] >> (8 * j)) & 255u);
        }
#pragma unroll
        for (int n = 0; n < kNT; ++n)
          if (n < nt) {
            const uint4 b = lds_v4(xc + n * 8 * (2 * kChunk) + 16 * ((4 * j + t) ^ ((g & 1) * 4)));
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_f16(d, a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
            mma_f16(d, a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = __fmaf_rn(d[i], f[i >> 1], acc[n][i]);
          }
      }
    }
  };

  auto step = [&](uint4 (&q)[2], uint32_t (&s)[2]) {
    if (c == c1) {  // the next item, and the next segments' activations on the way
      if (cur.end > i0) cur.item += workers;
      while (cur.item >= cur.end) {
        if (cur.end >= i1) return false;
        __syncthreads();
        cur.item = cur.end + worker;
        ++cur.seg;
        cur.end = min(i1, (cur.seg + 1) * tiles);
        e = expert_of(cur.seg);
        const int done = (cur.seg - seg0[e]) * L::kRows;
        first_row = row0[e] + done;
        ntok = min(L::kRows, row0[e + 1] - first_row);
        nt = (ntok + 7) / 8;
        factor = kBlock == 16 ? __fdiv_rn(p.amax[p.amax_per_expert ? e : 0], 2688.0f) : 1.0f;
        load_x();
        __syncthreads();
      }
      c = c0;
#pragma unroll
      for (int i = 0; i < kNT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    }
    multiply(q, s);
    load(q, s);
    if (++c == c1) finish();
    return true;
  };
  if (i0 < i1)
    while (step(ring[0], ring_s[0]) && step(ring[1], ring_s[1]) && step(ring[2], ring_s[2]) &&
           step(ring[3], ring_s[3])) {
    }

  if constexpr (kDown) {
    if (total == 0) {  // no slot is left: zeros
      for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < (int64_t)p.tokens * p.rows;
           i += (int64_t)gridDim.x * kThreads)
        p.y[i] = 0;
      return;
    }
    __syncthreads();
    // Row tiles that this CTA completes for the last segment.
    for (int i = i0 + tid; i < i1; i += kThreads) {
      __threadfence();
      const int tile = i % tiles;
      if (atomicAdd(&p.done[tile], 1) == segs - 1) closed[1 + atomicAdd(&closed[0], 1)] = tile;
    }
    __syncthreads();
    const int n = closed[0] * p.tokens;
    __threadfence();
    for (int q = tid; q < n * 16; q += kThreads) {
      const int token = (q >> 4) % p.tokens, at = 16 * closed[1 + (q >> 4) / p.tokens] + (q & 15);
      float sum = 0.0f;
      for (int j = 0; j < p.topk; ++j) {
        const int slot = token * p.topk + j;
        if (ids[slot] >= 0) sum = __fadd_rn(sum, __ldcg(p.parts + (int64_t)slot * p.rows + at));
      }
      uint16_t h;
      asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(sum));
      p.y[(int64_t)token * p.rows + at] = h;
    }
  }
}

// Warps that share an item: the split that keeps most warps busy, over the
// chunks of the contracted dimension and over the items.
int split_for(int width, int64_t items, int sms) {
  const int C = (width + kChunk - 1) / kChunk;
  int best = 1;
  double most = 0.0;
  for (int ks = 1; ks <= kWarps && ks <= C; ks *= 2) {
    const int64_t workers = (int64_t)sms * (kWarps / ks);
    const double by_items = (double)items / (double)((items + workers - 1) / workers * workers);
    const double by_chunks = (double)C / ((C + ks - 1) / ks * ks);
    const double all = by_items * by_chunks;
    if (all >= most * 0.98) {
      if (all > most) most = all;
      best = ks;
    }
  }
  return best;
}

template <bool kDown, int kBlock, int kNT>
cudaError_t launch(KernelArgs p, int64_t segments, const LaunchCtx& ctx) {
  const auto kernel = expert_mlp_kernel<kDown, kBlock, kNT>;
  static std::atomic<uint64_t> allowed{0};
  constexpr int kMost = 227 * 1024;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), kMost, allowed);
  if (e != cudaSuccess) return e;
  p.ks = split_for(p.width, segments * (p.rows / 16), ctx.num_sms);
  void* args[] = {&p};
  return launch_dependent(reinterpret_cast<const void*>(kernel), dim3((unsigned)ctx.num_sms), dim3(kThreads),
                          Layout<kNT>::bytes(p.width, p.slots, p.experts, p.num_tiles), ctx.stream, args);
}

// Rows of a segment: as many as the tokens, where shared memory holds them.
template <bool kDown, int kBlock>
cudaError_t launch_rows(const KernelArgs& p, int64_t experts_used, const LaunchCtx& ctx) {
  constexpr int kMost = 227 * 1024;
  auto fits = [&](int bytes) { return bytes <= kMost; };
  if (p.tokens > 16 && fits(Layout<4>::bytes(p.width, p.slots, p.experts, p.num_tiles)))
    return launch<kDown, kBlock, 4>(p, experts_used, ctx);
  if (p.tokens > 8 && fits(Layout<2>::bytes(p.width, p.slots, p.experts, p.num_tiles)))
    return launch<kDown, kBlock, 2>(p, experts_used, ctx);
  return launch<kDown, kBlock, 1>(p, experts_used, ctx);
}

}  // namespace

// One row tile's worth of rows always fits, whatever the call.
static_assert(Layout<1>::bytes(kMaxMlpWidth, kMaxMlpSlots, kMaxExperts, kMaxMlpWidth / 16) <= 227 * 1024,
              "shared memory of one CTA");

// The workspace: hidden values, weighted results, completion counts.
size_t expert_mlp_workspace(const ExpertMlpArgs& a) {
  return 4 * (size_t)(a.tokens * a.topk * (a.inner + a.hidden) + a.hidden / 16);
}

cudaError_t launch_expert_mlp(const ExpertMlpArgs& a, const LaunchCtx& ctx) {
  if (a.tokens == 0 || a.hidden == 0) return cudaSuccess;
  if (a.inner == 0) return cudaMemsetAsync(a.y, 0, (size_t)a.tokens * a.hidden * 2, ctx.stream);
  KernelArgs p = {};
  p.x = static_cast<const uint16_t*>(a.x);
  p.slots = (int)(a.tokens * a.topk);
  p.topk = a.topk;
  p.tokens = (int)a.tokens;
  p.experts = a.experts;
  p.ids = a.ids;
  p.gates = a.gates;
  p.hidden = static_cast<float*>(a.workspace);
  p.parts = p.hidden + (size_t)p.slots * a.inner;
  p.done = reinterpret_cast<int*>(p.parts + (size_t)p.slots * a.hidden);
  p.num_tiles = (int)(a.hidden / 16);
  p.y = static_cast<uint16_t*>(a.y);
  const int64_t used = p.slots < a.experts ? p.slots : a.experts;
  KernelArgs up = p, down = p;
  up.data = a.up.data, up.scale = a.up.scale, up.amax = a.up.amax, up.amax_per_expert = a.up.amax_per_row;
  up.width = (int)a.hidden, up.rows = (int)(2 * a.inner);
  down.data = a.down.data, down.scale = a.down.scale, down.amax = a.down.amax, down.amax_per_expert = a.down.amax_per_row;
  down.width = (int)a.inner, down.rows = (int)a.hidden;
  const cudaError_t e = a.block == 16 ? launch_rows<false, 16>(up, used, ctx) : launch_rows<false, 32>(up, used, ctx);
  if (e != cudaSuccess) return e;
  return a.block == 16 ? launch_rows<true, 16>(down, used, ctx) : launch_rows<true, 32>(down, used, ctx);
}

}  // namespace nvfp4
