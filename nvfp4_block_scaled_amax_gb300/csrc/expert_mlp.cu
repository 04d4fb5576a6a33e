// expert_mlp.cu -- a layer of gated experts over 4-bit weights for a few
// tokens:
//     y[t] = sum_j gates[t][j] Wd[e] (silu(Wg[e] x[t]) * (Wu[e] x[t])),   e = ids[t][j],
// in two kernels of one body and a third that adds: the first gives the hidden values of every slot
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
// A CTA of 12 warps serves an even share of the items, an item being 32 weight
// rows of one expert for up to 8 kNT of its rows ("segment": an expert and
// such a group of rows).  ks warps share an item's contracted dimension and
// join their sums through shared memory in the order of the warps.  The second
// kernel writes each slot's weighted result, and a last one adds the tokens'
// slots in order, so that nothing depends on timing.
#include "common.cuh"
#include "dependent.h"
#include "fp4.h"
#include "tokens.h"

namespace nvfp4 {
namespace {

constexpr int kWarps = 12, kThreads = 32 * kWarps;
constexpr int kChunk = 128;   // weights of a row that four lanes take at a time
constexpr int kItemRows = 32;  // weight rows of an item: two MMA tiles (first kernel: 16 gate rows and their up rows)
constexpr int kRedPitch = 36;  // floats of 32 rows in the joining buffer: the four lanes of a row meet other banks

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

template <int kN>
struct Count {
  static constexpr int value = kN;
};

// Shared memory: activations [chunk][row][256 bytes], the joining buffer, and
// the slots sorted by expert.
template <int kNT>
struct Layout {
  static constexpr int kRows = 8 * kNT;  // rows of a segment
  static constexpr int kRedFloats = kRows * kRedPitch;  // of a warp
  static constexpr __host__ __device__ int chunks(int width) { return (width + kChunk - 1) / kChunk; }
  static constexpr __host__ __device__ int x_bytes(int width) { return chunks(width) * kRows * 2 * kChunk; }
  static constexpr int kRedBytes = kWarps * kRedFloats * 4;
  static constexpr int kScaleBytes = kWarps * kRows * 4;
  static constexpr __host__ __device__ int list_bytes(int slots, int experts) {
    return 4 * (2 * (experts + 1) + experts) + 4 * slots + 2 * ((slots + 1) & ~1) * 2;
  }
  static constexpr int bytes(int width, int slots, int experts) {
    return 256 + x_bytes(width) + kRedBytes + kScaleBytes + list_bytes(slots, experts);
  }
};

template <bool kDown, int kBlock, int kNT>
__global__ void __launch_bounds__(kThreads, 1) expert_mlp_kernel(const __grid_constant__ KernelArgs p) {
  using L = Layout<kNT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((256u - (smem_u32(smem_raw) & 255u)) & 255u);
  const int C = L::chunks(p.width);
  float* red = reinterpret_cast<float*>(smem + L::x_bytes(p.width));
  float* xinv = red + L::kRedBytes / 4;                 // [ks][rows of the segment]
  int* row0 = reinterpret_cast<int*>(xinv + kWarps * L::kRows);  // [experts + 1] first sorted slot
  int* seg0 = row0 + p.experts + 1;                     // [experts + 1] first segment
  int* count = seg0 + p.experts + 1;                    // [experts]
  int* ids = count + p.experts;                         // [slots]
  uint16_t* sorted = reinterpret_cast<uint16_t*>(ids + p.slots);  // [slots]
  uint16_t* place = sorted + ((p.slots + 1) & ~1);      // [slots] place within the expert
  const int tid = threadIdx.x, w = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t xs = smem_u32(smem);

  // The second kernel starts when all CTAs of the first are past this point, and
  // those are past everything before the first: what neither kernel writes may
  // be read ahead of its own wait.
  if (!kDown) {
    grid_dependency_wait();
    grid_launch_dependents();
  }

  // Slots by expert, in ascending order.
  for (int s = tid; s < p.slots; s += kThreads) {
    const int e = p.ids[s];
    ids[s] = e >= 0 && e < p.experts ? e : -1;
  }
  for (int e = tid; e < p.experts; e += kThreads) count[e] = 0;
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
  const int tiles = p.rows / kItemRows;  // items of a segment
  const int64_t total = (int64_t)segs * tiles;
  const int i0 = (int)(total * blockIdx.x / gridDim.x), i1 = (int)(total * (blockIdx.x + 1) / gridDim.x);
  if (i0 == i1) {
    grid_dependency_wait();
    grid_launch_dependents();
    return;
  }

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
  const int first_seg = i0 / tiles;

  // Loads run two chunks ahead.  The lane's rows of an item: g, and 8, 16, 24
  // further (first kernel: gate row g, its up row, and both 8 further).
  const int64_t pitch = p.width / 2, spitch = p.width / kBlock;
  const int64_t row1 = kDown ? 8 : p.rows / 2, row2 = kDown ? 16 : 8;
  const int item_rows = kDown ? kItemRows : kItemRows / 2;  // that the base row moves by
  int a_item = i0 + worker, a_seg = first_seg, a_end = min(i1, (first_seg + 1) * tiles), ac = c0;
  bool more = true;
  const uint8_t *wp = nullptr, *sp = nullptr;
  auto aim = [&]() {  // to the next segment while the share of this one is used up
    while (a_item >= a_end) {
      if (a_end >= i1) {
        more = false;
        return;
      }
      a_item = a_end + worker;
      ++a_seg;
      a_end = min(i1, (a_seg + 1) * tiles);
    }
    const int64_t r = (int64_t)expert_of(a_seg) * p.rows + (a_item - a_seg * tiles) * item_rows + g;
    wp = p.data + r * pitch + 16 * t + 64 * c0;
    sp = p.scale + r * spitch + (kBlock == 16 ? 2 : 1) * (t + 4 * c0);
  };
  const int64_t wstep = (int64_t)workers * item_rows * pitch - 64 * (c1 - c0);
  const int64_t sstep = (int64_t)workers * item_rows * spitch - (kBlock == 16 ? 8 : 4) * (c1 - c0);
  struct Chunk {
    uint4 q[4];
    uint32_t s[4];
  };
  auto load = [&](Chunk& d) {
    if (!more) return;
    const bool there = ac * kChunk + 32 * t < p.width;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = (i & 1 ? row1 : 0) + (i & 2 ? row2 : 0);
      d.q[i] = load_weights(wp + r * pitch, there);
      if constexpr (kBlock == 16)
        d.s[i] = there ? __ldg(reinterpret_cast<const uint16_t*>(sp + r * spitch)) : 0u;
      else
        d.s[i] = there ? __ldg(sp + r * spitch) : 0u;
    }
    wp += 64;
    sp += kBlock == 16 ? 8 : 4;
    if (++ac == c1) {
      ac = c0;
      a_item += workers;
      if (a_item < a_end) {
        wp += wstep;
        sp += sstep;
      } else {
        aim();
      }
    }
  };
  Chunk ring[2];
  aim();
  load(ring[0]);
  load(ring[1]);

  if (kDown) {
    grid_dependency_wait();
    grid_launch_dependents();
  }

  int item = i1, end = i0, seg = first_seg - 1;  // "before" the first segment
  int c = c1, ntok = 0, nt = 0, first_row = 0;
  float factor = 1.0f;
  float acc[2][kNT][4];

  // The segment's activations into shared memory: a warp's share of a row at a
  // time, kBatch pieces of 8 elements of a lane read at once.
  auto load_x = [&]() {
    constexpr int kBatch = kDown ? 2 : 4;
    for (int q = w; q < ntok * p.ks; q += kWarps) {
      const int n = q / p.ks, part = q % p.ks;
      const int b0 = C * part / p.ks * (kChunk / 8), b1 = C * (part + 1) / p.ks * (kChunk / 8);
      const int slot = sorted[first_row + n];
      uint4 u[kBatch][kDown ? 2 : 1];
      auto fetch = [&](int b) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int at = b + 32 * i;
          const bool there = at < b1 && 8 * at < p.width;
#pragma unroll
          for (int h = 0; h < (kDown ? 2 : 1); ++h) u[i][h] = make_uint4(0, 0, 0, 0);
          if (there) {
            if constexpr (kDown) {
              const uint4* src = reinterpret_cast<const uint4*>(p.hidden + (int64_t)slot * p.width + 8 * at);
              u[i][0] = __ldcg(src), u[i][1] = __ldcg(src + 1);
            } else {
              u[i][0] = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)(slot / p.topk) * p.width + 8 * at));
            }
          }
        }
      };
      auto unpack = [&](int i, float (&v)[8]) {
        if constexpr (kDown) {
          v[0] = __uint_as_float(u[i][0].x), v[1] = __uint_as_float(u[i][0].y), v[2] = __uint_as_float(u[i][0].z);
          v[3] = __uint_as_float(u[i][0].w), v[4] = __uint_as_float(u[i][1].x), v[5] = __uint_as_float(u[i][1].y);
          v[6] = __uint_as_float(u[i][1].z), v[7] = __uint_as_float(u[i][1].w);
        } else {
          v[0] = bf16_lo(u[i][0].x), v[1] = bf16_hi(u[i][0].x), v[2] = bf16_lo(u[i][0].y), v[3] = bf16_hi(u[i][0].y);
          v[4] = bf16_lo(u[i][0].z), v[5] = bf16_hi(u[i][0].z), v[6] = bf16_lo(u[i][0].w), v[7] = bf16_hi(u[i][0].w);
        }
      };
      float m = 0.0f;
      for (int b = b0 + lane; b < b1; b += 32 * kBatch) {
        fetch(b);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          float v[8];
          unpack(i, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float a = fabsf(v[j]);
            m = a <= kFltMax ? fmaxf(m, a) : m;  // (an infinity or a NaN stays one whatever the others' scale)
          }
        }
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
      // 2^s with s = 14 - floor(log2 m), at most 126 (m may be subnormal)
      const int up = m == 0.0f ? 0 : min(14 - ((int)(__float_as_uint(m) >> 23) - 127), 126);
      const float scale = __uint_as_float((uint32_t)(127 + up) << 23);
      if (lane == 0) xinv[part * L::kRows + n] = __uint_as_float((uint32_t)(127 - up) << 23);
      const bool again = b1 - b0 > 32 * kBatch;  // what was read last is not all of it
      for (int b = b0 + lane; b < b1; b += 32 * kBatch) {
        if (again) fetch(b);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int at = b + 32 * i;
          if (at >= b1) break;
          float v[8];
          unpack(i, v);
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            asm("cvt.rn.f16x2.f32 %0, %1, %2;"
                : "=r"(h[j])
                : "f"(__fmul_rn(v[2 * j + 1], scale)), "f"(__fmul_rn(v[2 * j], scale)));
          // Pieces in the order in which lanes 4 n .. 4 n + 3 read them together; odd rows half a line further.
          const int piece = at & 15;
          const int to = (kBlock == 16 ? (piece & 3) * 4 + (piece >> 2) : piece) ^ ((n & 1) * 4);
          sts_v4(xs + ((at >> 4) * L::kRows + n) * (2 * kChunk) + 16 * to, h[0], h[1], h[2], h[3]);
        }
      }
    }
  };

  auto join = [&]() {  // the warps of a worker meet
    if (p.ks == 1)
      __syncwarp();
    else  // (at most six workers then)
      asm volatile("bar.sync %0, %1;" ::"r"(1 + worker), "r"(32 * p.ks) : "memory");
  };
  // The worker's sums of an item, joined; then what becomes of them.
  auto finish = [&]() {
    join();  // the sums of the item before are read
    float* mine = red + w * L::kRedFloats;
#pragma unroll
    for (int i = 0; i < kNT; ++i)
      if (i < nt) {
        const int n = 8 * i + 2 * t;
        const float f0 = xinv[k * L::kRows + n], f1 = xinv[k * L::kRows + n + 1];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          float* to = mine + n * kRedPitch + 16 * m + g;
          to[0] = __fmul_rn(acc[m][i][0], f0);
          to[kRedPitch] = __fmul_rn(acc[m][i][1], f1);
          to[8] = __fmul_rn(acc[m][i][2], f0);
          to[kRedPitch + 8] = __fmul_rn(acc[m][i][3], f1);
        }
      }
    join();
    const float* all = red + worker * p.ks * L::kRedFloats;
    const int tile = item - seg * tiles;
    constexpr int kOut = kDown ? 32 : 16;
    for (int o = k * 32 + lane; o < ntok * kOut; o += 32 * p.ks) {
      const int n = o / kOut, r = o % kOut, slot = sorted[first_row + n];
      // (first kernel: gate and up rows alternate in eights)
      const float* from = all + n * kRedPitch + (kDown ? r : (r & 7) + 2 * (r & 8));
      float a = 0.0f, b = 0.0f;
      for (int i = 0; i < p.ks; ++i, from += L::kRedFloats) {
        a = __fadd_rn(a, from[0]);
        if (!kDown) b = __fadd_rn(b, from[8]);
      }
      a = __fmul_rn(a, factor);
      if constexpr (kDown) {
        p.parts[(int64_t)slot * p.rows + kItemRows * tile + r] = __fmul_rn(a, p.gates[slot]);
      } else {
        b = __fmul_rn(b, factor);
        p.hidden[(int64_t)slot * (p.rows / 2) + kItemRows / 2 * tile + r] =
            __fmul_rn(__fdiv_rn(a, __fadd_rn(1.0f, expf(-a))), b);
      }
    }
  };

  // One chunk of kN x 8 rows of activations: its weights from the ring, 16 kN MMAs.
  const uint32_t xl = xs + g * (2 * kChunk) + 16 * (t ^ ((g & 1) * 4));
  auto multiply = [&](Chunk& d, auto rows) {
    constexpr int kN = decltype(rows)::value;
    const uint32_t xc = xl + c * (L::kRows * 2 * kChunk);
    uint32_t sc[4];
    if constexpr (kBlock == 16) {  // two E4M3 scales as FP16
#pragma unroll
      for (int i = 0; i < 4; ++i) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(sc[i]) : "h"((uint16_t)d.s[i]));
    } else {  // the chunk's four scales of each row
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        transpose4(d.q[i], t);
        sc[i] = d.s[i] << (8 * t);
        sc[i] |= __shfl_xor_sync(0xFFFFFFFFu, sc[i], 1);
        sc[i] |= __shfl_xor_sync(0xFFFFFFFFu, sc[i], 2);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 b[kN];
#pragma unroll
      for (int n = 0; n < kN; ++n) b[n] = lds_v4((xc ^ (64 * j)) + n * 8 * (2 * kChunk));
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t a[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4& q = d.q[2 * m + i];
          to_f16(j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w, a[i]);
          if constexpr (kBlock == 16) {
            const uint32_t both = __byte_perm(sc[2 * m + i], 0, j < 2 ? 0x1010 : 0x3232);
#pragma unroll
            for (int h = 0; h < 4; ++h) a[i][h] = mul_f16x2(a[i][h], both);
          }
        }
        if constexpr (kBlock == 16) {
#pragma unroll
          for (int n = 0; n < kN; ++n) mma_f16(acc[m][n], a[0][0], a[1][0], a[0][1], a[1][1], b[n].x, b[n].y);
#pragma unroll
          for (int n = 0; n < kN; ++n) mma_f16(acc[m][n], a[0][2], a[1][2], a[0][3], a[1][3], b[n].z, b[n].w);
        } else {
          const float f0 = power_of_two((sc[2 * m] >> (8 * j)) & 255u);
          const float f1 = power_of_two((sc[2 * m + 1] >> (8 * j)) & 255u);
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_f16(v, a[0][0], a[1][0], a[0][1], a[1][1], b[n].x, b[n].y);
            mma_f16(v, a[0][2], a[1][2], a[0][3], a[1][3], b[n].z, b[n].w);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] = __fmaf_rn(v[i], i < 2 ? f0 : f1, acc[m][n][i]);
          }
        }
      }
    }
  };

  auto step = [&](Chunk& d) {
    if (c == c1) {  // the next item, and the next segments' activations on the way
      if (end > i0) item += workers;
      while (item >= end) {
        if (end >= i1) return false;
        __syncthreads();
        item = end + worker;
        ++seg;
        end = min(i1, (seg + 1) * tiles);
        const int e = expert_of(seg);
        first_row = row0[e] + (seg - seg0[e]) * L::kRows;
        ntok = min(L::kRows, row0[e + 1] - first_row);
        nt = (ntok + 7) / 8;
        factor = kBlock == 16 ? __fdiv_rn(p.amax[p.amax_per_expert ? e : 0], 2688.0f) : 1.0f;
        load_x();
        __syncthreads();
      }
      c = c0;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < kNT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[m][i][j] = 0.0f;
    }
    if (kNT == 1 || nt == 1)
      multiply(d, Count<1>());
    else if (kNT == 2 || nt == 2)
      multiply(d, Count<kNT == 1 ? 1 : 2>());
    else
      multiply(d, Count<kNT>());
    load(d);
    if (++c == c1) finish();
    return true;
  };
  while (step(ring[0]) && step(ring[1])) {
  }
}

// y[t] = the sum of a token's weighted results in the order of its choices.
__global__ void __launch_bounds__(256) join_slots_kernel(const float* __restrict__ parts, const int32_t* __restrict__ ids,
                                                         int topk, int experts, int rows, int tokens, uint16_t* y) {
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

// Warps that share an item: the split that keeps most warps busy, over the
// chunks of the contracted dimension and over the items.
int split_for(int width, int64_t items, int sms) {
  const int C = (width + kChunk - 1) / kChunk;
  int best = 1;
  double most = 0.0;
  for (int ks = 1; ks <= kWarps && ks <= C; ++ks) {
    if (kWarps % ks != 0) continue;
    const int64_t workers = (int64_t)sms * (kWarps / ks);
    const double by_items = (double)items / (double)((items + workers - 1) / workers * workers);
    const double by_chunks = (double)C / ((C + ks - 1) / ks * ks);
    if (by_items * by_chunks > most * 1.02) {
      most = by_items * by_chunks;
      best = ks;
    }
  }
  return best;
}

constexpr int kMostShared = 227 * 1024;

template <bool kDown, int kBlock, int kNT>
cudaError_t launch(KernelArgs p, int64_t segments, const LaunchCtx& ctx) {
  const auto kernel = expert_mlp_kernel<kDown, kBlock, kNT>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), kMostShared, allowed);
  if (e != cudaSuccess) return e;
  p.ks = split_for(p.width, segments * (p.rows / kItemRows), ctx.num_sms);
  void* args[] = {&p};
  return launch_dependent(reinterpret_cast<const void*>(kernel), dim3((unsigned)ctx.num_sms), dim3(kThreads),
                          Layout<kNT>::bytes(p.width, p.slots, p.experts), ctx.stream, args);
}

// Rows of a segment: as many as the tokens, where shared memory holds them.
template <bool kDown, int kBlock>
cudaError_t launch_rows(const KernelArgs& p, int64_t tokens, int64_t experts_used, const LaunchCtx& ctx) {
  if (tokens > 16 && Layout<4>::bytes(p.width, p.slots, p.experts) <= kMostShared)
    return launch<kDown, kBlock, 4>(p, experts_used, ctx);
  if (tokens > 8 && Layout<2>::bytes(p.width, p.slots, p.experts) <= kMostShared)
    return launch<kDown, kBlock, 2>(p, experts_used, ctx);
  return launch<kDown, kBlock, 1>(p, experts_used, ctx);
}

}  // namespace

// One row tile's worth of rows always fits, whatever the call.
static_assert(Layout<1>::bytes(kMaxMlpWidth, kMaxMlpSlots, kMaxExperts) <= kMostShared, "shared memory of one CTA");

// The workspace: hidden values and weighted results of every slot.
size_t expert_mlp_workspace(const ExpertMlpArgs& a) { return 4 * (size_t)(a.tokens * a.topk * (a.inner + a.hidden)); }

cudaError_t launch_expert_mlp(const ExpertMlpArgs& a, const LaunchCtx& ctx) {
  if (a.tokens == 0 || a.hidden == 0) return cudaSuccess;
  if (a.inner == 0) return cudaMemsetAsync(a.y, 0, (size_t)a.tokens * a.hidden * 2, ctx.stream);
  KernelArgs p = {};
  p.x = static_cast<const uint16_t*>(a.x);
  p.slots = (int)(a.tokens * a.topk);
  p.topk = a.topk;
  p.experts = a.experts;
  p.ids = a.ids;
  p.gates = a.gates;
  p.hidden = static_cast<float*>(a.workspace);
  p.parts = p.hidden + (size_t)p.slots * a.inner;
  const int64_t used = p.slots < a.experts ? p.slots : a.experts;
  KernelArgs up = p, down = p;
  up.data = a.up.data, up.scale = a.up.scale, up.amax = a.up.amax, up.amax_per_expert = a.up.amax_per_row;
  up.width = (int)a.hidden, up.rows = (int)(2 * a.inner);
  down.data = a.down.data, down.scale = a.down.scale, down.amax = a.down.amax, down.amax_per_expert = a.down.amax_per_row;
  down.width = (int)a.inner, down.rows = (int)a.hidden;
  cudaError_t e = a.block == 16 ? launch_rows<false, 16>(up, a.tokens, used, ctx)
                                : launch_rows<false, 32>(up, a.tokens, used, ctx);
  if (e != cudaSuccess) return e;
  e = a.block == 16 ? launch_rows<true, 16>(down, a.tokens, used, ctx) : launch_rows<true, 32>(down, a.tokens, used, ctx);
  if (e != cudaSuccess) return e;
  int rows = down.rows, tokens = (int)a.tokens;
  const int64_t want = ((int64_t)tokens * rows / 4 + 255) / 256;
  void* y = a.y;
  void* args[] = {&p.parts, &p.ids, &p.topk, &p.experts, &rows, &tokens, &y};
  return launch_dependent(reinterpret_cast<const void*>(join_slots_kernel),
                          dim3((unsigned)(want < 8 * ctx.num_sms ? want : 8 * ctx.num_sms)), dim3(256), 0, ctx.stream, args);
}

}  // namespace nvfp4
