// mxfp4_cast.cu -- the MXFP4 cast, rows and transposed columns in one pass, and
// its reading back.
//
// For a block of 32 elements with a = max|x|:  the scale is the power of two
// 2^(floor(log2 a) - 2), not below 2^-127, stored as its exponent + 127 (for a = 0:
// 0), and q = E2M1_rn_satfinite(x / scale); the quotient is exact, so a code
// is rounded once.  With a's FP32 exponent field E the stored byte is max(E - 2,
// 0) and the factor 1 / scale is the FP32 number with exponent field 254 - byte:
// 2 .. 254, always a normal number.  A block with an infinity or a NaN gets the
// byte 255 (NaN) and codes 0.  The column-wise output is the same cast of x
// transposed.
//
// A 128 x 128 tile holds whole blocks of both directions, so one CTA casts it
// from registers with one read of x: TMA brings the tile, a thread takes 8
// rows x 8 columns, a row's maxima meet over the four lanes of its block, a
// column's through shared memory, and the codes leave through shared memory by
// TMA, which also cuts off what lies past the edges.  The four scales of a row
// are one word of a 512-byte tile of the swizzled layout.
//
// Memory-bound: 2 or 4 bytes in and 17/32 of a byte per direction out for every
// element.  Both directions, swizzled scales: 8192 x 5120 BF16 21.9 us (5.85 TB/s,
// 88 % of what a copy reaches), 8192 x 8192 FP32 55.4 us (6.1 TB/s); rows alone, BF16
// 17.5 us (6.05 TB/s).  Compact scales of lines that are no multiple of four long
// cost 1.0 us at 2080 x 4128 FP32, of 12.2 us.  What the two directions of BF16 took
// longest was to unpack and scale each element twice, on the pipe that also rounds
// and compares; a multiply-add that takes BF16 halves does both on another (29.3 us
// without it).  Reading back, 8192 x 5120: 17 us, 6.2 TB/s.
#include "common.cuh"
#include "dependent.h"
#include "fp4.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;
constexpr int kCodeBytes = kTile * kTile / 2;

struct CastKernelArgs {
  int64_t M, N;
  int tiles_n;
  int64_t tiles;
  uint8_t* scale_row;
  uint8_t* scale_col;
  int swizzled;
  unsigned* status;
};

// CTAs of an SM: by shared memory, but for both directions of BF16 three by
// measurement (8192 x 5120: 21.9 us; four, of 64 registers a thread, 24.3).
template <bool kBf16, bool kBoth>
constexpr int kPerSm = kBf16 ? (kBoth ? 3 : 4) : 2;

template <bool kBf16>
struct Smem {
  static constexpr int kInBytes = kTile * kTile * (kBf16 ? 2 : 4);
  static constexpr int kBytes = 1024 + kInBytes + 2 * kCodeBytes;
};

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int32_t c0, int32_t c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(src)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
// Per BF16 half, the larger magnitude (its sign is of no use), or NaN.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Two maxima, each as the upper half of an FP32 number, -> the bytes of their
// scales in the halves of a word: max(E - 2, 0), and 255 for E = 255.
__device__ __forceinline__ uint32_t scale_bytes(uint32_t maxima) {
  const uint32_t e = (maxima >> 7) & 0x00FF00FFu;
  uint32_t b;
  asm("max.u16x2 %0, %1, %2;" : "=r"(b) : "r"(e), "r"(0x00020002u));
  return b - 0x00020002u + (((e + 0x00010001u) & 0x01000100u) >> 7);
}
__device__ __forceinline__ uint32_t byte_of(uint32_t bytes, int half) { return half ? bytes >> 16 : bytes & 0xFFFFu; }
// 1 / scale (of a block that is not finite: anything; its codes become 0).
__device__ __forceinline__ float encode_of(uint32_t byte) { return __uint_as_float(0x7F000000u - (byte << 23)); }
// Two values times two factors.
__device__ __forceinline__ void mul2(float& a, float& b, float x, float y, float f, float g) {
  asm("{\n .reg .b64 p, q;\n mov.b64 p, {%2, %3};\n mov.b64 q, {%4, %5};\n mul.rn.f32x2 p, p, q;\n mov.b64 {%0, %1}, p;\n}"
      : "=f"(a), "=f"(b)
      : "f"(x), "f"(y), "f"(f), "f"(g));
}

// Two BF16 values times the halves of f, exact in FP32 (adding -0 leaves a product as it is, a -0 too).
__device__ __forceinline__ void mul2(float& a, float& b, uint32_t x, uint32_t f) {
  asm("{\n .reg .b16 p, q, f, g;\n mov.b32 {p, q}, %2;\n mov.b32 {f, g}, %3;\n"
      " fma.rn.f32.bf16 %0, p, f, 0f80000000;\n fma.rn.f32.bf16 %1, q, g, 0f80000000;\n}"
      : "=f"(a), "=f"(b)
      : "r"(x), "r"(f));
}

// Four scales of line r (a row, or a column), blocks 4 t .. of C.
__device__ __forceinline__ void put_scales(uint8_t* base, int64_t r, int t, int64_t C, bool swizzled, uint32_t word) {
  const int64_t c = 4 * (int64_t)t;
  if (swizzled) {  // (whole tiles)
    *reinterpret_cast<uint32_t*>(base + swizzled_scale_offset(r, c, C)) = word;
    return;
  }
  uint8_t* p = base + r * C + c;
  const int n = (int)min((int64_t)4, C - c);
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 3);
  if (n == 4 && off == 0) {
    *reinterpret_cast<uint32_t*>(p) = word;
  } else if (n == 4 && off == 2) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)word;
    *reinterpret_cast<uint16_t*>(p + 2) = (uint16_t)(word >> 16);
  } else if (n == 4) {
    p[0] = (uint8_t)word;
    *reinterpret_cast<uint16_t*>(p + 1) = (uint16_t)(word >> 8);
    p[3] = (uint8_t)(word >> 24);
  } else {
    for (int i = 0; i < n; ++i) p[i] = (uint8_t)(word >> (8 * i));
  }
}

template <bool kBf16, bool kRow, bool kCol>
__global__ void __launch_bounds__(kThreads, (kPerSm<kBf16, kRow && kCol>))
mxfp4_cast_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap rmap,
                  const __grid_constant__ CUtensorMap cmap, const __grid_constant__ CastKernelArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full;
  __shared__ __align__(16) uint32_t col_max[kThreads / 32][kTile / 2];
  __shared__ __align__(16) uint8_t row_sc[4][kTile], col_sc[4][kTile];  // [block][line]
  const uint32_t in = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t out_row = in + Smem<kBf16>::kInBytes, out_col = out_row + kCodeBytes;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int g = lane & 15;             // columns 8 g .. 8 g + 7
  const int rg = 2 * w + (lane >> 4);  // rows 8 rg .. 8 rg + 7
  if (tid == 0) {
    mbar_init(&full, 1);
    fence_mbar_init();
    tma_prefetch_desc(&xmap);
    if (kRow) tma_prefetch_desc(&rmap);
    if (kCol) tma_prefetch_desc(&cmap);
  }
  grid_begin();
  __syncthreads();
  constexpr int kBox = kBf16 ? 64 : 32;  // columns of an input box (128 bytes)
  const uint64_t policy = l2_policy_evict_first();
  auto load = [&](int64_t t) {
    const int32_t m = (int32_t)(t / a.tiles_n) * kTile, n = (int32_t)(t % a.tiles_n) * kTile;
    mbar_arrive_expect_tx(&full, Smem<kBf16>::kInBytes);
#pragma unroll
    for (int k = 0; k < kTile / kBox; ++k)
      tma_load_2d(smem_raw + (in - smem_u32(smem_raw)) + k * kTile * 128, &xmap, n + k * kBox, m, &full, policy);
  };
  if (tid == 0 && blockIdx.x < a.tiles) load(blockIdx.x);
  uint32_t phase = 0;
  for (int64_t t = blockIdx.x; t < a.tiles; t += gridDim.x) {
    const bool ok = mbar_wait_bounded(&full, phase, a.status);
    phase ^= 1;
    // 8 x 8 elements: BF16 in four words a row, FP32 in eight
    constexpr int kW = kBf16 ? 4 : 8;
    uint32_t x[8][kW];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 8 * rg + i;  // r & 7 == i
      if constexpr (kBf16) {
        const uint4 v = lds128(in + (g >> 3) * (kTile * 128) + r * 128 + (((g & 7) ^ i) * 16));
        x[i][0] = v.x; x[i][1] = v.y; x[i][2] = v.z; x[i][3] = v.w;
      } else {
        // the two halves in either order, so that eight lanes touch eight different 16-byte places
        const uint32_t row = in + (g >> 2) * (kTile * 128) + r * 128;
        const int odd = (g >> 2) & 1;
        const uint4 p = lds128(row + (((2 * (g & 3) + odd) ^ i) * 16));
        const uint4 q = lds128(row + (((2 * (g & 3) + 1 - odd) ^ i) * 16));
        x[i][0] = odd ? q.x : p.x; x[i][1] = odd ? q.y : p.y; x[i][2] = odd ? q.z : p.z; x[i][3] = odd ? q.w : p.w;
        x[i][4] = odd ? p.x : q.x; x[i][5] = odd ? p.y : q.y; x[i][6] = odd ? p.z : q.z; x[i][7] = odd ? p.w : q.w;
      }
    }
    // everyone has its elements, and (below) the previous codes are stored
    if (tid == 0) bulk_wait_read_all();
    if (!__syncthreads_and(ok)) break;
    if (tid == 0 && t + gridDim.x < a.tiles) load(t + gridDim.x);
    const int tm = (int)(t / a.tiles_n), tn = (int)(t % a.tiles_n);
    const int64_t m0 = (int64_t)tm * kTile, n0 = (int64_t)tn * kTile;

    // Maxima of the thread's rows (then over the four lanes of a block) and
    // columns (over 16 rows), two to a word, as the upper halves of FP32 numbers.
    uint32_t rm[4], cm[4] = {0, 0, 0, 0};
    if constexpr (kBf16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (kRow) m = larger(m, x[i][k]);
          if (kCol) cm[k] = larger(cm[k], x[i][k]);
        }
        // the larger half of rows i and i + 1 side by side in one word
        m = larger(m, __byte_perm(m, m, 0x1032));
        if (i & 1) rm[i >> 1] = __byte_perm(rm[i >> 1], m, 0x5410); else rm[i >> 1] = m;
      }
    } else {
      float r[8], c[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) c[k] = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float v = __uint_as_float(x[i][k]);
          if (kRow) r[i] = larger(r[i], v);
          if (kCol) c[k] = larger(c[k], v);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        rm[k] = __byte_perm(__float_as_uint(r[2 * k]), __float_as_uint(r[2 * k + 1]), 0x7632);
        cm[k] = __byte_perm(__float_as_uint(c[2 * k]), __float_as_uint(c[2 * k + 1]), 0x7632);
      }
    }
    uint32_t rs[4], cs[4];  // the scale bytes of rows / columns 2 k, 2 k + 1
    if constexpr (kRow) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        rm[k] = larger(rm[k], __shfl_xor_sync(0xFFFFFFFFu, rm[k], 1));
        rm[k] = larger(rm[k], __shfl_xor_sync(0xFFFFFFFFu, rm[k], 2));
        rs[k] = scale_bytes(rm[k]);
      }
      if ((g & 3) == 0)
        *reinterpret_cast<uint2*>(&row_sc[g >> 2][8 * rg]) =
            make_uint2(__byte_perm(rs[0], rs[1], 0x6420), __byte_perm(rs[2], rs[3], 0x6420));
    }
    if constexpr (kCol) {
#pragma unroll
      for (int k = 0; k < 4; ++k) cm[k] = larger(cm[k], __shfl_xor_sync(0xFFFFFFFFu, cm[k], 16));
      if (lane < 16) *reinterpret_cast<uint4*>(&col_max[w][4 * g]) = make_uint4(cm[0], cm[1], cm[2], cm[3]);
    }
    __syncthreads();
    if constexpr (kCol) {  // the maxima of two warps make a block of 32 rows
      const uint4 u = *reinterpret_cast<const uint4*>(&col_max[w & ~1][4 * g]);
      const uint4 v = *reinterpret_cast<const uint4*>(&col_max[w | 1][4 * g]);
      cs[0] = scale_bytes(larger(u.x, v.x)), cs[1] = scale_bytes(larger(u.y, v.y));
      cs[2] = scale_bytes(larger(u.z, v.z)), cs[3] = scale_bytes(larger(u.w, v.w));
      if (lane < 16 && (w & 1) == 0)
        *reinterpret_cast<uint2*>(&col_sc[w >> 1][8 * g]) =
            make_uint2(__byte_perm(cs[0], cs[1], 0x6420), __byte_perm(cs[2], cs[3], 0x6420));
    }
    // Columns k and k + 1 of a row times the factors of their blocks, whose scales' bytes are the halves of a word.
    auto scaled = [&](float& u, float& v, int i, int k, uint32_t bytes) {
      if constexpr (kBf16)
        mul2(u, v, x[i][k >> 1], (0x01FE01FEu - bytes) << 7 & 0x7F807F80u);
      else
        mul2(u, v, __uint_as_float(x[i][k]), __uint_as_float(x[i][k + 1]), encode_of(byte_of(bytes, 0)),
             encode_of(byte_of(bytes, 1)));
    };
    auto any_bad = [](const uint32_t (&b)[4]) {  // a block that is not finite
      uint32_t e = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) e |= b[k] + 0x00010001u;
      return (e & 0x01000100u) != 0;
    };
    // Rows of 64 bytes; 16-byte places swizzled by bits 1 and 2 of the row, as TMA expects them.
    if constexpr (kRow) {
      uint32_t q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t both = __byte_perm(rs[i >> 1], 0, i & 1 ? 0x4242 : 0x4040);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; k += 2) scaled(v[k], v[k + 1], i, k, both);
        q[i] = e2m1x8(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
      }
      if (any_bad(rs))
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (byte_of(rs[i >> 1], i & 1) == 255u) q[i] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        sts_u32(out_row + (8 * rg + i) * 64 + (((g >> 2) ^ (i >> 1)) & 3) * 16 + (g & 3) * 4, q[i]);
    }
    if constexpr (kCol) {
      uint32_t c[8];
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        float v[8], u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) scaled(v[i], u[i], i, k, cs[k >> 1]);
        c[k] = e2m1x8(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
        c[k + 1] = e2m1x8(u[0], u[1], u[2], u[3], u[4], u[5], u[6], u[7]);
      }
      if (any_bad(cs))
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (byte_of(cs[k >> 1], k & 1) == 255u) c[k] = 0;
      // Lane g stores its column k ^ (g & 7) in turn k (three rounds of swaps
      // arrange them), so that a turn's stores fall into different banks.
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) {
        const bool swap = g & d;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (!(k & d)) {
            const uint32_t p = c[k], q = c[k | d];
            c[k] = swap ? q : p;
            c[k | d] = swap ? p : q;
          }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int kk = k ^ (g & 7);  // column 8 g + kk, a row of the output
        sts_u32(out_col + (8 * g + kk) * 64 + (((rg >> 2) ^ (kk >> 1)) & 3) * 16 + (rg & 3) * 4, c[k]);
      }
    }
    fence_proxy_async_shared();
    __syncthreads();
    if (tid == 0) {
      if (kRow) tma_store_2d(&rmap, out_row, (int32_t)(n0 / 2), (int32_t)m0);
      if (kCol) tma_store_2d(&cmap, out_col, (int32_t)(m0 / 2), (int32_t)n0);
      bulk_commit();
    }
    // four bytes of a line, one from each block
    auto word = [](const uint8_t (&sc)[4][kTile], int line) {
      return (uint32_t)sc[0][line] | (uint32_t)sc[1][line] << 8 | (uint32_t)sc[2][line] << 16 | (uint32_t)sc[3][line] << 24;
    };
    if (tid < kTile) {
      if (kRow && m0 + tid < a.M) put_scales(a.scale_row, m0 + tid, tn, a.N / 32, a.swizzled, word(row_sc, tid));
    } else {
      const int c = tid - kTile;
      if (kCol && n0 + c < a.N) put_scales(a.scale_col, n0 + c, tm, a.M / 32, a.swizzled, word(col_sc, c));
    }
  }
  if (tid == 0) bulk_wait_all();
}

template <bool kBf16, bool kRow, bool kCol>
cudaError_t launch(const CUtensorMap& x, const CUtensorMap& r, const CUtensorMap& c, const CastKernelArgs& k,
                   const LaunchCtx& ctx) {
  const auto kernel = mxfp4_cast_kernel<kBf16, kRow, kCol>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), Smem<kBf16>::kBytes, allowed);
  if (e != cudaSuccess) return e;
  const int64_t room = (int64_t)ctx.num_sms * kPerSm<kBf16, kRow && kCol>;
  CUtensorMap maps[3] = {x, r, c};
  CastKernelArgs args = k;
  void* p[] = {&maps[0], &maps[1], &maps[2], &args};
  return launch_dependent(reinterpret_cast<const void*>(kernel), dim3((unsigned)(k.tiles < room ? k.tiles : room)),
                          dim3(kThreads), Smem<kBf16>::kBytes, ctx.stream, p);
}

template <bool kBf16>
cudaError_t launch_directions(const CUtensorMap& x, const CUtensorMap& r, const CUtensorMap& c, bool row, bool col,
                              const CastKernelArgs& k, const LaunchCtx& ctx) {
  if (row && col) return launch<kBf16, true, true>(x, r, c, k, ctx);
  if (row) return launch<kBf16, true, false>(x, r, c, k, ctx);
  return launch<kBf16, false, true>(x, r, c, k, ctx);
}

// The value of a scale byte: 2^(byte - 127), 255 NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}
// Eight codes -> their values times s.
__device__ __forceinline__ void decode8(uint32_t q, float s, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n .reg .b8 q0, q1, q2, q3;\n mov.b32 {q0, q1, q2, q3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, q0;\n cvt.rn.f16x2.e2m1x2 %1, q1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, q2;\n cvt.rn.f16x2.e2m1x2 %3, q3;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(q));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}"
        : "=f"(lo), "=f"(hi)
        : "r"(h[i]));
    v[2 * i] = __fmul_rn(lo, s);
    v[2 * i + 1] = __fmul_rn(hi, s);
  }
}

// A thread reads half a block, 8 bytes, and writes its 16 values.  (The operand may be
// written by the kernel before, beside which this one begins: nothing here is __restrict__.)
template <bool kOutBf16>
__global__ void __launch_bounds__(kThreads) mxfp4_dequantize_kernel(const uint8_t* data, const uint8_t* scale,
                                                                    int64_t halves, int64_t cols, int swizzled,
                                                                    void* out) {
  grid_begin();
  const int64_t per_row = cols / 16;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < halves; i += (int64_t)gridDim.x * kThreads) {
    const uint2 q = *reinterpret_cast<const uint2*>(data + 8 * i);
    int64_t at = i >> 1;
    if (swizzled) {
      const int64_t r = halves >> 32 ? i / per_row : (int64_t)((uint32_t)i / (uint32_t)per_row);
      at = swizzled_scale_offset(r, (i - r * per_row) >> 1, per_row >> 1);
    }
    const float s = scale_value(scale[at]);
    float v[16];
    decode8(q.x, s, *reinterpret_cast<float(*)[8]>(v));
    decode8(q.y, s, *reinterpret_cast<float(*)[8]>(v + 8));
    if constexpr (kOutBf16) {
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[k]) : "f"(v[2 * k + 1]), "f"(v[2 * k]));
      st_cs_v8(static_cast<uint8_t*>(out) + 32 * i, o);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(v[8 * h + k]);
        st_cs_v8(static_cast<uint8_t*>(out) + 64 * i + 32 * h, o);
      }
    }
  }
}

}  // namespace

cudaError_t launch_mxfp4_cast(const void* x, const MxCastArgs& a, const LaunchCtx& ctx) {
  if (a.M == 0 || a.N == 0) return cudaSuccess;
  CUtensorMap xm, rm = {}, cm = {};
  cudaError_t e = make_x_tensor_map(&xm, x, a.bf16, a.M, a.N);
  if (e == cudaSuccess && a.data_row) e = make_fp4_tensor_map(&rm, a.data_row, a.M, a.N / 2);
  if (e == cudaSuccess && a.data_col) e = make_fp4_tensor_map(&cm, a.data_col, a.N, a.M / 2);
  if (e != cudaSuccess) return e;
  CastKernelArgs k = {};
  k.M = a.M;
  k.N = a.N;
  k.tiles_n = (int)((a.N + kTile - 1) / kTile);
  k.tiles = (a.M + kTile - 1) / kTile * k.tiles_n;
  k.scale_row = a.scale_row;
  k.scale_col = a.scale_col;
  k.swizzled = a.swizzled;
  k.status = ctx.status;
  const bool row = a.data_row != nullptr, col = a.data_col != nullptr;
  return a.bf16 ? launch_directions<true>(xm, rm, cm, row, col, k, ctx)
                : launch_directions<false>(xm, rm, cm, row, col, k, ctx);
}

cudaError_t launch_mxfp4_dequantize(const uint8_t* data, const uint8_t* scale, int64_t rows, int64_t cols, bool swizzled,
                                    void* out, bool out_bf16, const LaunchCtx& ctx) {
  int64_t halves = rows * (cols / 16);
  if (halves == 0) return cudaSuccess;
  const int64_t want = (halves + kThreads - 1) / kThreads, most = (int64_t)ctx.num_sms * 16;
  const auto kernel = out_bf16 ? mxfp4_dequantize_kernel<true> : mxfp4_dequantize_kernel<false>;
  int sw = swizzled;
  void* args[] = {&data, &scale, &halves, &cols, &sw, &out};
  return launch_dependent(reinterpret_cast<const void*>(kernel), dim3((unsigned)(want < most ? want : most)),
                          dim3(kThreads), 0, ctx.stream, args);
}

}  // namespace nvfp4
