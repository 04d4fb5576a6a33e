// expert_mlp.cuh -- what the kernels of the gated expert layer share:
// activations as sums of 4-bit operands (expert_mlp.cu says why), and partial
// results on their way through a cluster.
#pragma once

#include "fp4_tiles.cuh"
#include "tokens.h"

namespace nvfp4 {
namespace fp4 {

constexpr int kTerms = 8;

// ---------------------------------------------------------------------------
// Terms
// ---------------------------------------------------------------------------
// The sum of a row's terms, the smallest first.
__device__ __forceinline__ float add_terms(const uint32_t* v) {
  float sum = __uint_as_float(v[kTerms - 1]);
#pragma unroll
  for (int i = kTerms - 2; i >= 0; --i) sum = __fmaf_rn(sum, i == 0 ? 0.25f : 0.125f, __uint_as_float(v[i]));
  return sum;
}

// Four elements of a block into terms: put(i, codes) gets the four codes of each
// term i; the block's scale byte is returned.  The block lies in 4 (NVFP4) or 8
// (MXFP4) neighbouring lanes.
template <int kBlock, class Put>
__device__ __forceinline__ uint32_t to_terms(float (&v)[4], float unit, Put&& put) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v[j])));
#pragma unroll
  for (int d = 1; d < kBlock / 4; d <<= 1)
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(__shfl_xor_sync(0xFFFFFFFFu, m, d)));
  uint32_t byte;
  float value, inv;  // the scale, and its reciprocal (any rounding: what it leaves goes to the next term)
  if constexpr (kBlock == 16) {
    // the next E4M3 number not below a sixth of the largest; its value through FP16, which holds them all
    const float q = __fmul_rn(m, __fdividef(1.0f / 6.0f, unit));
    byte = e4m3_rn_satfinite(q);
    auto decoded = [](uint32_t c) {
      float f;
      asm("{\n .reg .b32 h;\n .reg .b16 lo, hi;\n cvt.rn.f16x2.e4m3x2 h, %1;\n mov.b32 {lo, hi}, h;\n cvt.f32.f16 %0, lo;\n}"
          : "=f"(f)
          : "h"((uint16_t)c));
      return f;
    };
    byte += byte < 126u && decoded(byte) < q;
    value = __fmul_rn(decoded(byte), unit);
    inv = byte == 0 ? 0.0f : __fdividef(1.0f, value);
    if (!(q <= 449.0f)) byte = 127u, inv = 0.0f;  // not finite: the whole row becomes NaN
  } else {
    // the next power of two not below a sixth of the largest (and 2^-105, so that no term's leaves FP32's range)
    const uint32_t bits = __float_as_uint(m), e = (bits >> 23) + ((bits & 0x7FFFFFu) > 0x400000u);
    byte = e < 24u ? 22u : e - 2u;
    value = __uint_as_float(byte << 23);
    inv = __uint_as_float((254u - byte) << 23);
    if (!(m <= kFltMax)) byte = 255u, inv = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kTerms; ++i) {
    uint16_t h;
    asm("{\n .reg .b8 lo, hi;\n"
        " cvt.rn.satfinite.e2m1x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 hi, %4, %3;\n"
        " mov.b16 %0, {lo, hi};\n}"
        : "=h"(h)
        : "f"(__fmul_rn(v[0], inv)), "f"(__fmul_rn(v[1], inv)), "f"(__fmul_rn(v[2], inv)), "f"(__fmul_rn(v[3], inv)));
    if (inv == 0.0f) h = 0;  // (an infinity times 0)
    put(i, h);
    float c[4];
    asm("{\n .reg .b8 lo, hi;\n .reg .b32 p, q;\n .reg .b16 a, b, c, d;\n mov.b16 {lo, hi}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 p, lo;\n cvt.rn.f16x2.e2m1x2 q, hi;\n mov.b32 {a, b}, p;\n mov.b32 {c, d}, q;\n"
        " cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n cvt.f32.f16 %2, c;\n cvt.f32.f16 %3, d;\n}"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "h"(h));
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __fmaf_rn(-c[j], value, v[j]);
    value = __fmul_rn(value, i == 0 ? 0.25f : 0.125f);
    inv = __fmul_rn(inv, i == 0 ? 4.0f : 8.0f);
  }
  return byte;
}

// The scale of the block of this element, at rows n0 .. of a segment's tiles (one
// for each term), by the lanes of the block.
template <int kBlock>
__device__ __forceinline__ void put_scale(uint8_t* segment, int n0, int64_t element, uint32_t byte) {
  constexpr int kLanes = kBlock / 4;
  uint8_t* tile = segment + element / (4 * kBlock) * kScaleTile + element % (4 * kBlock) / kBlock;
#pragma unroll
  for (int i = 0; i < kTerms; i += kLanes) {
    const int term = i + (threadIdx.x & (kLanes - 1)), n = n0 + term;
    if (term < kTerms) tile[n % 32 * 16 + n / 32 * 4] = (uint8_t)byte;
  }
}
// A number's magnitude, of what is not finite 0.
__device__ __forceinline__ float finite_magnitude(float v) {
  const float a = fabsf(v);
  return a <= kFltMax ? a : 0.0f;
}
// Power of two at which scales up to 448 reach a sixth of `largest` (and 2^-95: as above).
__device__ __forceinline__ float unit_of(float largest) {
  const int e = (int)(__float_as_uint(largest) >> 23) - 127;  // floor(log2)
  return __uint_as_float((uint32_t)(max(-95, e - 10) + 127) << 23);
}

__device__ __forceinline__ void store_async(uint32_t dst, float v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(dst),
               "r"(__float_as_uint(v)), "r"(bar)
               : "memory");
}

// The four writing warps meet, and stop together if one of them gave up waiting.
__device__ __forceinline__ bool together(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(all)
      : "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}

// expert_mlp_few.cu: the layer for one or two tokens, in two launches.
bool few_tokens(const ExpertMlpArgs& a, const LaunchCtx& ctx);
size_t few_tokens_workspace(const ExpertMlpArgs& a);
cudaError_t launch_few_tokens(const ExpertMlpArgs& a, const LaunchCtx& ctx);

}  // namespace fp4
}  // namespace nvfp4
