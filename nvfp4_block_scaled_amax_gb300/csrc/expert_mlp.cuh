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
// Four elements of a block into terms: v is left with the remainders.  The
// block lies in 4 (NVFP4) or 8 (MXFP4) neighbouring lanes.  codes[i]: four codes
// of term i; scales: byte i the scale of term i.
template <int kBlock>
__device__ __forceinline__ void to_terms(float (&v)[4], float unit, uint32_t (&codes)[kTerms], uint32_t (&scales)[2]) {
  scales[0] = scales[1] = 0;
  float inv_unit6 = __fdiv_rn(1.0f / 6.0f, unit);
#pragma unroll
  for (int i = 0; i < kTerms; ++i) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = fabsf(v[j]);
      m = a >= m ? a : a != a ? __int_as_float(0x7F800000) : m;  // (a NaN counts as an infinity)
    }
#pragma unroll
    for (int d = 1; d < kBlock / 4; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    uint32_t byte;
    float value, inv;  // the scale, and its reciprocal (any rounding: what it leaves goes to the next term)
    if constexpr (kBlock == 16) {
      const float q = __fmul_rn(m, inv_unit6);
      byte = e4m3_rn_satfinite(q);
      if (byte < 126u && e4m3_decode(byte) < q) ++byte;
      value = __fmul_rn(e4m3_decode(byte), unit);
      inv = byte == 0 ? 0.0f : __fdividef(1.0f, value);
      unit = __fmul_rn(unit, 0.25f);
      inv_unit6 = __fmul_rn(inv_unit6, 4.0f);
      if (!(q <= 449.0f)) byte = 127u;  // not finite: the whole row becomes NaN
    } else {
      const uint32_t e = __float_as_uint(m) >> 23;
      byte = e < 2u ? 0u : e - 2u;
      value = __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
      inv = __uint_as_float((254u - byte) << 23);
      if (!(m <= kFltMax)) byte = 255u;
    }
    if (!(m <= kFltMax)) inv = 0.0f;
    uint16_t h;
    asm("{\n .reg .b8 lo, hi;\n"
        " cvt.rn.satfinite.e2m1x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 hi, %4, %3;\n"
        " mov.b16 %0, {lo, hi};\n}"
        : "=h"(h)
        : "f"(__fmul_rn(v[0], inv)), "f"(__fmul_rn(v[1], inv)), "f"(__fmul_rn(v[2], inv)), "f"(__fmul_rn(v[3], inv)));
    if (inv == 0.0f) h = 0;  // (an infinity times 0)
    codes[i] = h;
    scales[i >> 2] |= byte << (8 * (i & 3));
    uint32_t f01, f23;
    asm("{\n .reg .b8 lo, hi;\n mov.b16 {lo, hi}, %2;\n cvt.rn.f16x2.e2m1x2 %0, lo;\n cvt.rn.f16x2.e2m1x2 %1, hi;\n}"
        : "=r"(f01), "=r"(f23)
        : "h"(h));
    float c[4];
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}"
        : "=f"(c[0]), "=f"(c[1])
        : "r"(f01));
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}"
        : "=f"(c[2]), "=f"(c[3])
        : "r"(f23));
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __fmaf_rn(-c[j], value, v[j]);
  }
}

// Their places: four codes of each term in rows of `pitch` bytes, and the
// lane's share of the block's scales (row n0 + i of a segment is term i).
template <int kBlock>
__device__ __forceinline__ void store_codes(uint8_t* row, int64_t pitch, int64_t element, const uint32_t (&codes)[kTerms]) {
#pragma unroll
  for (int i = 0; i < kTerms; ++i)
    *reinterpret_cast<uint16_t*>(row + i * pitch + element / 2) = (uint16_t)codes[i];
}
template <int kBlock>
__device__ __forceinline__ void store_scales(uint8_t* segment, int n0, int64_t element, int lane,
                                             const uint32_t (&scales)[2]) {
  constexpr int kLanes = kBlock / 4, kEach = kTerms / kLanes;
  uint8_t* tile = segment + element / (4 * kBlock) * kScaleTile + element % (4 * kBlock) / kBlock;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int term = (lane % kLanes) * kEach + i, n = n0 + term;
    tile[n % 32 * 16 + n / 32 * 4] = (uint8_t)(scales[term >> 2] >> (8 * (term & 3)));
  }
}
// Power of two at which scales up to 448 reach a sixth of `largest`.
__device__ __forceinline__ float unit_of(float largest) {
  const int e = (int)(__float_as_uint(largest) >> 23) - 127;  // floor(log2)
  return __uint_as_float((uint32_t)(max(-100, e - 10) + 127) << 23);
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
