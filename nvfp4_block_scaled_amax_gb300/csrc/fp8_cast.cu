// fp8_cast.cu -- the cast to E4M3 with one FP32 scale for each block of 128,
// rows and transposed columns in one pass.
//
// For a block (128 consecutive elements of a row, or a 128 x 128 tile) with
// a = max(max|x|, 2^-100):  s = a / 448,  r = 448 / a  (IEEE FP32 divisions)
// and q = E4M3_rn_satfinite(x * r).  The floor keeps s and r normal numbers
// for a block of zeros or of tiny values.  The column-wise output is the
// same cast of x transposed.
#include "common.cuh"
#include "fp8.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;
constexpr int kPitch = kTile + 1;  // floats: a column's 128 values lie in 32 different banks, four each

// Four FP32 values -> four E4M3 codes, v0 in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(float v0, float v1, float v2, float v3) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v1), "f"(v0));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v3), "f"(v2));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// One CTA per 128 x 128 tile.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads) fp8_cast_kernel(const void* xv, Fp8CastArgs a) {
  extern __shared__ float tile[];  // [128][kPitch]
  __shared__ float amax_r[kTile], amax_c[kTile], amax_t;
  constexpr int kVec = kBf16 ? 8 : 4;
  const int64_t n0 = (int64_t)blockIdx.x * kTile, m0 = (int64_t)blockIdx.y * kTile;
  const int64_t bz = blockIdx.z;
  const int64_t nb = (a.N + kTile - 1) / kTile, mb = (a.M + kTile - 1) / kTile;
  const int rows = (int)min((int64_t)kTile, a.M - m0), cols = (int)min((int64_t)kTile, a.N - n0);
  const char* x = static_cast<const char*>(xv) + (bz * a.M * a.N) * (kBf16 ? 2 : 4);
  for (int i = threadIdx.x; i < kTile * kTile / kVec; i += kThreads) {
    const int r = i / (kTile / kVec), c = i % (kTile / kVec) * kVec;
    float f[kVec] = {};
    if (r < rows && c < cols) {
      const uint4 v = *reinterpret_cast<const uint4*>(x + ((m0 + r) * a.N + n0 + c) * (kBf16 ? 2 : 4));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (kBf16) {
          f[2 * k] = bf16_lo(w[k]);
          f[2 * k + 1] = bf16_hi(w[k]);
        } else {
          f[k] = __uint_as_float(w[k]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kVec; ++k) tile[r * kPitch + c + k] = f[k];
  }
  __syncthreads();
  {
    // threads 0..127: rows, 128..255: columns
    const int i = threadIdx.x & 127;
    float m = 0.0f;
    if (threadIdx.x < 128)
      for (int c = 0; c < kTile; ++c) m = fmaxf(m, fabsf(tile[i * kPitch + c]));
    else
      for (int r = 0; r < kTile; ++r) m = fmaxf(m, fabsf(tile[r * kPitch + i]));
    (threadIdx.x < 128 ? amax_r : amax_c)[i] = m;
  }
  __syncthreads();
  if (a.block_rows == 128) {
    if (threadIdx.x == 0) {
      float m = 0.0f;
      for (int r = 0; r < kTile; ++r) m = fmaxf(m, amax_r[r]);
      amax_t = m;
    }
    __syncthreads();
    if (threadIdx.x < 128) amax_r[threadIdx.x] = amax_c[threadIdx.x] = amax_t;
    __syncthreads();
  }
  const float floor_amax = 7.888609052210118e-31f;  // 2^-100
  {
    const int i = threadIdx.x & 127;
    const bool col = threadIdx.x >= 128;
    const float m = fmaxf((col ? amax_c : amax_r)[i], floor_amax);
    const float s = __fdiv_rn(m, 448.0f);
    if (a.block_rows == 128) {
      if (threadIdx.x == 0 && a.scale_row) a.scale_row[(bz * mb + blockIdx.y) * nb + blockIdx.x] = s;
      if (threadIdx.x == 128 && a.scale_col) a.scale_col[(bz * nb + blockIdx.x) * mb + blockIdx.y] = s;
    } else {
      if (!col && a.scale_row && i < rows) a.scale_row[(bz * nb + blockIdx.x) * a.M + m0 + i] = s;
      if (col && a.scale_col && i < cols) a.scale_col[(bz * mb + blockIdx.y) * a.N + n0 + i] = s;
    }
    (col ? amax_c : amax_r)[i] = __fdiv_rn(448.0f, m);  // now the encode factor
  }
  __syncthreads();
  if (a.data_row)
    for (int i = threadIdx.x; i < kTile * kTile / 16; i += kThreads) {
      const int r = i >> 3, c = (i & 7) * 16;
      if (r >= rows || c >= cols) continue;
      const float f = amax_r[r];
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float* p = tile + r * kPitch + c + 4 * k;
        w[k] = e4m3x4(__fmul_rn(p[0], f), __fmul_rn(p[1], f), __fmul_rn(p[2], f), __fmul_rn(p[3], f));
      }
      *reinterpret_cast<uint4*>(a.data_row + (bz * a.M + m0 + r) * a.N + n0 + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  if (a.data_col)
    for (int i = threadIdx.x; i < kTile * kTile / 16; i += kThreads) {
      const int c = i >> 3, r = (i & 7) * 16;
      if (c >= cols || r >= rows) continue;
      const float f = amax_c[c];
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float* p = tile + (r + 4 * k) * kPitch + c;
        w[k] = e4m3x4(__fmul_rn(p[0], f), __fmul_rn(p[kPitch], f), __fmul_rn(p[2 * kPitch], f),
                      __fmul_rn(p[3 * kPitch], f));
      }
      *reinterpret_cast<uint4*>(a.data_col + (bz * a.N + n0 + c) * a.M + m0 + r) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace

cudaError_t launch_fp8_cast(const void* x, const Fp8CastArgs& a, const LaunchCtx& ctx) {
  if (a.batch == 0 || a.M == 0 || a.N == 0) return cudaSuccess;
  const dim3 grid((unsigned)fp8_blocks(a.N), (unsigned)fp8_blocks(a.M), (unsigned)a.batch);
  const int smem = kTile * kPitch * (int)sizeof(float);
  const auto kernel = a.bf16 ? fp8_cast_kernel<true> : fp8_cast_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, smem, ctx.stream>>>(x, a);
  return cudaGetLastError();
}

}  // namespace nvfp4
