// fp4_matmul.cu -- the product of 4-bit operands:
//     c[m][n] = fa fb sum_k a[m][k] sa[m][k / b] b[n][k] sb[n][k / b]
// with b = 16 and E4M3 scales (NVFP4; fa, fb = amax / 2688) or b = 32 and
// powers of two (MXFP4; fa = fb = 1).  The tensor cores take codes and scales
// as they are (tcgen05 block_scale) and sum in FP32 in tensor memory.
#include "fp4_tiles.cuh"

namespace nvfp4 {

cudaError_t launch_fp4_matmul(const Fp4MatmulArgs& a, const LaunchCtx& ctx) {
  using namespace fp4;
  if (a.a.rows == 0 || a.b.rows == 0) return cudaSuccess;
  if (a.K == 0) return cudaMemsetAsync(a.out, 0, (size_t)a.a.rows * a.b.rows * (a.out_bf16 ? 2 : 4), ctx.stream);
  MatmulKernelArgs p = {};
  p.a = a.a;
  p.b = a.b;
  p.K = a.K;
  p.out = a.out;
  p.out_bf16 = a.out_bf16;
  p.status = ctx.status;
  return launch_matmul_thin(a, p, ctx);
}

}  // namespace nvfp4
