// gemm_fp8.cu -- product of e4m3 operands with an fp32 scale for each block
// of 128.
//
//   out[m][n] = sum over blocks b, ascending, of
//               fmaf(sum_{k in b} q[m][k] * w[n][k], s[b][m] * ws[n/128][b], acc)
//
// The plain form of the kernel: a 64 x 64 tile per CTA, both operands widened
// to fp32 in shared memory, one block's products summed in fp32 before they
// are scaled.
#include <cuda_fp8.h>

#include "qg_common.cuh"

namespace qg {

__device__ __forceinline__ float e4m3_to_f32(uint8_t v) {
  __nv_fp8_e4m3 h;
  h.__x = v;
  return (float)h;
}

__global__ void __launch_bounds__(256) gemm_fp8_plain_kernel(
    const uint8_t* __restrict__ q, const float* __restrict__ scale, int64_t lds, int M, int K,
    const uint8_t* __restrict__ w, int64_t ldw, const float* __restrict__ w_scale, int N,
    void* __restrict__ out, int out_f32, int64_t ldo) {
  __shared__ float As[16][65], Bs[16][65];
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int KB = (K + 127) / 128;
  float acc[4][4] = {};
  for (int b = 0; b < KB; ++b) {
    float sum[4][4] = {};
    for (int k0 = b * 128; k0 < min(K, b * 128 + 128); k0 += 16) {  // K % 16 == 0
      __syncthreads();
      const int kk = threadIdx.x & 15;
      for (int r = threadIdx.x >> 4; r < 64; r += 16) {
        As[kk][r] = m0 + r < M ? e4m3_to_f32(q[(int64_t)(m0 + r) * K + k0 + kk]) : 0.0f;
        Bs[kk][r] = n0 + r < N ? e4m3_to_f32(w[(int64_t)(n0 + r) * ldw + k0 + kk]) : 0.0f;
      }
      __syncthreads();
      for (int k = 0; k < 16; ++k)
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j) sum[i][j] = fmaf(As[k][ty * 4 + i], Bs[k][tx * 4 + j], sum[i][j]);
    }
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + ty * 4 + i;
      const float sm = m < M ? scale[b * lds + m] : 0.0f;
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx * 4 + j;
        const float f = n < N ? sm * w_scale[(int64_t)(n >> 7) * KB + b] : 0.0f;
        acc[i][j] = fmaf(sum[i][j], f, acc[i][j]);
      }
    }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= M || n >= N) continue;
      if (out_f32)
        reinterpret_cast<float*>(out)[m * ldo + n] = acc[i][j];
      else
        reinterpret_cast<uint16_t*>(out)[m * ldo + n] = f32_to_bf16_rne(acc[i][j]);
    }
}

cudaError_t launch_gemm_fp8(const uint8_t* q, const float* scale, int64_t lds, int64_t M, int64_t K,
                            const uint8_t* w, int64_t ldw, const float* w_scale, int64_t N,
                            void* out, bool out_f32, int64_t ldo, uint32_t* err, bool pdl,
                            cudaStream_t st) {
  (void)err;
  (void)pdl;
  // token tiles in grid.y: at most 65535 of them per launch
  for (int64_t m0 = 0; m0 < M; m0 += 65535 * 64) {
    const int64_t mc = M - m0 < 65535 * 64 ? M - m0 : 65535 * 64;
    gemm_fp8_plain_kernel<<<dim3((unsigned)ceil_div(N, 64), (unsigned)ceil_div(mc, 64)), 256, 0, st>>>(
        q + m0 * K, scale + m0, lds, (int)mc, (int)K, w, ldw, w_scale, (int)N,
        reinterpret_cast<char*>(out) + m0 * ldo * (out_f32 ? 4 : 2), out_f32, ldo);
  }
  return cudaGetLastError();
}

}  // namespace qg
