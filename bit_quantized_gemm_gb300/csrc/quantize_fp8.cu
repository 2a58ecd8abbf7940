// quantize_fp8.cu -- per-token, per-128-block e4m3 activation quantization.
//
// For row m and block b (128 consecutive k; the last one may be shorter):
//   s[b][m] = max |x[m][k]| * fl(1/448)  (one fp32 product; fl(1/448) is the
//                                          fp32 value nearest to 1/448)
//   q[m][k] = e4m3(clamp(x[m][k] / s, -448, 448))   (IEEE quotient, then to
//                                          nearest e4m3, ties to even)
// and s = 0 gives q = 0. NaN and infinities spread by IEEE rules: a block
// that holds a NaN has s = NaN and q = NaN; one that holds an infinity has
// s = inf, q = NaN there and 0 elsewhere, so the row's products are NaN.
//
// A lane owns 16 consecutive values (K is a multiple of 16), eight lanes a
// block, so the block's maximum takes three shuffles and q leaves in one
// 16-byte store per lane. HBM-bound: 2 (bf16) or 4 (fp32) bytes read and 1
// written per value.
#include "qg_common.cuh"

namespace qg {

// 16 consecutive values as fp32
template <bool kBf16>
__device__ __forceinline__ void load16(const void* row, int64_t k, float (&v)[16]) {
  if (kBf16) {
    const int4* p = reinterpret_cast<const int4*>(reinterpret_cast<const uint16_t*>(row) + k);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int4 raw = __ldg(p + h);
      const uint32_t w[4] = {(uint32_t)raw.x, (uint32_t)raw.y, (uint32_t)raw.z, (uint32_t)raw.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[8 * h + 2 * i] = __uint_as_float(w[i] << 16);
        v[8 * h + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(row) + k);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const float4 a = __ldg(p + h);
      v[4 * h] = a.x; v[4 * h + 1] = a.y; v[4 * h + 2] = a.z; v[4 * h + 3] = a.w;
    }
  }
}

// maximum that keeps a NaN (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// e4m3 of four values (round to nearest even, saturating; NaN stays NaN)
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

template <bool kBf16>
__global__ void __launch_bounds__(128) quantize_act_fp8_kernel(
    const void* __restrict__ x, int64_t ldx, int K, int64_t units, int units_per_row,
    uint8_t* __restrict__ q, float* __restrict__ scale, int64_t lds) {
  // the GEMM of the layer call may start now; it waits for this grid before
  // it reads the activations
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);  // 512 values of one row
  if (unit >= units) return;
  const int64_t m = unit / units_per_row;
  const int k = (int)(unit - m * units_per_row) * 512 + lane * 16;
  const bool valid = k < K;
  const char* row = reinterpret_cast<const char*>(x) + m * ldx * (kBf16 ? 2 : 4);
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  if (valid) load16<kBf16>(row, k, v);
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = max_nan(amax, fabsf(v[i]));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (!valid) return;
  const float s = amax * (1.0f / 448.0f);
  if ((lane & 7) == 0) scale[(int64_t)(k >> 7) * lds + m] = s;
  uint4 o4;
  uint32_t* o = reinterpret_cast<uint32_t*>(&o4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = s == 0.0f ? 0.0f : __fdiv_rn(v[4 * i + j], s);
    o[i] = e4m3x4(y[0], y[1], y[2], y[3]);
  }
  *reinterpret_cast<uint4*>(q + m * (int64_t)K + k) = o4;
}

cudaError_t launch_quantize_act_fp8(const void* x, bool bf16, int64_t M, int64_t K, int64_t ldx,
                                    uint8_t* q, float* scale, int64_t lds, cudaStream_t st) {
  const int upr = (int)ceil_div(K, 512);
  const int64_t units = M * upr;
  const unsigned grid = (unsigned)ceil_div(units, 4);
  if (bf16)
    quantize_act_fp8_kernel<true><<<grid, 128, 0, st>>>(x, ldx, (int)K, units, upr, q, scale, lds);
  else
    quantize_act_fp8_kernel<false><<<grid, 128, 0, st>>>(x, ldx, (int)K, units, upr, q, scale, lds);
  return cudaGetLastError();
}

}  // namespace qg
