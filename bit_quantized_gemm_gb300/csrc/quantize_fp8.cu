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
// 16-byte store per lane. HBM-bound for fp32 (4 bytes read and 1 written per
// value: 4096 x 17408 54 us, 6.6 TB/s); for bf16 (2 read) the instructions are
// as near a bound (issue slots 81 % used at 8192 x 17408, 75 us, 5.7 TB/s).
#include "quantize_fp8.cuh"

namespace qg {

// A warp's unit is 512 values of a row, kUnits of them loaded before the first
// is worked on.
template <bool kBf16, int kUnits>
__global__ void __launch_bounds__(128, kBf16 ? 12 : 8) quantize_act_fp8_kernel(
    const void* __restrict__ x, int64_t ldx, int K, int64_t units, int units_per_row,
    uint8_t* __restrict__ q, float* __restrict__ scale, int64_t lds) {
  // the GEMM of the layer call may start now; it waits for this grid before
  // it reads the activations
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t unit0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 5)) * kUnits;
  if (unit0 >= units) return;
  int64_t m = unit0 / units_per_row;
  int u = (int)(unit0 - m * units_per_row);
  const int64_t m0 = m;
  const int u0 = u;
  Raw16<kBf16> v[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int k = u * 512 + lane * 16;
    if (unit0 + i < units && k < K)
      v[i].load(reinterpret_cast<const char*>(x) + m * ldx * (kBf16 ? 2 : 4), k);
    else
      v[i].zero();
    if (++u == units_per_row) {
      u = 0;
      ++m;
    }
  }
  m = m0;
  u = u0;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int k = u * 512 + lane * 16;
    float amax = v[i].absmax();
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (unit0 + i < units && k < K) {
      const float s = amax * (1.0f / 448.0f);
      if ((lane & 7) == 0) scale[(int64_t)(k >> 7) * lds + m] = s;
      *reinterpret_cast<uint4*>(q + m * (int64_t)K + k) = e4m3x16([&](int j) { return v[i].at(j); }, s);
    }
    if (++u == units_per_row) {
      u = 0;
      ++m;
    }
  }
}

template <bool kBf16, int kUnits>
static void launch_q8(const void* x, int64_t M, int64_t K, int64_t ldx, uint8_t* q, float* scale,
                      int64_t lds, cudaStream_t st) {
  const int upr = (int)ceil_div(K, 512);
  const int64_t units = M * upr;
  quantize_act_fp8_kernel<kBf16, kUnits><<<(unsigned)ceil_div(units, 4 * kUnits), 128, 0, st>>>(
      x, ldx, (int)K, units, upr, q, scale, lds);
}

cudaError_t launch_quantize_act_fp8(const void* x, bool bf16, int64_t M, int64_t K, int64_t ldx,
                                    uint8_t* q, float* scale, int64_t lds, cudaStream_t st) {
  // Two units a warp where bf16 rows fill the SMs several times over (their
  // units are 1 KB): 8192 x 17408 75 us, 85 with one (5.7 and 5.0 TB/s); 2048 x
  // 2560 5.9 us, 5.7 with one. fp32 rows: 4096 x 17408 61 us, 53 with one.
  if (!bf16)
    launch_q8<false, 1>(x, M, K, ldx, q, scale, lds, st);
  else if (M * ceil_div(K, 512) < 16384)
    launch_q8<true, 1>(x, M, K, ldx, q, scale, lds, st);
  else
    launch_q8<true, 2>(x, M, K, ldx, q, scale, lds, st);
  return cudaGetLastError();
}

}  // namespace qg
