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
#include "qg_common.cuh"

namespace qg {

// maximum that keeps a NaN (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 16 consecutive values as they lie in memory (bf16 ones are unpacked where
// they are used: a unit in flight is 8 registers then, not 16)
template <bool kBf16>
struct Raw16 {
  static constexpr int kWords = kBf16 ? 2 : 4;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const void* row, int64_t k) {
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(row) + k * (kBf16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldcs(p + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float at(int i) const {  // value i (a constant)
    const uint4& q = w[i / (16 / kWords)];
    const int j = i % (16 / kWords);
    if (kBf16) {
      const uint32_t u = j < 2 ? q.x : j < 4 ? q.y : j < 6 ? q.z : q.w;
      return __uint_as_float((j & 1) ? u & 0xFFFF0000u : u << 16);
    }
    return __uint_as_float(j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w);
  }
  __device__ __forceinline__ float absmax() const {  // NaN if there is one
    if (kBf16) {  // without their signs, the bits are in the order of the values
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        m = __vmaxu2(m, w[i].x & 0x7FFF7FFFu);
        m = __vmaxu2(m, w[i].y & 0x7FFF7FFFu);
        m = __vmaxu2(m, w[i].z & 0x7FFF7FFFu);
        m = __vmaxu2(m, w[i].w & 0x7FFF7FFFu);
      }
      return __uint_as_float(max(m << 16, m & 0xFFFF0000u));
    }
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max_nan(m, fabsf(at(j)));
    return m;
  }
};

// e4m3 of four values (round to nearest even, saturating; NaN stays NaN)
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// e4m3 of x / s for values 4j.. of a lane, with the IEEE quotient. The quotient
// lies between x * lo and x * hi, lo and hi being 1/s less and more 4 units in
// the last place (1/s and the product are off by at most half a unit each, the
// rounded quotient by another half): where both give the same e4m3 value, it is
// the quotient's too. Else (about one value in 10^5) the division decides.
template <bool kBf16>
__device__ __forceinline__ uint32_t quotient_e4m3x4(const Raw16<kBf16>& v, int j, float s, float2 lo,
                                                    float2 hi) {
  const float2 x = make_float2(v.at(4 * j), v.at(4 * j + 1)), y = make_float2(v.at(4 * j + 2), v.at(4 * j + 3));
  const float2 xl = __fmul2_rn(x, lo), yl = __fmul2_rn(y, lo);
  const float2 xh = __fmul2_rn(x, hi), yh = __fmul2_rn(y, hi);
  const uint32_t a = e4m3x4(xl.x, xl.y, yl.x, yl.y), b = e4m3x4(xh.x, xh.y, yh.x, yh.y);
  if (__builtin_expect(a == b, 1)) return a;
  return e4m3x4(__fdiv_rn(x.x, s), __fdiv_rn(x.y, s), __fdiv_rn(y.x, s), __fdiv_rn(y.y, s));
}

// The four divided outright: s is subnormal (its reciprocal is not exact
// enough), zero (q = 0), infinite or not a number.
__device__ __noinline__ uint32_t divide_e4m3x4(float a, float b, float c, float d, float s) {
  if (s == 0.0f) return 0;
  return e4m3x4(__fdiv_rn(a, s), __fdiv_rn(b, s), __fdiv_rn(c, s), __fdiv_rn(d, s));
}

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
      uint32_t o[4];
      const float inv = act_scale_rcp(s);
      if (inv != 0.0f) {
        const float l = inv * (1.0f - 0x1p-22f), h = inv * (1.0f + 0x1p-22f);
        const float2 lo = make_float2(l, l), hi = make_float2(h, h);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = quotient_e4m3x4<kBf16>(v[i], j, s, lo, hi);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = divide_e4m3x4(v[i].at(4 * j), v[i].at(4 * j + 1), v[i].at(4 * j + 2), v[i].at(4 * j + 3), s);
      }
      *reinterpret_cast<uint4*>(q + m * (int64_t)K + k) = make_uint4(o[0], o[1], o[2], o[3]);
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
