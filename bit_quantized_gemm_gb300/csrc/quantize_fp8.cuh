// quantize_fp8.cuh -- what the kernels that write e4m3 activations share: raw
// vectors of 16 values, e4m3 conversion, the quotient by a block's scale.
#pragma once

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
  __device__ __forceinline__ float2 two(int i) const { return make_float2(at(2 * i), at(2 * i + 1)); }
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

// e4m3 of four values divided by s, with the IEEE quotient. The quotient
// lies between x * lo and x * hi, lo and hi being 1/s less and more 4 units in
// the last place (1/s and the product are off by at most half a unit each, the
// rounded quotient by another half): where both give the same e4m3 value, it is
// the quotient's too. Else (about one value in 10^5) the division decides.
__device__ __forceinline__ uint32_t quotient_e4m3x4(float2 x, float2 y, float s, float2 lo, float2 hi) {
  const float2 xl = __fmul2_rn(x, lo), yl = __fmul2_rn(y, lo);
  const float2 xh = __fmul2_rn(x, hi), yh = __fmul2_rn(y, hi);
  const uint32_t a = e4m3x4(xl.x, xl.y, yl.x, yl.y), b = e4m3x4(xh.x, xh.y, yh.x, yh.y);
  if (__builtin_expect(a == b, 1)) return a;
  return e4m3x4(__fdiv_rn(x.x, s), __fdiv_rn(x.y, s), __fdiv_rn(y.x, s), __fdiv_rn(y.y, s));
}

// The four divided outright: s is subnormal (its reciprocal is not exact
// enough), zero (q = 0), infinite or not a number.
static __device__ __noinline__ uint32_t divide_e4m3x4(float a, float b, float c, float d, float s) {
  if (s == 0.0f) return 0;
  return e4m3x4(__fdiv_rn(a, s), __fdiv_rn(b, s), __fdiv_rn(c, s), __fdiv_rn(d, s));
}

// A lane's 16 values divided by the scale s of their block: 16 bytes of e4m3. `at` gives value i.
template <class At>
__device__ __forceinline__ uint4 e4m3x16(const At& at, float s) {
  uint32_t o[4];
  const float inv = act_scale_rcp(s);
  if (inv != 0.0f) {
    const float l = inv * (1.0f - 0x1p-22f), h = inv * (1.0f + 0x1p-22f);
    const float2 lo = make_float2(l, l), hi = make_float2(h, h);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = quotient_e4m3x4(make_float2(at(4 * j), at(4 * j + 1)), make_float2(at(4 * j + 2), at(4 * j + 3)), s,
                             lo, hi);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = divide_e4m3x4(at(4 * j), at(4 * j + 1), at(4 * j + 2), at(4 * j + 3), s);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The same of values that come out of fp32 arithmetic themselves, as products
// with fl(1/s) (an IEEE quotient would differ beside ties of e4m3 alone, by less
// than what the values are off; a third of the instructions).
__device__ __forceinline__ uint4 e4m3x16_by_product(const float2 (&y)[8], float s) {
  const float inv = act_scale_rcp(s);
  uint32_t o[4];
  if (inv != 0.0f) {
    const float2 f = make_float2(inv, inv);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = __fmul2_rn(y[2 * j], f), b = __fmul2_rn(y[2 * j + 1], f);
      o[j] = e4m3x4(a.x, a.y, b.x, b.y);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = divide_e4m3x4(y[2 * j].x, y[2 * j].y, y[2 * j + 1].x, y[2 * j + 1].y, s);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// max |y| of 16 values; NaN if there is one
__device__ __forceinline__ float absmax16(const float2 (&y)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(y[i].x), "f"(y[i].y));
  return m;
}

}  // namespace qg
