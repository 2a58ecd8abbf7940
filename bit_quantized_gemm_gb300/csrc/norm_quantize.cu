// norm_quantize.cu -- root-mean-square norm of a row, with the residual's
// addition, and silu(gate) * up, each into 8-bit activations.
//
// Norm, row m of K values:
//   h[k] = x[k] + residual[k], rounded to their type and stored (h = x without
//          a residual). The norm reads the rounded h, so that it equals the
//          norm of what the next layer finds in memory.
//   r    = 1 / sqrt(sum h^2 / K + eps)    (fp32: IEEE quotients and root)
//   y[k] = (h[k] * r) * weight[k]         (fp32, not rounded to the input's type)
// and y is quantized as qg_quantize_act_fp8 or qg_quantize_act would.
// Gate, row m of 2K values: y[k] = g / (1 + e^-g) * u, g = x[k], u = x[K + k].
//
// The sum of squares: a lane's 16 values in order, the 32 lanes of a unit (512
// values) as a butterfly, a row's units by their number -- whichever warps hold
// them. So a row's bits depend neither on its batch nor on the launch.
//
// HBM-bound: 2 + 2 bytes read and 2 + 1 written a value (bf16, residual). Every
// value is read once and held in registers over the row's barrier; a CTA takes
// rows in turn and has the next row's loads in flight while it works on one, so
// the barrier costs no bandwidth. The weight lies in registers for all rows.
#include "quantize_fp8.cuh"

namespace qg {

struct NormArgs {
  const void* x;
  const void* res;     // or null
  const void* weight;  // bf16 or fp32
  void* sum;           // with res
  uint8_t* q;          // e4m3 or int8 (int8: or null)
  uint16_t* q16;       // int8: or null
  int32_t* bsum;       // int8: or null
  float* scale;        // e4m3: [ceil(K/128)][lds]; int8: [M]
  int64_t ldx, ldr, ldsum, lds, M;
  int K, weight_bf16;
  float eps;
};

// the 16 values of x + res, rounded to their type, in place of x
template <bool kBf16>
__device__ __forceinline__ void add_rounded(Raw16<kBf16>& x, const Raw16<kBf16>& r) {
#pragma unroll
  for (int i = 0; i < Raw16<kBf16>::kWords; ++i) {
    constexpr int kPer = 16 / Raw16<kBf16>::kWords;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kBf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x.at(i * kPer + 2 * j) + r.at(i * kPer + 2 * j),
                                                       x.at(i * kPer + 2 * j + 1) + r.at(i * kPer + 2 * j + 1));
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[j] = __float_as_uint(x.at(i * 4 + j) + r.at(i * 4 + j));
      }
    }
    x.w[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// a lane's 16 values quantized to int8 with the row's scale s (as
// qg_quantize_act does): bytes, fp16 copy, sums of 32 (a pair of lanes)
template <class At>
__device__ __forceinline__ void emit_int8(const NormArgs& a, const At& at, int64_t m, int k, bool valid, float s,
                                          float inv) {
  float f[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    // (a NaN scale: 0, the products are NaN by the scale)
    const float v = s > 0.0f ? qround(at(i), s, inv) : 0.0f;
    f[i] = fminf(127.0f, fmaxf(-127.0f, v));
  }
  if (valid && a.q) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t b[4], lo, hi;
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = (uint32_t)__float2int_rz(f[4 * i + j]);
      asm("prmt.b32 %0, %1, %2, 0x0040;" : "=r"(lo) : "r"(b[0]), "r"(b[1]));
      asm("prmt.b32 %0, %1, %2, 0x0040;" : "=r"(hi) : "r"(b[2]), "r"(b[3]));
      asm("prmt.b32 %0, %1, %2, 0x5410;" : "=r"(w[i]) : "r"(lo), "r"(hi));
    }
    *reinterpret_cast<uint4*>(a.q + m * (int64_t)a.K + k) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (valid && a.q16) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);  // exact
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    uint4* p = reinterpret_cast<uint4*>(a.q16 + m * (int64_t)a.K + k);
    p[0] = make_uint4(w[0], w[1], w[2], w[3]);
    p[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  if (a.bsum) {  // (the same for every lane)
    float part = 0.0f;  // exact: |sum| <= 32 * 127
#pragma unroll
    for (int i = 0; i < 16; ++i) part += f[i];
    part += __shfl_xor_sync(0xffffffffu, part, 1);
    if (valid && (threadIdx.x & 1) == 0) a.bsum[m * (int64_t)(a.K / kBlk) + k / kBlk] = (int32_t)part;
  }
}

constexpr int kNormMaxWarps = 32, kNormMaxUnits = kMaxK / 512;

// One row at a time by the W = blockDim.y warps of a group; blockDim.z groups a
// CTA, each with rows of its own, in step. A warp holds kU units of 512 values.
template <bool kBf16, bool kFp8, int kU>
__global__ void __launch_bounds__(kU == 4 ? 1024 : kU == 2 ? 544 : 512)
    norm_quantize_kernel(const NormArgs a) {
  griddep_launch_dependents();
  // [row parity][group][unit], then the int8 maxima likewise by warp
  __shared__ float part[2][kNormMaxUnits], top[2][kNormMaxWarps];
  const int lane = threadIdx.x, warp = threadIdx.y, W = blockDim.y, group = threadIdx.z;
  const int K = a.K, units = (K + 511) >> 9;
  const int64_t step = (int64_t)gridDim.x * blockDim.z;
  float* const row_part = part[0] + group * units;  // (units x groups is at most kNormMaxUnits)
  float* const row_top = top[0] + group * W;
  constexpr bool kAhead = kU <= 2;  // the next row's loads during this one's work; the weight in registers
  constexpr int kHeld = kAhead ? kU : 1;

  auto where = [&](int u) { return ((u * W + warp) << 9) + lane * 16; };  // k of this lane in its unit u
  auto load_weight = [&](int k, float (&w)[16]) {
    if (a.weight_bf16) {
      Raw16<true> r;
      const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.weight) + k);
      r.w[0] = __ldg(p);
      r.w[1] = __ldg(p + 1);
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = r.at(i);
    } else {
      const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.weight) + k);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = __ldg(p + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
    }
  };
  float w[kHeld][16];
  if (kAhead) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
      if (where(u) < K) load_weight(where(u), w[u]);
  }
  Raw16<kBf16> v[kU], r[kU];
  auto load = [&](int64_t m) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = where(u);
      v[u].zero();
      if (m < a.M && k < K) {
        v[u].load(reinterpret_cast<const char*>(a.x) + m * a.ldx * (kBf16 ? 2 : 4), k);
        if (a.res) r[u].load(reinterpret_cast<const char*>(a.res) + m * a.ldr * (kBf16 ? 2 : 4), k);
      }
    }
  };
  int64_t m = (int64_t)blockIdx.x * blockDim.z + group;
  load(m);
  // (the groups of a CTA pass the barriers together: trips by the first group's row)
  for (int odd = 0; m - group < a.M; m += step, odd ^= 1) {
    const bool row = m < a.M;
    Raw16<kBf16> h[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = where(u);
      h[u] = v[u];
      if (a.res && row && k < K) {
        add_rounded(h[u], r[u]);
        uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<char*>(a.sum) + (m * a.ldsum + k) * (kBf16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < Raw16<kBf16>::kWords; ++i) p[i] = h[u].w[i];
      }
    }
    if (kAhead) load(m + step);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int unit = u * W + warp;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) s = fmaf(h[u].at(i), h[u].at(i), s);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0 && unit < units) row_part[odd * kNormMaxUnits + unit] = s;
    }
    __syncthreads();
    float sum = 0.0f;
    for (int u = lane; u < units; u += 32) sum += row_part[odd * kNormMaxUnits + u];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float rms = __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, (float)K) + a.eps));

    auto normed = [&](int u, float (&y)[16]) {
      if (!kAhead && where(u) < K) load_weight(where(u), w[0]);
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = (h[u].at(i) * rms) * w[kAhead ? u : 0][i];
    };
    if (kFp8) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int k = where(u);
        float y[16], amax = 0.0f;
        normed(u, y);
        if (k < K) {
#pragma unroll
          for (int i = 0; i < 16; ++i) amax = max_nan(amax, fabsf(y[i]));
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (row && k < K) {
          const float s = amax * (1.0f / 448.0f);
          if ((lane & 7) == 0) a.scale[(int64_t)(k >> 7) * a.lds + m] = s;
          *reinterpret_cast<uint4*>(a.q + m * (int64_t)K + k) = e4m3x16([&](int i) { return y[i]; }, s);
        }
      }
    } else {
      float amax = 0.0f;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        float y[16];
        normed(u, y);
        if (where(u) < K) {
#pragma unroll
          for (int i = 0; i < 16; ++i) amax = max_nan(amax, fabsf(y[i]));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (lane == 0) row_top[odd * kNormMaxWarps + warp] = amax;
      __syncthreads();
      amax = lane < W ? row_top[odd * kNormMaxWarps + lane] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float s = act_scale(amax), inv = act_scale_rcp(s);
      if (row && warp == 0 && lane == 0) a.scale[m] = s;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        float y[16];
        normed(u, y);
        emit_int8(a, [&](int i) { return y[i]; }, m, where(u), row && where(u) < K, s, inv);
      }
    }
    if (!kAhead) load(m + step);
  }
}

template <bool kBf16, bool kFp8, int kU>
static cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
  const int units = (int)ceil_div(a.K, 512), W = (int)ceil_div(units, kU);
  // short rows: several to a CTA, 256 threads in all
  const int groups = W >= 8 ? 1 : 8 / W;
  auto kern = norm_quantize_kernel<kBf16, kFp8, kU>;
  int per_sm = 0;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, 32 * W * groups, 0);
  if (e != cudaSuccess) return e;
  const int64_t ctas = ceil_div(a.M, groups), most = (int64_t)num_sms() * (per_sm > 0 ? per_sm : 1);
  kern<<<(unsigned)(ctas < most ? ctas : most), dim3(32, W, groups), 0, st>>>(a);
  return cudaGetLastError();
}

template <bool kBf16, bool kFp8>
static cudaError_t launch_norm_any(const NormArgs& a, cudaStream_t st) {
  if (a.K <= 512 * 16) return launch_norm<kBf16, kFp8, 1>(a, st);
  if (a.K <= 512 * 2 * 17) return launch_norm<kBf16, kFp8, 2>(a, st);
  return launch_norm<kBf16, kFp8, 4>(a, st);
}

cudaError_t launch_norm_quantize(const void* x, const void* res, bool bf16, int64_t M, int64_t K, int64_t ldx,
                                 int64_t ldr, const void* weight, bool weight_bf16, float eps, void* sum,
                                 int64_t ldsum, bool fp8, uint8_t* q, uint16_t* q16, int32_t* bsum, float* scale,
                                 int64_t lds, cudaStream_t st) {
  const NormArgs a{x, res, weight, sum, q, q16, bsum, scale, ldx, ldr, ldsum, lds, M, (int)K, weight_bf16, eps};
  if (fp8) return bf16 ? launch_norm_any<true, true>(a, st) : launch_norm_any<false, true>(a, st);
  return bf16 ? launch_norm_any<true, false>(a, st) : launch_norm_any<false, false>(a, st);
}

// ------------------------------------------------------------------------ gate
// silu(g) * u = g * sigmoid(g) * u, sigmoid(g) = (g < 0 ? t : 1) / (1 + t), t =
// e^-|g|, so that nothing overflows. The hardware's 2^x and 1/x: with the
// product |g| log2 e rounded once, silu is off by less than (4 + |g|) 2^-23 of
// itself; t below 2^-126 counts as 0.
__device__ __forceinline__ float silu_mul(float g, float u) {
  float t, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fabsf(g) * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
  return g * (g < 0.0f ? t : 1.0f) * r * u;
}

template <bool kBf16>
__global__ void __launch_bounds__(128) silu_mul_quantize_kernel(const void* __restrict__ x, int64_t ldx, int K,
                                                                int64_t units, int units_per_row,
                                                                uint8_t* __restrict__ q, float* __restrict__ scale,
                                                                int64_t lds) {
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (unit >= units) return;
  const int64_t m = unit / units_per_row;
  const int k = (int)(unit - m * units_per_row) * 512 + lane * 16;
  Raw16<kBf16> g, u;
  g.zero();
  u.zero();
  if (k < K) {
    const char* row = reinterpret_cast<const char*>(x) + m * ldx * (kBf16 ? 2 : 4);
    g.load(row, k);
    u.load(row, (int64_t)K + k);
  }
  float y[16], amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    y[i] = silu_mul(g.at(i), u.at(i));
    amax = max_nan(amax, fabsf(y[i]));
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (k < K) {
    const float s = amax * (1.0f / 448.0f);
    if ((lane & 7) == 0) scale[(int64_t)(k >> 7) * lds + m] = s;
    *reinterpret_cast<uint4*>(q + m * (int64_t)K + k) = e4m3x16([&](int i) { return y[i]; }, s);
  }
}

cudaError_t launch_silu_mul_quantize_fp8(const void* x, bool bf16, int64_t M, int64_t K, int64_t ldx, uint8_t* q,
                                         float* scale, int64_t lds, cudaStream_t st) {
  const int upr = (int)ceil_div(K, 512);
  const int64_t units = M * upr;
  const unsigned grid = (unsigned)ceil_div(units, 4);
  if (bf16)
    silu_mul_quantize_kernel<true><<<grid, 128, 0, st>>>(x, ldx, (int)K, units, upr, q, scale, lds);
  else
    silu_mul_quantize_kernel<false><<<grid, 128, 0, st>>>(x, ldx, (int)K, units, upr, q, scale, lds);
  return cudaGetLastError();
}

}  // namespace qg
