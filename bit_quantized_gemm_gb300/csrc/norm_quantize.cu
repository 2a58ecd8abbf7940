// norm_quantize.cu -- root-mean-square norm of a row, with the residual's
// addition, and silu(gate) * up, each into 8-bit activations.
//
// Norm, row m of K values:
//   h[k] = x[k] + residual[k], rounded to their type and stored (h = x without
//          a residual). The norm reads the rounded h, so that it equals the
//          norm of what the next layer finds in memory.
//   r    = 1 / sqrt(sum h^2 / K + eps)    (fp32: the hardware's root, refined once)
//   y[k] = (h[k] * r) * weight[k]         (fp32, not rounded to the input's type)
// and y is quantized: e4m3 per 128 values with s = max|y| * fl(1/448), or int8
// per row with s = max|y| / 127, by products with fl(1/s).
// Gate, row m of 2K values: y[k] = g / (1 + e^-g) * u, g = x[k], u = x[K + k].
//
// The sum of squares: a lane's 16 values in two chains, the 32 lanes of a unit
// (512 values) as a butterfly, a row's units by their number -- whichever warps
// hold them. So a row's bits depend neither on its batch nor on the launch.
//
// With a residual HBM-bound: 2 + 2 bytes read and 2 + 1 written a value (bf16). Every
// value is read once and held by its lane over the row's barrier -- in registers with
// one unit a warp and weights of the rows' type, partly in local memory (spills of 32
// to 208 bytes a thread with two units a warp or fp32 weights of bf16 rows, up to 980
// with four, K > 17408); several rows' CTAs on an SM fill one another's waits. 8192 x
// 5120 bf16 with a residual: 47.2 us, 6.25 TB/s (a plain copy: 6.77). A ring of bulk
// copies in shared memory instead of the registers was slower. Without a residual the
// same instructions move half the bytes, and they and the barrier are what bounds it:
// 31.8 us, 3.95 TB/s. One row: 2.1 us, a launch and two trips to memory. The gate reads
// 4 bytes and writes 1 a value: 8192 x 17408 116.5 us, 6.15 TB/s; beside memory, the
// two special-function results a value are what it issues most.
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
  int K;
  float eps;
};

// the 16 values of x + r, each rounded once to their type, in place of x
__device__ __forceinline__ void add_rounded(Raw16<true>& x, const Raw16<true>& r) {
  auto add = [](uint32_t& a, uint32_t b) { asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b)); };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    add(x.w[i].x, r.w[i].x);
    add(x.w[i].y, r.w[i].y);
    add(x.w[i].z, r.w[i].z);
    add(x.w[i].w, r.w[i].w);
  }
}
__device__ __forceinline__ void add_rounded(Raw16<false>& x, const Raw16<false>& r) {
  auto add = [](uint32_t& a, uint32_t b) { a = __float_as_uint(__uint_as_float(a) + __uint_as_float(b)); };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    add(x.w[i].x, r.w[i].x);
    add(x.w[i].y, r.w[i].y);
    add(x.w[i].z, r.w[i].z);
    add(x.w[i].w, r.w[i].w);
  }
}

// 1 / sqrt(v): the hardware's, and one step of Newton's iteration (v = 0 and
// infinity have none: it would make a NaN of them)
__device__ __forceinline__ float rsqrt_refined(float v) {
  float r;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  const float e = fmaf(-v * r, r, 1.0f);
  return v > 0.0f && v < 3.0e38f ? fmaf(0.5f * r, e, r) : r;
}

// a lane's 16 values quantized to int8 with the row's scale s: bytes, fp16 copy,
// sums of 32 (a pair of lanes). Where s is normal, |y * fl(1/s)| rounds to at most
// 127; a subnormal s = max|y| / 127 has only a few bits, and quotients by it are
// clamped (max|y| = 190 * 2^-149 gives s = 2^-149). s = 0, NaN or infinite: q is 0.
__device__ __forceinline__ void emit_int8(const NormArgs& a, const float2 (&y)[8], int64_t m, int k, bool valid,
                                          float s, float inv) {
  float2 f[8];  // whole numbers + 1.5 * 2^23: the low byte is the int8 value
  const float magic = 12582912.0f;
  if (inv != 0.0f) {
    const float2 i2 = make_float2(inv, inv), m2 = make_float2(magic, magic);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __ffma2_rn(y[i], i2, m2);
  } else {
    // s is subnormal (its reciprocal is not exact enough), or there is nothing to divide by
    const bool divide = s > 0.0f && s < 3.4e38f;
    auto quotient = [&](float v) { return fminf(fmaxf(__fdiv_rn(v, s), -127.0f), 127.0f) + magic; };
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = divide ? make_float2(quotient(y[i].x), quotient(y[i].y)) : make_float2(magic, magic);
  }
  if (a.q || a.bsum) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo, hi;
      asm("prmt.b32 %0, %1, %2, 0x0040;" : "=r"(lo) : "r"(__float_as_uint(f[2 * i].x)), "r"(__float_as_uint(f[2 * i].y)));
      asm("prmt.b32 %0, %1, %2, 0x0040;"
          : "=r"(hi)
          : "r"(__float_as_uint(f[2 * i + 1].x)), "r"(__float_as_uint(f[2 * i + 1].y)));
      asm("prmt.b32 %0, %1, %2, 0x5410;" : "=r"(w[i]) : "r"(lo), "r"(hi));
    }
    if (valid && a.q) *reinterpret_cast<uint4*>(a.q + m * (int64_t)a.K + k) = make_uint4(w[0], w[1], w[2], w[3]);
    if (a.bsum) {  // (the same for every lane)
      int part = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) part = __dp4a((int)w[i], 0x01010101, part);
      part += __shfl_xor_sync(0xffffffffu, part, 1);
      if (valid && (threadIdx.x & 1) == 0) a.bsum[m * (int64_t)(a.K / kBlk) + k / kBlk] = part;
    }
  }
  if (valid && a.q16) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __half2 h = __floats2half2_rn(f[i].x - magic, f[i].y - magic);  // exact
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    uint4* p = reinterpret_cast<uint4*>(a.q16 + m * (int64_t)a.K + k);
    p[0] = make_uint4(w[0], w[1], w[2], w[3]);
    p[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

constexpr int kNormMaxWarps = 32, kNormMaxUnits = kMaxK / 512;

// Registers decide how many rows an SM works on at once: 8192 x 5120 bf16 with a
// residual 48.2 us with 40 (five CTAs), 51.4 with 52 (three); without one 31.0 and
// 36.8. Rows in two units a warp, 8192 x 17408 bf16 without a residual: 132 us with
// 56 (two CTAs), 145 with 77 (one). (Measured with bf16 weights: fp32 weights of bf16
// rows have the same registers, spill, and take 58.3 us where those take 45.8.)
template <bool kBf16, bool kWBf16, int kU>
constexpr int kNormRegs = kU == 4 ? 64 : kU == 2 ? (kBf16 ? 56 : 96) : kBf16 ? 40 : kWBf16 ? 48 : 56;

// A row by the W = blockDim.y warps of a group (threadIdx.z: the groups of a CTA
// have a row each). A warp holds kU units of 512 values.
template <bool kBf16, bool kWBf16, bool kFp8, int kU>
__global__ void __maxnreg__((kNormRegs<kBf16, kWBf16, kU>)) norm_quantize_kernel(const NormArgs a) {
  // sums by group and unit (at most kNormMaxUnits), int8 maxima by group and warp
  __shared__ float part[kNormMaxUnits], top[kNormMaxWarps];
  const int lane = threadIdx.x, warp = threadIdx.y, W = blockDim.y, group = threadIdx.z;
  const int K = a.K, units = (K + 511) >> 9;
  const int64_t m = (int64_t)blockIdx.x * blockDim.z + group;
  const bool row = m < a.M;
  auto at = [&](int u) { return ((u * W + warp) << 9) + lane * 16; };  // k of this lane in its unit u
  Raw16<kBf16> h[kU];
  constexpr bool kHeld = kU <= 2;  // the weight, too, before the barrier
  Raw16<kWBf16> w[kHeld ? kU : 1];
  auto load_weight = [&](int u) {
    if (at(u) >= K) return;
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(a.weight) +
                                                    (size_t)at(u) * (kWBf16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < Raw16<kWBf16>::kWords; ++i) w[kHeld ? u : 0].w[i] = __ldg(p + i);
  };
  {
    Raw16<kBf16> r[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = at(u);
      h[u].zero();
      if (row && k < K) {
        h[u].load(reinterpret_cast<const char*>(a.x) + m * a.ldx * (kBf16 ? 2 : 4), k);
        if (a.res) r[u].load(reinterpret_cast<const char*>(a.res) + m * a.ldr * (kBf16 ? 2 : 4), k);
      }
    }
    if (kHeld) {
#pragma unroll
      for (int u = 0; u < kU; ++u) load_weight(u);
    }
    if (a.res) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int k = at(u);
        if (row && k < K) {
          add_rounded(h[u], r[u]);
          uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<char*>(a.sum) + (m * a.ldsum + k) * (kBf16 ? 2 : 4));
#pragma unroll
          for (int i = 0; i < Raw16<kBf16>::kWords; ++i) p[i] = h[u].w[i];
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int unit = u * W + warp;
    float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i) s2 = __ffma2_rn(h[u].two(i), h[u].two(i), s2);
    float s = s2.x + s2.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0 && unit < units) part[group * units + unit] = s;
  }
  __syncthreads();
  float sum = lane < units ? part[group * units + lane] : 0.0f;
  if (units > 32)
    for (int u = lane + 32; u < units; u += 32) sum += part[u];  // (one group)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float rms = rsqrt_refined(__fdividef(sum, (float)K) + a.eps);
  const float2 rms2 = make_float2(rms, rms);

  auto normed = [&](int u, float2 (&y)[8]) {
    if (!kHeld) load_weight(u);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fmul2_rn(__fmul2_rn(h[u].two(i), rms2), w[kHeld ? u : 0].two(i));
  };
  if (kFp8) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = at(u);
      float2 y[8];
      normed(u, y);
      float amax = k < K ? absmax16(y) : 0.0f;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (row && k < K) {
        const float s = amax * (1.0f / 448.0f);
        if ((lane & 7) == 0) a.scale[(int64_t)(k >> 7) * a.lds + m] = s;
        *reinterpret_cast<uint4*>(a.q + m * (int64_t)K + k) = e4m3x16_by_product(y, s);
      }
    }
  } else {
    float amax = 0.0f;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float2 y[8];
      normed(u, y);
      if (at(u) < K) amax = max_nan(amax, absmax16(y));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) top[group * W + warp] = amax;
    __syncthreads();
    amax = lane < W ? top[group * W + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = act_scale(amax), inv = act_scale_rcp(s);
    if (row && warp == 0 && lane == 0) a.scale[m] = s;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float2 y[8];
      normed(u, y);
      emit_int8(a, y, m, at(u), row && at(u) < K, s, inv);
    }
  }
}

template <bool kBf16, bool kWBf16, bool kFp8, int kU>
static cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
  const int W = (int)ceil_div(ceil_div(a.K, 512), kU);
  const int groups = W >= 8 ? 1 : 8 / W;  // short rows: several to a CTA, 256 threads in all
  norm_quantize_kernel<kBf16, kWBf16, kFp8, kU>
      <<<(unsigned)ceil_div(a.M, groups), dim3(32, W, groups), 0, st>>>(a);
  return cudaGetLastError();
}

template <bool kBf16, bool kWBf16, bool kFp8>
static cudaError_t launch_norm_k(const NormArgs& a, cudaStream_t st) {
  // one unit a warp up to 20 warps (4096 x 9728 bf16: 48.1 us, 58.6 in two units),
  // two up to 17 (4096 x 14336 int8: 91 us, 104 in one); with an SM for every row one up
  // to 32 (16 x 14128 bf16, residual: 3.7 us, 4.6 in two)
  if (a.K <= 512 * 20 || (a.K <= 512 * 32 && a.M <= num_sms()))
    return launch_norm<kBf16, kWBf16, kFp8, 1>(a, st);
  if (a.K <= 512 * 2 * 17) return launch_norm<kBf16, kWBf16, kFp8, 2>(a, st);
  return launch_norm<kBf16, kWBf16, kFp8, 4>(a, st);
}

template <bool kBf16, bool kFp8>
static cudaError_t launch_norm_w(const NormArgs& a, bool weight_bf16, cudaStream_t st) {
  return weight_bf16 ? launch_norm_k<kBf16, true, kFp8>(a, st) : launch_norm_k<kBf16, false, kFp8>(a, st);
}

cudaError_t launch_norm_quantize(const void* x, const void* res, bool bf16, int64_t M, int64_t K, int64_t ldx,
                                 int64_t ldr, const void* weight, bool weight_bf16, float eps, void* sum,
                                 int64_t ldsum, bool fp8, uint8_t* q, uint16_t* q16, int32_t* bsum, float* scale,
                                 int64_t lds, cudaStream_t st) {
  const NormArgs a{x, res, weight, sum, q, q16, bsum, scale, ldx, ldr, ldsum, lds, M, (int)K, eps};
  if (fp8) return bf16 ? launch_norm_w<true, true>(a, weight_bf16, st) : launch_norm_w<false, true>(a, weight_bf16, st);
  return bf16 ? launch_norm_w<true, false>(a, weight_bf16, st) : launch_norm_w<false, false>(a, weight_bf16, st);
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
  float2 y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    y[i] = make_float2(silu_mul(g.at(2 * i), u.at(2 * i)), silu_mul(g.at(2 * i + 1), u.at(2 * i + 1)));
  float amax = absmax16(y);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (k < K) {
    const float s = amax * (1.0f / 448.0f);
    if ((lane & 7) == 0) scale[(int64_t)(k >> 7) * lds + m] = s;
    *reinterpret_cast<uint4*>(q + m * (int64_t)K + k) = e4m3x16_by_product(y, s);
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
