// lora.cu -- low-rank adapters of many requests beside a shared projection.
//
//   h[m][r]   = sum_k x[m][k] * A[id][r][k]        id = ids[m]
//   out[m][n] = base[m][n] + sum_r (scaling[id] * h[m][r]) * B[id][n][r]
// A row whose id is not one of the adapters keeps base's bits.
//
// Two kernels. `shrink` forms scaling * h and leaves it as the sum of two bf16
// numbers (off by 2^-17 of itself: the sum of the two products is then as good
// as one with an fp32 h); `expand`, its programmatic dependent, adds the second
// product to base. Both use warp-level m16n8k16 MMAs with operands straight from
// global memory: the products are short (rank 8 to 128) beside what is moved, x
// and the adapters once, base and out.
//
// Rows may come in any order. Of each 32 (16) consecutive rows a warp finds the
// different ids by votes and takes them one after another, so rows of one
// request that follow one another cost one pass, rows of 32 requests 32.
#include "qg_common.cuh"

namespace qg {

struct LoraArgs {
  const void* x;
  const uint16_t *a, *b;  // bf16 [count][rank][K], [count][N][rank]
  const int64_t* ids;
  const float* scaling;   // [count] or null
  const void* base;
  void* out;
  uint32_t *hi, *lo;      // [M][rank up to 16] pairs of bf16
  int64_t ldx, ldb, ldo, M;
  int K, N, rank, count;
};

// D (16 x 8) += A (16 x 16) * B (16 x 8), bf16 operands, fp32 sums
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// the id of row m as an adapter's number, -1 for none
__device__ __forceinline__ int adapter_of(const LoraArgs& a, int64_t m) {
  if (m >= a.M) return -1;
  const int64_t id = __ldg(a.ids + m);
  return id >= 0 && id < a.count ? (int)id : -1;
}

constexpr int kShrinkRows = 32, kShrinkCluster = 8, kShrinkWarps = 8;

// A cluster of eight CTAs forms h of the rows of one adapter among 32: each of
// its 64 warps sums its share of K over all those rows, the warps' sums are
// added in order within a CTA, then the CTAs' in order. The shares depend on K
// alone, so a row's bits do not depend on the other rows of its call.
// A's rows are the MMA's 16, the rows of x its 8. A lane loads 8 consecutive k
// of a row (16 bytes): they are k 8t.. of 32, t = lane % 4, of both operands, in
// whatever order the MMA sums them.
template <bool kBf16, int RT>  // RT tiles of 16 ranks
__global__ void __cluster_dims__(kShrinkCluster, 1, 1) __launch_bounds__(32 * kShrinkWarps)
    lora_shrink_kernel(const LoraArgs a) {
  griddep_launch_dependents();
  extern __shared__ float part[];  // [warp][row][rank], then [row][rank]
  constexpr int RP = RT * 16;
  float* const sum = part + kShrinkWarps * kShrinkRows * RP;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t rank = cluster_ctarank();
  const int64_t m0 = (int64_t)blockIdx.y * kShrinkRows;
  const int mine = adapter_of(a, m0 + lane);
  const uint32_t same = __match_any_sync(0xffffffffu, mine);
  // one lane of each adapter's rows
  uint32_t leaders = __ballot_sync(0xffffffffu, mine >= 0 && (int)lane == __ffs(same) - 1);
  const int share = (int)rank * kShrinkWarps + warp, units = (a.K + 31) >> 5;
  const int u0 = units * share / (kShrinkCluster * kShrinkWarps);
  const int u1 = units * (share + 1) / (kShrinkCluster * kShrinkWarps);
  for (int j = 0; leaders; ++j, leaders &= leaders - 1) {
    if (j % (int)gridDim.z != (int)blockIdx.z) continue;
    const int first = __ffs(leaders) - 1;
    const int id = __shfl_sync(0xffffffffu, mine, first);
    const uint32_t rows = __shfl_sync(0xffffffffu, same, first);
    const int count = __popc(rows), tiles = (count + 7) >> 3;
    // this lane's rows of x: number g of each eight (past the last: the last)
    const char* px[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = __fns(rows, 0, min(8 * i + g, count - 1) + 1);
      px[i] = reinterpret_cast<const char*>(a.x) + (m0 + row) * a.ldx * (kBf16 ? 2 : 4);
    }
    const uint16_t* pa = a.a + (int64_t)id * a.rank * a.K;
    float acc[RT][4][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][i][c] = 0.0f;
    for (int u = u0; u < u1; ++u) {
      const int k = u * 32 + t * 8;
      const bool in = k < a.K;
      uint4 wa[RT][2];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = r * 16 + h * 8 + g;
          wa[r][h] = in && row < a.rank ? __ldg(reinterpret_cast<const uint4*>(pa + (int64_t)row * a.K + k))
                                        : make_uint4(0, 0, 0, 0);
        }
      // x as one bf16 number a value, or as the sum of three (24 bits)
      constexpr int P = kBf16 ? 1 : 3;
      uint32_t xv[4][P][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= tiles) break;
        if (kBf16) {
          const uint4 v = in ? *reinterpret_cast<const uint4*>(px[i] + (int64_t)k * 2) : make_uint4(0, 0, 0, 0);
          xv[i][0][0] = v.x;
          xv[i][0][1] = v.y;
          xv[i][0][2] = v.z;
          xv[i][0][3] = v.w;
        } else {
          const float4* p = reinterpret_cast<const float4*>(px[i] + (int64_t)k * 4);
          const float4 z = make_float4(0, 0, 0, 0), v0 = in ? p[0] : z, v1 = in ? p[1] : z;
          float f[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int q = 0; q < P; ++q)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t w = bf16x2(f[2 * c], f[2 * c + 1]);
              xv[i][q][c] = w;
              // (an infinity's rest would be NaN)
              f[2 * c] = isfinite(bf16_lo(w)) ? f[2 * c] - bf16_lo(w) : 0.0f;
              f[2 * c + 1] = isfinite(bf16_hi(w)) ? f[2 * c + 1] - bf16_hi(w) : 0.0f;
            }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= tiles) break;
#pragma unroll
        for (int q = 0; q < P; ++q)
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const uint32_t f0[4] = {wa[r][0].x, wa[r][1].x, wa[r][0].y, wa[r][1].y};
            const uint32_t f1[4] = {wa[r][0].z, wa[r][1].z, wa[r][0].w, wa[r][1].w};
            mma_bf16_16816(acc[r][i], f0, xv[i][q][0], xv[i][q][1]);
            mma_bf16_16816(acc[r][i], f1, xv[i][q][2], xv[i][q][3]);
          }
      }
    }
    // acc[r][i]: ranks 16r + g (c 0, 1) and + 8 (c 2, 3) of rows 8i + 2t and + 1
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= tiles) break;
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          part[(warp * kShrinkRows + 8 * i + 2 * t + (c & 1)) * RP + r * 16 + g + 8 * (c >> 1)] = acc[r][i][c];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < count * RP; e += 32 * kShrinkWarps) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kShrinkWarps; ++w) s += part[w * kShrinkRows * RP + e];
      sum[e] = s;
    }
    cluster_sync();
    const float scale = a.scaling ? __ldg(a.scaling + id) : 1.0f;
    for (int e = ((int)rank * 32 * kShrinkWarps + (int)threadIdx.x) * 2; e < count * RP;
         e += 2 * 32 * kShrinkWarps * kShrinkCluster) {
      float v[2] = {0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < kShrinkCluster; ++c) {
        const uint32_t p = map_to_cta(sum + e, c);
        v[0] += ld_cluster_f32(p);
        v[1] += ld_cluster_f32(p + 4);
      }
      // (ranks that only pad: 0, also where x is infinite)
      const bool real = e % RP < a.rank;
      v[0] = real ? v[0] * scale : 0.0f;
      v[1] = real ? v[1] * scale : 0.0f;
      const uint32_t hi = bf16x2(v[0], v[1]);
      const uint32_t lo = bf16x2(isfinite(bf16_lo(hi)) ? v[0] - bf16_lo(hi) : 0.0f,
                                 isfinite(bf16_hi(hi)) ? v[1] - bf16_hi(hi) : 0.0f);
      const int64_t at = (m0 + __fns(rows, 0, e / RP + 1)) * (RP / 2) + (e % RP) / 2;
      a.hi[at] = hi;
      a.lo[at] = lo;
    }
    cluster_sync();  // the sums have been read
  }
}

constexpr int kExpandWarps = 4, kExpandRows = 64, kExpandCols = 64;

// A warp adds to 64 columns of 64 rows, 16 rows and 32 columns at a time. The
// MMA's columns are dealt out so that a lane's outputs of four MMAs are 8
// consecutive columns of two rows: column 2t + i of MMA j is column 8t + 2j + i.
// Ranks likewise: a lane's are 4t.. of 16.
template <bool kBf16, int RT>
__global__ void __launch_bounds__(32 * kExpandWarps) lora_expand_kernel(const LoraArgs a, const int vec) {
  constexpr int RP = RT * 16, kEs = kBf16 ? 2 : 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int col0 = ((int)blockIdx.x * kExpandWarps + warp) * kExpandCols;
  griddep_wait();
  if (col0 >= a.N) return;
  const int64_t r0 = (int64_t)blockIdx.y * kExpandRows;
  for (int64_t m0 = r0; m0 < min(r0 + kExpandRows, a.M); m0 += 16) {
    const int mine = lane < 16 ? adapter_of(a, m0 + lane) : -1;
    const uint32_t with = __ballot_sync(0xffffffffu, mine >= 0);
    if (with == 0 && a.base == a.out && a.ldb == a.ldo) continue;
    uint2 hi[RT][2], lo[RT][2];  // rows g and g + 8, ranks 16r + 4t..
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t at = (m0 + g + 8 * h) * (RP / 2) + r * 8 + t * 2;
        const bool has = with >> (g + 8 * h) & 1;  // (else it was never written)
        hi[r][h] = has ? *reinterpret_cast<const uint2*>(a.hi + at) : make_uint2(0, 0);
        lo[r][h] = has ? *reinterpret_cast<const uint2*>(a.lo + at) : make_uint2(0, 0);
      }
#pragma unroll
    for (int half = 0; half < kExpandCols / 32; ++half) {
      const int c0 = col0 + half * 32;
      if (c0 >= a.N) break;
      const int n0 = c0 + 8 * t;  // this lane's eight columns
      // base as it lies in memory
      uint32_t raw[2][kBf16 ? 4 : 8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t m = m0 + g + 8 * h;
        const char* p = reinterpret_cast<const char*>(a.base) + (m * a.ldb + n0) * kEs;
#pragma unroll
        for (int i = 0; i < (kBf16 ? 4 : 8); ++i) raw[h][i] = 0;
        if (m < a.M) {
          if (vec && n0 + 8 <= a.N) {
#pragma unroll
            for (int i = 0; i < (kBf16 ? 1 : 2); ++i) {
              const uint4 v = *reinterpret_cast<const uint4*>(p + 16 * i);
              raw[h][4 * i] = v.x;
              raw[h][4 * i + 1] = v.y;
              raw[h][4 * i + 2] = v.z;
              raw[h][4 * i + 3] = v.w;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (n0 + i < a.N) {
                if (kBf16)
                  raw[h][i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
                else
                  raw[h][i % (kBf16 ? 4 : 8)] = reinterpret_cast<const uint32_t*>(p)[i];
              }
          }
        }
      }
      float y[2][8];  // what is added to the rows
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) y[h][i] = 0.0f;
      for (uint32_t left = with; left;) {
        const int id = __shfl_sync(0xffffffffu, mine, __ffs(left) - 1);
        const uint32_t rows = __ballot_sync(0xffffffffu, mine == id);
        left &= ~rows;
        const uint16_t* pb = a.b + (int64_t)id * a.N * a.rank + 4 * t;
        float acc[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = c0 + 8 * (g >> 1) + 2 * j + (g & 1);
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[j][c] = 0.0f;
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const uint2 w = n < a.N && r * 16 + 4 * t < a.rank
                                ? __ldg(reinterpret_cast<const uint2*>(pb + (int64_t)n * a.rank + r * 16))
                                : make_uint2(0, 0);
            const uint32_t fl[4] = {lo[r][0].x, lo[r][1].x, lo[r][0].y, lo[r][1].y};
            const uint32_t fh[4] = {hi[r][0].x, hi[r][1].x, hi[r][0].y, hi[r][1].y};
            mma_bf16_16816(acc[j], fl, w.x, w.y);
            mma_bf16_16816(acc[j], fh, w.x, w.y);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (rows >> (g + 8 * h) & 1) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              y[h][2 * j] = acc[j][2 * h];
              y[h][2 * j + 1] = acc[j][2 * h + 1];
            }
          }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t m = m0 + g + 8 * h;
        if (m >= a.M) continue;
        if (with >> (g + 8 * h) & 1) {  // (a row without an adapter keeps base's bits)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (kBf16) {
              raw[h][i] = bf16x2(bf16_lo(raw[h][i]) + y[h][2 * i], bf16_hi(raw[h][i]) + y[h][2 * i + 1]);
            } else {
              constexpr int W = kBf16 ? 4 : 8;
              raw[h][2 * i % W] = __float_as_uint(__uint_as_float(raw[h][2 * i % W]) + y[h][2 * i]);
              raw[h][(2 * i + 1) % W] = __float_as_uint(__uint_as_float(raw[h][(2 * i + 1) % W]) + y[h][2 * i + 1]);
            }
          }
        }
        char* p = reinterpret_cast<char*>(a.out) + (m * a.ldo + n0) * kEs;
        if (vec && n0 + 8 <= a.N) {
#pragma unroll
          for (int i = 0; i < (kBf16 ? 1 : 2); ++i)
            *reinterpret_cast<uint4*>(p + 16 * i) =
                make_uint4(raw[h][4 * i], raw[h][4 * i + 1], raw[h][4 * i + 2], raw[h][4 * i + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n0 + i < a.N) {
              if (kBf16)
                reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(raw[h][i / 2] >> (16 * (i & 1)));
              else
                reinterpret_cast<uint32_t*>(p)[i] = raw[h][i % (kBf16 ? 4 : 8)];
            }
        }
      }
    }
  }
}

template <bool kXBf16, bool kBf16, int RT>
static cudaError_t launch_lora(const LoraArgs& a, cudaStream_t st) {
  const int windows = (int)ceil_div(a.M, kShrinkRows);
  // CTAs of a window share its adapters out: as many as fill the SMs eight times
  int z = 8 * num_sms() / (windows * kShrinkCluster);
  z = z < 1 ? 1 : z > kShrinkRows ? kShrinkRows : z;
  z = z < a.M ? z : (int)a.M;
  constexpr int smem = (kShrinkWarps + 1) * kShrinkRows * RT * 16 * 4;
  auto shrink = lora_shrink_kernel<kXBf16, RT>;
  static std::atomic<uint64_t> attr_set{0};
  cudaError_t e = smem_attr_once_per_device(shrink, smem, attr_set);
  if (e != cudaSuccess) return e;
  shrink<<<dim3(kShrinkCluster, windows, z), 32 * kShrinkWarps, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  constexpr int es = kBf16 ? 2 : 4;
  auto at16 = [](const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * es)) % 16 == 0; };
  const int vec = at16(a.base, a.ldb) && at16(a.out, a.ldo);
  return launch_kernel(lora_expand_kernel<kBf16, RT>,
                       dim3((unsigned)ceil_div(a.N, kExpandCols * kExpandWarps), (unsigned)ceil_div(a.M, kExpandRows)),
                       dim3(32 * kExpandWarps), 0, st, true, a, vec);
}

template <bool kXBf16, bool kBf16>
static cudaError_t launch_lora_any(const LoraArgs& a, cudaStream_t st) {
  if (a.rank <= 16) return launch_lora<kXBf16, kBf16, 1>(a, st);
  if (a.rank <= 32) return launch_lora<kXBf16, kBf16, 2>(a, st);
  if (a.rank <= 64) return launch_lora<kXBf16, kBf16, 4>(a, st);
  return launch_lora<kXBf16, kBf16, 8>(a, st);
}

// ranks that a row of the workspace holds
int lora_padded_rank(int64_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

cudaError_t launch_add_lora(const void* base, bool bf16, int64_t ldb, const void* x, bool x_bf16, int64_t M,
                            int64_t K, int64_t ldx, const void* A, const void* B, int64_t count, int64_t rank,
                            int64_t N, const int64_t* ids, const float* scaling, void* out, int64_t ldo, void* ws,
                            cudaStream_t st) {
  uint32_t* hi = reinterpret_cast<uint32_t*>(ws);
  const LoraArgs a{x, reinterpret_cast<const uint16_t*>(A), reinterpret_cast<const uint16_t*>(B), ids, scaling, base,
                   out, hi, hi + M * (lora_padded_rank(rank) / 2), ldx, ldb, ldo, M, (int)K, (int)N, (int)rank,
                   (int)count};
  if (x_bf16) return bf16 ? launch_lora_any<true, true>(a, st) : launch_lora_any<true, false>(a, st);
  return bf16 ? launch_lora_any<false, true>(a, st) : launch_lora_any<false, false>(a, st);
}

}  // namespace qg
