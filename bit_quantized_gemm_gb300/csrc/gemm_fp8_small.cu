// gemm_fp8_small.cu -- block-scaled e4m3 product for few tokens (decode).
//
//   out[m][n] = chain over blocks b of 128, ascending:
//               acc = fmaf(sum_{k in b} q[m][k] * w[n][k], s[b][m] * ws[n/128][b], acc)
//
// Bound by reading the weights once: N*K bytes. So the weights are the MMA's
// long operand (R rows in tensor-memory lanes) and the tokens its short one
// (BM columns), and every CTA streams its R rows along K through a TMA ring
// as deep as shared memory allows. Each block of 128 accumulates from zero in
// its own tensor-memory buffer (BM columns), and the epilogue warps apply the
// chain while the next blocks' MMAs run: a thread owns one weight row and up
// to 32 tokens, the token scales come through the ring with the operands, the
// weight scale is one number per tile and block.
// The chain of an output is not split over CTAs, so its bits do not depend on
// the batch or the tile.
//
// Warps: 0 TMA producer, 1 MMA issuer, then the epilogue (4 per 32 tokens).
#include <cuda.h>

#include "qg_common.cuh"

namespace qg {

bool make_tmap_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols,
                  int64_t rows, int64_t pitch, uint32_t box_cols, uint32_t box_rows,
                  CUtensorMapSwizzle swizzle);

struct Fp8SmallArgs {
  const float* w_scale;  // [ceil(N/128)][KB]
  void* out;
  int64_t ldo;
  int M, N, KB, stages;
  int out_f32, pdl;
  uint32_t* err;
};

constexpr int kFp8SmallMaxStages = 16;

// G blocks of K share a ring stage, a group of tensor-memory buffers and their
// barriers: a barrier wait costs 100-200 cycles beside running MMAs, more than
// the MMAs of one block of few tokens.
template <int R, int BM>
struct Fp8SmallCfg {
  static constexpr int G = BM <= 32 ? 4 : 2;
  static constexpr uint32_t kW = R * 128, kQ = BM * 128, kS = BM * 4;
  static constexpr uint32_t kStage = G * (kW + kQ + kS);
  // groups of buffers: 256 columns, so that two CTAs can share an SM
  static constexpr int kGroups = 256 / (G * BM);
  static constexpr uint32_t kCols = kGroups * G * BM;
  // epilogue warps: four (a quarter of the lanes each) per 32 columns
  static constexpr int kCpt = BM < 32 ? BM : 32;  // columns per thread
  static constexpr int kEpi = 4 * (BM / kCpt);
  static constexpr int kThreads = 64 + 32 * kEpi;
  static_assert(kGroups >= 2 && (kCols & (kCols - 1)) == 0, "tensor memory");
};

struct Fp8SmallBars {
  uint64_t full[kFp8SmallMaxStages], empty[kFp8SmallMaxStages];
  uint64_t tfull[4], tempty[4];
  uint64_t mdrain;
  uint32_t tmem_base, tmem_busy;
};

template <int R, int BM>
__global__ void __launch_bounds__(Fp8SmallCfg<R, BM>::kThreads)
    gemm_fp8_small_kernel(const __grid_constant__ CUtensorMap tmW,
                          const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmS, const Fp8SmallArgs a) {
  using C = Fp8SmallCfg<R, BM>;
  constexpr int G = C::G;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Fp8SmallBars S;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int stages = a.stages, KB = a.KB;
  const int NS = (KB + G - 1) / G;               // stages of K; the tail's blocks past K read as zero
  uint8_t* sw = base;                            // weight tiles [stage][G]
  uint8_t* sq = sw + stages * G * C::kW;         // token tiles [stage][G]
  uint8_t* ss = sq + stages * G * C::kQ;         // token scales [stage][G][BM]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * R, m0 = blockIdx.y * BM;

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1 + C::kEpi);  // the MMAs' commit and the epilogue warps (scales)
    }
    for (int i = 0; i < C::kGroups; ++i) {
      mbar_init(&S.tfull[i], 1);
      mbar_init(&S.tempty[i], C::kEpi);
    }
    mbar_init(&S.mdrain, 1);
    S.tmem_busy = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmS);
  }
  if (warp == 1) {
    tmem_alloc(&S.tmem_base, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;

  if (warp == 0) {
    auto load_w = [&](int i, int s) {
      mbar_arrive_expect_tx(&S.full[s], C::kStage);
#pragma unroll
      for (int g = 0; g < G; ++g)
        tma_load_2d(sw + (s * G + g) * C::kW, &tmW, &S.full[s], (i * G + g) * 128, n0);
    };
    auto load_q = [&](int i, int s) {
#pragma unroll
      for (int g = 0; g < G; ++g)
        tma_load_2d(sq + (s * G + g) * C::kQ, &tmQ, &S.full[s], (i * G + g) * 128, m0);
      tma_load_2d(ss + s * G * C::kS, &tmS, &S.full[s], m0, i * G);
    };
    // the first round of the ring: as a programmatic dependent of the
    // quantize kernel, the weights are requested before the wait for its grid
    const int P = min(NS, stages);
    for (int i = 0; i < P; ++i)
      if (elect_one()) {
        load_w(i, i);
        if (!a.pdl) load_q(i, i);
      }
    if (a.pdl) {
      griddep_wait();
      for (int i = 0; i < P; ++i)
        if (elect_one()) load_q(i, i);
    }
    bool ok = true;
    int s = 0;
    uint32_t phase = 0;
    int last = P;  // loads issued
    for (int i = P; i < NS; ++i) {
      ok = mbar_wait_warp(&S.empty[s], phase, a.err);
      if (!ok) break;
      if (elect_one()) {
        load_w(i, s);
        load_q(i, s);
      }
      ++last;
      if (++s == stages) { s = 0; phase ^= 1; }
    }
    // every load has landed and (unless a wait gave up) every stage has been
    // released before the CTA exits
    for (int i = max(0, last - stages); i < last; ++i) {
      mbar_wait_warp(&S.full[i % stages], (uint32_t)(i / stages) & 1u, a.err);
      if (ok) mbar_wait_warp(&S.empty[i % stages], (uint32_t)(i / stages) & 1u, a.err);
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_e4m3_f32(R, BM);
    int s = 0, t = 0;
    uint32_t phase = 0, tphase = 1;
    bool ok = true;
    for (int i = 0; i < NS; ++i) {
      ok = mbar_wait_warp2(&S.full[s], phase, &S.tempty[t], tphase, a.err);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint32_t wa = smem_u32(sw + (s * G + g) * C::kW);
          const uint32_t qa = smem_u32(sq + (s * G + g) * C::kQ);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_e4m3_ss(tmem + (t * G + g) * BM, smem_desc_sw128(wa + k * 32),
                        smem_desc_sw128(qa + k * 32), idesc, k);
        }
        mma_commit(&S.tfull[t]);
        mma_commit(&S.empty[s]);
      }
      __syncwarp();
      if (++s == stages) { s = 0; phase ^= 1; }
      if (++t == C::kGroups) { t = 0; tphase ^= 1; }
    }
    if (!ok) {
      if (elect_one()) mma_commit(&S.mdrain);
      __syncwarp();
      if (!mbar_wait_warp(&S.mdrain, 0, a.err)) atomicExch(&S.tmem_busy, 1u);
    }
  } else {
    const int quarter = warp & 3, c0 = ((warp - 2) >> 2) * C::kCpt;  // lanes and columns of this warp
    constexpr int kCpt = C::kCpt;
    // M = 128: row i in lane i; M = 64: rows 16w.. in the first lanes of quarter w
    const int n = n0 + quarter * (R / 4) + lane;
    const bool nvalid = lane < R / 4 && n < a.N;
    // the weight scales of 32 blocks, one per lane, the next 32 on their way
    // (a tile lies inside one block of rows)
    const float* wsp = a.w_scale + (int64_t)(n0 >> 7) * KB;
    float w_cur = lane < KB ? __ldg(wsp + lane) : 0.0f;
    float w_nxt = 32 + lane < KB ? ldg_f32_pinned(wsp + 32 + lane) : 0.0f;
    if (a.pdl) griddep_wait();  // the output may be what an earlier kernel still reads
    float acc[kCpt];
#pragma unroll
    for (int j = 0; j < kCpt; ++j) acc[j] = 0.0f;
    int s = 0, t = 0;
    uint32_t phase = 0, tphase = 0;
    bool ok = true;
    for (int i = 0; i < NS; ++i) {
      ok = mbar_wait_warp2(&S.full[s], phase, &S.tfull[t], tphase, a.err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + t * G * BM + c0;
      const float* sc = reinterpret_cast<const float*>(ss + s * G * C::kS) + c0;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int b = i * G + g;
        const float wsc = __shfl_sync(0xffffffffu, w_cur, b & 31);
        if ((b & 31) == 31) {
          w_cur = w_nxt;
          w_nxt = b + 33 + lane < KB ? ldg_f32_pinned(wsp + b + 33 + lane) : 0.0f;
        }
        const float2 w2 = make_float2(wsc, wsc);
        uint32_t v[kCpt];
        tmem_ld(taddr + g * BM, v);
        float2 f[kCpt / 2];
#pragma unroll
        for (int j = 0; j < kCpt; j += 4) {
          const float4 f4 = *reinterpret_cast<const float4*>(sc + g * BM + j);
          f[j / 2] = __fmul2_rn(make_float2(f4.x, f4.y), w2);
          f[j / 2 + 1] = __fmul2_rn(make_float2(f4.z, f4.w), w2);
        }
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < kCpt; ++j) asm volatile("" : "+r"(v[j]));
        if (g + 1 == G) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&S.tempty[t]);
            mbar_arrive(&S.empty[s]);  // this warp has read the stage's scales, too
          }
        }
        if (b >= KB) continue;  // past K
#pragma unroll
        for (int j = 0; j < kCpt; j += 2) {
          const float2 r = __ffma2_rn(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])),
                                      f[j / 2], make_float2(acc[j], acc[j + 1]));
          acc[j] = r.x;
          acc[j + 1] = r.y;
        }
      }
      if (++s == stages) { s = 0; phase ^= 1; }
      if (++t == C::kGroups) { t = 0; tphase ^= 1; }
    }
    if (ok && nvalid) {
      const int64_t o = (int64_t)(m0 + c0) * a.ldo + n;
      const int mc = a.M - m0 - c0;
#pragma unroll
      for (int j = 0; j < kCpt; ++j) {
        if (j >= mc) continue;
        if (a.out_f32)
          reinterpret_cast<float*>(a.out)[o + j * a.ldo] = acc[j];
        else
          reinterpret_cast<uint16_t*>(a.out)[o + j * a.ldo] = f32_to_bf16_rne(acc[j]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1 && S.tmem_busy == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

template <int R, int BM>
static cudaError_t launch_small(const CUtensorMap& tw, const uint8_t* q, const float* scale, int64_t lds,
                                int64_t K, Fp8SmallArgs a, bool pdl, cudaStream_t st) {
  using C = Fp8SmallCfg<R, BM>;
  CUtensorMap tq, ts;
  if (!make_tmap_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, K, a.M, K, 128, BM,
                    CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&ts, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, scale, align_up(a.M, 4), a.KB, lds * 4, BM,
                    C::G, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorNotSupported;
  const dim3 grid((unsigned)ceil_div(a.N, R), (unsigned)ceil_div(a.M, BM));
  // one CTA per SM takes the whole shared memory for its ring; two share it
  const int64_t ctas = (int64_t)grid.x * grid.y;
  const int budget = (ctas <= num_sms() ? 224 : 110) * 1024 - 1024;
  int stages = budget / (int)C::kStage;
  stages = stages > kFp8SmallMaxStages ? kFp8SmallMaxStages : stages;
  const int ns = (int)ceil_div(a.KB, C::G);
  stages = stages > ns ? ns : stages;
  a.stages = stages;
  const size_t smem = (size_t)stages * C::kStage + 1024;
  auto kern = gemm_fp8_small_kernel<R, BM>;
  static std::atomic<uint64_t> attr_set{0};
  const cudaError_t e = smem_attr_once_per_device(kern, 224 * 1024, attr_set);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, grid, dim3(C::kThreads), smem, st, pdl, tw, tq, ts, a);
}

cudaError_t launch_gemm_fp8_small(const uint8_t* q, const float* scale, int64_t lds, int64_t M,
                                  int64_t K, const uint8_t* w, int64_t ldw, const float* w_scale,
                                  int64_t N, void* out, bool out_f32, int64_t ldo, uint32_t* err,
                                  bool pdl, cudaStream_t st) {
  const int bm = M <= 16 ? 16 : M <= 32 ? 32 : 64;
  // 128-row tiles read the tokens half as often; 64-row tiles fill the SMs
  const int r = ceil_div(N, 128) * ceil_div(M, bm) * 4 >= 3 * num_sms() ? 128 : 64;
  CUtensorMap tw;
  if (!make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, K, N, ldw, 128, r,
                    CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorNotSupported;
  Fp8SmallArgs a{w_scale, out, ldo, (int)M, (int)N, (int)ceil_div(K, 128), 0, out_f32, pdl, err};
  if (r == 64) switch (bm) {
    case 16: return launch_small<64, 16>(tw, q, scale, lds, K, a, pdl, st);
    case 32: return launch_small<64, 32>(tw, q, scale, lds, K, a, pdl, st);
    default: return launch_small<64, 64>(tw, q, scale, lds, K, a, pdl, st);
  }
  switch (bm) {
    case 16: return launch_small<128, 16>(tw, q, scale, lds, K, a, pdl, st);
    case 32: return launch_small<128, 32>(tw, q, scale, lds, K, a, pdl, st);
    default: return launch_small<128, 64>(tw, q, scale, lds, K, a, pdl, st);
  }
}

}  // namespace qg
