// gemm_fp8_small.cu -- block-scaled e4m3 product for few tokens (decode).
//
//   out[m][n] = chain over blocks b of 128, ascending:
//               acc = fmaf(sum_{k in b} q[m][k] * w[n][k], s[b][m] * ws[n/128][b], acc)
//
// Bound by reading the weights once: N*K bytes. So the weights are the MMA's
// long operand (R rows in tensor-memory lanes) and the tokens its short one
// (BM columns), and every CTA streams the rows of its tiles along K through a
// TMA ring as deep as shared memory allows; the ring runs on from tile to tile.
// Each block of 128 accumulates from zero in its own tensor-memory buffer (BM
// columns), and the epilogue warps apply the chain while the next blocks' MMAs
// run. The chain of an output is not split over CTAs, so its bits do not depend
// on the batch or the tile.
//
// The epilogue reads tensor memory as 16-lane fragments: a thread has 2 (R = 64)
// or 4 weight rows and a quarter of the tokens, so that all lanes of a 64-row
// tile have work, and a token's scale is read from shared memory once for those
// rows (17408 -> 5120, 64 tokens: 31 us; 37 with one row and 32 tokens a thread).
// The scales come through the ring with the operands, the weight scale is one
// number per tile and block.
//
// An MMA of this size takes 56 cycles from one issuing thread; each block of a
// stage has an issuing warp of its own (17408 -> 5120, 1 token: 20.5 us with one
// warp, 19.2 with two, 17.9 with four).
//
// Measured (from a CUDA graph): 16 tokens, 4096 -> 131072: 82.5 us, 6.56 TB/s of the
// 6.69 that a copy reaches; 64 tokens 87 us; 5120 -> 17408: 16.8 us, 18.4-19.1 with 64
// tokens, of which about 4 are a launch's fixed share; 17408 -> 5120: 17.7 us and
// 26.6 (80 tiles, each 136 blocks after one another: 163 cycles of MMAs a block,
// 200 to 340 with the handshakes and the loads).
//
// Warps: 0 TMA producer, 1..G MMA issuers, then the epilogue (4 per 32 tokens).
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
// the MMAs of one block of few tokens. (Of 128 rows and more than 16 tokens, a
// stage of four would leave a ring of two: 32 tokens, 5120 -> 17408 19.6 us, 17.2
// with stages of two.)
template <int R, int BM>
struct Fp8SmallCfg {
  static constexpr int G = R == 128 && BM > 16 ? 2 : 4;
  static constexpr uint32_t kW = R * 128, kQ = BM * 128, kS = BM * 4;
  static constexpr uint32_t kStage = G * (kW + kQ + kS);
  // groups of buffers: four, or what fits (the CTA has the SM's 512 columns)
  static constexpr uint32_t kCols = 4 * G * BM < 512 ? 4 * G * BM : 512;
  static constexpr int kGroups = kCols / (G * BM);
  // epilogue warps: four (a quarter of the lanes each) per 32 columns
  static constexpr int kCpt = BM < 32 ? BM : 32;  // columns per warp
  static constexpr int kEpi = 4 * (BM / kCpt), kEpi0 = 1 + G;
  static constexpr int kThreads = 32 * (kEpi0 + kEpi);
  static_assert(kGroups >= 2 && kGroups <= 4, "tensor memory");
};

struct Fp8SmallBars {
  uint64_t full[kFp8SmallMaxStages], empty[kFp8SmallMaxStages];
  uint64_t tfull[4], tempty[4];
  uint64_t mdrain[4];  // [issuer]
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
  const int tiles = (a.N + R - 1) / R, step = gridDim.x;
  const int total = (tiles - (int)blockIdx.x + step - 1) / step * NS;  // stages of this CTA's tiles

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], G + C::kEpi);  // the issuers' commits and the epilogue warps (scales)
    }
    for (int i = 0; i < C::kGroups; ++i) {
      mbar_init(&S.tfull[i], G);
      mbar_init(&S.tempty[i], C::kEpi);
    }
    for (int i = 0; i < G; ++i) mbar_init(&S.mdrain[i], 1);
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
    auto load_w = [&](int n0, int i, int s) {
      mbar_arrive_expect_tx(&S.full[s], C::kStage);
#pragma unroll
      for (int g = 0; g < G; ++g)
        tma_load_2d(sw + (s * G + g) * C::kW, &tmW, &S.full[s], (i * G + g) * 128, n0);
    };
    auto load_q = [&](int i, int s) {
#pragma unroll
      for (int g = 0; g < G; ++g)
        tma_load_2d(sq + (s * G + g) * C::kQ, &tmQ, &S.full[s], (i * G + g) * 128, 0);
      tma_load_2d(ss + s * G * C::kS, &tmS, &S.full[s], 0, i * G);
    };
    int n0 = blockIdx.x * R, i = 0;  // tile and stage of K
    auto next = [&] {
      if (++i == NS) { i = 0; n0 += step * R; }
    };
    // the first round of the ring: as a programmatic dependent of the
    // quantize kernel, the weights are requested before the wait for its grid
    const int P = min(total, stages);
    for (int l = 0; l < P; ++l, next())
      if (elect_one()) {
        load_w(n0, i, l);
        if (!a.pdl) load_q(i, l);
      }
    if (a.pdl) {
      griddep_wait();
      for (int l = 0; l < P; ++l)
        if (elect_one()) load_q(l % NS, l);
    }
    bool ok = true;
    int s = 0;
    uint32_t phase = 0;
    int last = P;  // loads issued
    for (; last < total; ++last, next()) {
      ok = mbar_wait_warp(&S.empty[s], phase, a.err);
      if (!ok) break;
      if (elect_one()) {
        // the epilogue warps read the slot's scales through the generic proxy
        // (ld.shared); the loads below rewrite them through the async proxy,
        // ordered after those reads only by this fence
        fence_proxy_async_smem();
        load_w(n0, i, s);
        load_q(i, s);
      }
      if (++s == stages) { s = 0; phase ^= 1; }
    }
    // every load has landed and (unless a wait gave up) every stage has been
    // released before the CTA exits
    for (int i = max(0, last - stages); i < last; ++i) {
      mbar_wait_warp(&S.full[i % stages], (uint32_t)(i / stages) & 1u, a.err);
      if (ok) mbar_wait_warp(&S.empty[i % stages], (uint32_t)(i / stages) & 1u, a.err);
    }
  } else if (warp <= G) {
    // one block of every stage
    constexpr uint32_t idesc = idesc_e4m3_f32(R, BM);
    const int g = warp - 1;
    int s = 0, t = 0;
    uint32_t phase = 0, tphase = 1;
    bool ok = true;
    for (int i = 0; i < total; ++i) {
      ok = mbar_wait_warp2(&S.full[s], phase, &S.tempty[t], tphase, a.err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t wa = smem_u32(sw + (s * G + g) * C::kW);
      const uint32_t qa = smem_u32(sq + (s * G + g) * C::kQ);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_e4m3_ss(tmem + (t * G + g) * BM, smem_desc_sw128(wa + k * 32),
                      smem_desc_sw128(qa + k * 32), idesc, k);
        mma_commit(&S.tfull[t]);
        mma_commit(&S.empty[s]);
      }
      __syncwarp();
      if (++s == stages) { s = 0; phase ^= 1; }
      if (++t == C::kGroups) { t = 0; tphase ^= 1; }
    }
    if (!ok) {
      if (elect_one()) mma_commit(&S.mdrain[g]);
      __syncwarp();
      if (!mbar_wait_warp(&S.mdrain[g], 0, a.err)) atomicExch(&S.tmem_busy, 1u);
    }
  } else {
    const int quarter = warp & 3, c0 = ((warp - C::kEpi0) >> 2) * C::kCpt;  // lanes and columns of this warp
    constexpr int kCpt = C::kCpt;
    constexpr int H = R / 64;  // 16-lane halves of the quarter in use
    // R = 128: row i in lane i; R = 64: rows 16w.. in the first lanes of quarter w
    const int row = quarter * (R / 4) + (lane >> 2);
    // the weight scales of 32 blocks, one per lane, the next 32 on their way
    // (a tile lies inside one block of rows)
    auto scales = [&](int tile) { return a.w_scale + (int64_t)(tile * R >> 7) * KB; };
    float w_first = lane < KB ? __ldg(scales(blockIdx.x) + lane) : 0.0f;  // a tile's first
    if (a.pdl) griddep_wait();  // the output may be what an earlier kernel still reads
    int s = 0, t = 0;
    uint32_t phase = 0, tphase = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < tiles && ok; tile += step) {
      const float* wsp = scales(tile);
      float w_cur = w_first;
      float w_nxt = 32 + lane < KB ? ldg_f32_pinned(wsp + 32 + lane) : 0.0f;
      if (tile + step < tiles && lane < KB) w_first = ldg_f32_pinned(scales(tile + step) + lane);
      float acc[H][kCpt / 2];
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < kCpt / 2; ++j) acc[h][j] = 0.0f;
      for (int i = 0; i < NS; ++i) {
        ok = mbar_wait_warp2(&S.full[s], phase, &S.tfull[t], tphase, a.err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + t * G * BM + c0;
        const float* sc = reinterpret_cast<const float*>(ss + s * G * C::kS) + c0 + 2 * (lane & 3);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int b = i * G + g;
          uint32_t v[H][kCpt / 2];
#pragma unroll
          for (int h = 0; h < H; ++h) tmem_ld_frag(taddr + (h << 20) + g * BM, v[h]);
          const float wsc = __shfl_sync(0xffffffffu, w_cur, b & 31);
          if ((b & 31) == 31) {
            w_cur = w_nxt;
            w_nxt = b + 33 + lane < KB ? ldg_f32_pinned(wsp + b + 33 + lane) : 0.0f;
          }
          const float2 w2 = make_float2(wsc, wsc);
          float2 f[kCpt / 8];
#pragma unroll
          for (int j = 0; j < kCpt / 8; ++j)
            f[j] = __fmul2_rn(*reinterpret_cast<const float2*>(sc + g * BM + 8 * j), w2);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int j = 0; j < kCpt / 2; ++j) asm volatile("" : "+r"(v[h][j]));
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
          for (int j = 0; j < kCpt / 8; ++j)
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
              for (int u = 0; u < 4; u += 2) {
                float* ac = acc[h] + 4 * j + u;
                const float2 r = __ffma2_rn(make_float2(__uint_as_float(v[h][4 * j + u]),
                                                        __uint_as_float(v[h][4 * j + u + 1])),
                                            f[j], make_float2(ac[0], ac[1]));
                ac[0] = r.x;
                ac[1] = r.y;
              }
        }
        if (++s == stages) { s = 0; phase ^= 1; }
        if (++t == C::kGroups) { t = 0; tphase ^= 1; }
      }
      if (!ok) break;
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < kCpt / 2; ++j) {
          const int m = c0 + 8 * (j >> 2) + 2 * (lane & 3) + (j & 1);
          const int n = tile * R + row + 16 * h + 8 * (j >> 1 & 1);
          if (m >= a.M || n >= a.N) continue;
          const int64_t o = (int64_t)m * a.ldo + n;
          if (a.out_f32)
            reinterpret_cast<float*>(a.out)[o] = acc[h][j];
          else
            reinterpret_cast<uint16_t*>(a.out)[o] = f32_to_bf16_rne(acc[h][j]);
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
      !make_tmap_2d(&ts, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, scale, a.M, a.KB, lds * 4, BM,
                    C::G, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorNotSupported;
  // one CTA per SM, with the whole shared memory for its ring
  const int64_t tiles = ceil_div(a.N, R);
  const dim3 grid((unsigned)(tiles < num_sms() ? tiles : num_sms()));
  int stages = 223 * 1024 / (int)C::kStage;
  stages = stages > kFp8SmallMaxStages ? kFp8SmallMaxStages : stages;
  a.stages = stages;
  const size_t smem = (size_t)stages * C::kStage + 1024;
  auto kern = gemm_fp8_small_kernel<R, BM>;
  static std::atomic<uint64_t> attr_set{0};
  const cudaError_t e = smem_attr_once_per_device(kern, 224 * 1024, attr_set);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, grid, dim3(C::kThreads), smem, st, pdl, tw, tq, ts, a);
}

// Tile of up to 64 tokens. 64-row tiles while all of them run at once, else 128-row
// tiles, which read the tokens half as often (16 tokens: 17408 -> 5120, 80 tiles 17.7
// us, 24.4 as 40 of 128; 5120 -> 10000, 157 tiles 13.8 us, 12.6 as 79)
void fp8_small_tile(int64_t M, int64_t N, int sms, int* tokens, int* rows) {
  *tokens = M <= 16 ? 16 : M <= 32 ? 32 : 64;
  *rows = ceil_div(N, 64) <= sms ? 64 : 128;
}

cudaError_t launch_gemm_fp8_small(const uint8_t* q, const float* scale, int64_t lds, int64_t M,
                                  int64_t K, const uint8_t* w, int64_t ldw, const float* w_scale,
                                  int64_t N, void* out, bool out_f32, int64_t ldo, uint32_t* err,
                                  bool pdl, cudaStream_t st) {
  int bm, r;
  fp8_small_tile(M, N, num_sms(), &bm, &r);
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
