// gemm_fp8_grouped.cu -- block-scaled e4m3 product of each row with the weights
// of its expert. Rows are sorted by expert: expert e owns rows offsets[e] up to
// offsets[e + 1], numbers that only the device knows.
//
//   out[m][n] = chain over blocks b of 128, ascending, e the expert of row m:
//               acc = fmaf(sum_{k in b} q[m][k] * w[e][n][k], s[b][m] * ws[e][n/128][b], acc)
//
// The order of gemm_fp8, so that a row's bits are those of gemm_fp8 with its
// expert's weights, whatever the other rows are.
//
// Every CTA forms the list of tiles from the offsets (a scan over the experts,
// then a 32-way search per tile) and takes every gridDim-th tile of it: no
// kernel before this one, no workspace, nothing to wait for on the host.
//
// Few rows an expert: bound by reading the weights once, as gemm_fp8 of few tokens,
// and made alike: a tile is R weight rows of one expert (the MMA's long operand, in
// tensor-memory lanes) and up to BM of its rows (columns), a persistent CTA's ring of
// TMA loads runs on from tile to tile, blocks of 128 accumulate from zero in buffers
// of their own. The tiles of the same weights follow one another, so that weights
// come from HBM once. 512 rows of 64 experts, 2560 -> 2432: 63.5 us, 6.3 TB/s.
// Many rows an expert: the prefill kernel's tiles (gemm_fp8_large.cu).
#include <cuda.h>

#include "gemm_grouped.cuh"

namespace qg {

bool make_tmap_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols,
                  int64_t rows, int64_t pitch, uint32_t box_cols, uint32_t box_rows,
                  CUtensorMapSwizzle swizzle);
bool make_tmap_3d(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols,
                  int64_t rows, int64_t mats, int64_t pitch, int64_t mat_pitch, uint32_t box_cols,
                  uint32_t box_rows, CUtensorMapSwizzle swizzle);

cudaError_t launch_gemm_fp8_grouped_large(const uint8_t* q, const float* scale, int64_t lds, int64_t M, int64_t K,
                                          const int64_t* offsets, int64_t E, const uint8_t* w, int64_t ldw,
                                          int64_t lde, const float* w_scale, int64_t N, void* out, bool out_f32,
                                          int64_t ldo, uint32_t* err, cudaStream_t st);
void fp8_grouped_large_tile(int64_t M, int64_t N, int64_t E, int sms, int* tokens, int* rows);

struct Fp8GroupedArgs {
  const int64_t* offsets;  // [E + 1]
  const float* w_scale;    // [E][ceil(N/128)][KB]
  void* out;
  int64_t ldo;
  int M, N, E, KB, NB, stages;
  int out_f32;
  uint32_t* err;
};

constexpr int kGroupedMaxStages = 16;

// G blocks of K share a ring stage, a group of tensor-memory buffers and their
// barriers.
template <int R, int BM>
struct GroupedCfg {
  static constexpr int G = R == 128 && BM > 16 ? 2 : 4;
  // a row of scales has to start on a multiple of four rows: four more are loaded
  static constexpr uint32_t kW = R * 128, kQ = BM * 128, kSRow = BM + 4;
  static constexpr uint32_t kSBytes = G * kSRow * 4, kS = (kSBytes + 127) / 128 * 128;
  static constexpr uint32_t kStage = G * (kW + kQ) + kS, kLoad = G * (kW + kQ) + kSBytes;
  static constexpr uint32_t kCols = 4 * G * BM < 512 ? 4 * G * BM : 512;
  static constexpr int kGroups = kCols / (G * BM);
  static constexpr int kCpt = BM < 32 ? BM : 32;  // columns per epilogue warp
  static constexpr int kEpi = 4 * (BM / kCpt), kEpi0 = 1 + G;
  static constexpr int kThreads = 32 * (kEpi0 + kEpi);
  static_assert(kGroups >= 2 && kGroups <= 4, "tensor memory");
};

struct GroupedBars {
  uint64_t full[kGroupedMaxStages], empty[kGroupedMaxStages];
  uint64_t tfull[4], tempty[4];
  uint64_t mdrain[4];  // [issuer]
  uint32_t tmem_base, tmem_busy;
};

template <int R, int BM>
__global__ void __launch_bounds__(GroupedCfg<R, BM>::kThreads, 1)
    gemm_fp8_grouped_kernel(const __grid_constant__ CUtensorMap tmW,
                            const __grid_constant__ CUtensorMap tmQ,
                            const __grid_constant__ CUtensorMap tmS, const Fp8GroupedArgs a) {
  using C = GroupedCfg<R, BM>;
  constexpr int G = C::G;
  extern __shared__ uint8_t smem_raw[];
  __shared__ GroupedBars S;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int stages = a.stages, KB = a.KB;
  const int NS = (KB + G - 1) / G;               // stages of K; the tail's blocks past K read as zero
  uint8_t* sw = base;                            // weight tiles [stage][G]
  uint8_t* sq = sw + stages * G * C::kW;         // rows' tiles [stage][G]
  uint8_t* ss = sq + stages * G * C::kQ;         // rows' scales [stage][G][BM + 4]
  int* first = reinterpret_cast<int*>(ss + stages * C::kS);  // [E + 1]
  int* before = first + a.E + 1;                             // [E + 1]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

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
  if (warp == 0) {
    if (elect_one()) {
      tma_prefetch_desc(&tmW);
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmS);
    }
    __syncwarp();
  }
  if (warp == 1) {
    tmem_alloc(&S.tmem_base, C::kCols);
    tmem_relinquish();
  }
  if (warp == 2) GroupedTiles::fill(a.offsets, a.E, a.M, BM, first, before);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  const GroupedTiles T{first, before, a.E, (a.N + R - 1) / R};
  const int tiles = T.total(), step = gridDim.x;
  const int total =
      (int)blockIdx.x < tiles ? (tiles - (int)blockIdx.x + step - 1) / step * NS : 0;  // stages of this CTA's tiles

  if (warp == 0) {
    bool ok = true;
    int s = 0, loads = 0;
    uint32_t phase = 1;
    for (int t = blockIdx.x; t < tiles && ok; t += step) {
      int e, mi, ni;
      T.at(t, e, mi, ni);
      const int m0 = first[e] + mi * BM, n0 = ni * R;
      for (int i = 0; i < NS; ++i) {
        ok = mbar_wait_warp(&S.empty[s], phase, a.err);
        if (!ok) break;
        if (elect_one()) {
          // the epilogue warps read the slot's scales through the generic proxy
          // (ld.shared); the loads below rewrite them through the async proxy,
          // ordered after those reads only by this fence
          fence_proxy_async_smem();
          mbar_arrive_expect_tx(&S.full[s], C::kLoad);
#pragma unroll
          for (int g = 0; g < G; ++g)
            tma_load_3d(sw + (s * G + g) * C::kW, &tmW, &S.full[s], (i * G + g) * 128, n0, e);
#pragma unroll
          for (int g = 0; g < G; ++g)
            tma_load_2d(sq + (s * G + g) * C::kQ, &tmQ, &S.full[s], (i * G + g) * 128, m0);
          tma_load_2d(ss + s * C::kS, &tmS, &S.full[s], m0 & ~3, i * G);
        }
        __syncwarp();
        ++loads;
        if (++s == stages) { s = 0; phase ^= 1; }
      }
    }
    // every load has landed and (unless a wait gave up) every stage has been
    // released before the CTA exits
    for (int i = max(0, loads - stages); i < loads; ++i) {
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
    auto scales = [&](int e, int ni) { return a.w_scale + ((int64_t)e * a.NB + (ni * R >> 7)) * KB; };
    int e = 0, mi = 0, ni = 0;
    float w_first = 0.0f;  // a tile's first
    if ((int)blockIdx.x < tiles) {
      T.at(blockIdx.x, e, mi, ni);
      if (lane < KB) w_first = __ldg(scales(e, ni) + lane);
    }
    int s = 0, t = 0;
    uint32_t phase = 0, tphase = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < tiles && ok; tile += step) {
      const float* wsp = scales(e, ni);
      const int m0 = first[e] + mi * BM, rows = min(BM, first[e + 1] - m0), n0 = ni * R;
      float w_cur = w_first;
      float w_nxt = 32 + lane < KB ? ldg_f32_pinned(wsp + 32 + lane) : 0.0f;
      if (tile + step < tiles) {
        T.at(tile + step, e, mi, ni);
        if (lane < KB) w_first = ldg_f32_pinned(scales(e, ni) + lane);
      }
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
        const float* sc = reinterpret_cast<const float*>(ss + s * C::kS) + (m0 & 3) + c0 + 2 * (lane & 3);
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
          for (int j = 0; j < kCpt / 8; ++j) {
            const float* p = sc + g * C::kSRow + 8 * j;
            f[j] = __fmul2_rn(make_float2(p[0], p[1]), w2);
          }
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
          const int n = n0 + row + 16 * h + 8 * (j >> 1 & 1);
          if (m >= rows || n >= a.N) continue;
          const int64_t o = (int64_t)(m0 + m) * a.ldo + n;
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
static cudaError_t launch_grouped(const uint8_t* q, const float* scale, int64_t lds, int64_t K, const uint8_t* w,
                                  int64_t ldw, int64_t lde, Fp8GroupedArgs a, cudaStream_t st) {
  using C = GroupedCfg<R, BM>;
  CUtensorMap tw, tq, ts;
  if (!make_tmap_3d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, K, a.N, a.E, ldw, lde, 128, R,
                    CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, K, a.M, K, 128, BM,
                    CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&ts, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, scale, a.M, a.KB, lds * 4, C::kSRow,
                    C::G, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorNotSupported;
  // one CTA per SM, with the whole shared memory for its ring
  const int64_t most = ((a.M < a.E ? a.M : a.E) + a.M / BM) * ceil_div(a.N, R);
  const unsigned grid = (unsigned)(most < num_sms() ? most : num_sms());
  const int list = GroupedTiles::bytes(a.E);
  int stages = (223 * 1024 - list) / (int)C::kStage;
  stages = stages > kGroupedMaxStages ? kGroupedMaxStages : stages;
  a.stages = stages;
  const size_t smem = (size_t)stages * C::kStage + list + 1024;
  auto kern = gemm_fp8_grouped_kernel<R, BM>;
  static std::atomic<uint64_t> attr_set{0};
  const cudaError_t e = smem_attr_once_per_device(kern, 224 * 1024, attr_set);
  if (e != cudaSuccess) return e;
  kern<<<grid, C::kThreads, smem, st>>>(tw, tq, ts, a);
  return cudaGetLastError();
}

// Tiles of 16 columns while all of them run at once (at most one more than the full
// ones for every expert with rows): weights in 64 rows, 1 row of 64 experts, 17408 ->
// 2560 18.7 us (128 rows 24.7), else in 128, 100 rows of 2 experts, 2560 -> 2432 7.9
// (32 columns 8.7; the prefill kernel 9.9). Then by the mean rows of an expert: 512
// rows of 64 experts 64.0, 65.6, 70.1; 2048 rows 78.8, 71.1, 73.8; 3000 rows 99, 83,
// 72.8; 160 rows of 8 13.8, 14.8, 14.1. (Measured with nearly even experts: their rows
// are not known here, and any tile is right for any of them.)
void fp8_grouped_tile(int64_t M, int64_t N, int64_t E, int sms, int* tokens, int* rows) {
  const int64_t tiles = (M < E ? M : E) + M / 16, mean = M / E;
  *tokens = 16;
  *rows = 64;
  if (ceil_div(N, 64) * tiles <= sms) return;
  *rows = 128;
  if (ceil_div(N, 128) * tiles <= sms || mean <= 12) return;
  *tokens = 32;
  if (mean <= 32) return;
  fp8_grouped_large_tile(M, N, E, sms, tokens, rows);
}

cudaError_t launch_gemm_fp8_grouped(const uint8_t* q, const float* scale, int64_t lds, int64_t M, int64_t K,
                                    const int64_t* offsets, int64_t E, const uint8_t* w, int64_t ldw, int64_t lde,
                                    const float* w_scale, int64_t N, void* out, bool out_f32, int64_t ldo,
                                    uint32_t* err, cudaStream_t st) {
  const Fp8GroupedArgs a{offsets, w_scale, out, ldo, (int)M, (int)N, (int)E, (int)ceil_div(K, 128),
                         (int)ceil_div(N, 128), 0, out_f32, err};
  int tokens, rows;
  fp8_grouped_tile(M, N, E, num_sms(), &tokens, &rows);
  if (tokens == 16 && rows == 64) return launch_grouped<64, 16>(q, scale, lds, K, w, ldw, lde, a, st);
  if (tokens == 16) return launch_grouped<128, 16>(q, scale, lds, K, w, ldw, lde, a, st);
  if (tokens == 32) return launch_grouped<128, 32>(q, scale, lds, K, w, ldw, lde, a, st);
  return launch_gemm_fp8_grouped_large(q, scale, lds, M, K, offsets, E, w, ldw, lde, w_scale, N, out, out_f32, ldo, err,
                                       st);
}

}  // namespace qg
