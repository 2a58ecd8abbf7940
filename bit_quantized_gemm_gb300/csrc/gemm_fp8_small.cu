// gemm_fp8_small.cu -- block-scaled e4m3 product for few tokens (decode).
//
//   out[m][n] = chain over blocks b of 128, ascending:
//               acc = fmaf(sum_{k in b} q[m][k] * w[n][k], s[b][m] * ws[n/128][b], acc)
//
// Bound by reading the weights once: N*K bytes. So the weights are the MMA's
// long operand (R rows in tensor-memory lanes) and the tokens its short one
// (BM columns), and every CTA streams its R rows along K through a TMA ring
// as deep as shared memory allows. Each block of 128 accumulates from zero in
// its own tensor-memory buffer (BM columns; the next blocks' MMAs run
// meanwhile), and four epilogue warps apply the chain: a thread owns one
// weight row and all BM tokens, the block's token scales come through the
// ring with its operands, the weight scale is one number per tile and block.
// The chain of an output is not split over CTAs, so its bits do not depend on
// the batch or the tile.
//
// Warps (192 threads): 0 TMA producer, 1 MMA issuer, 2..5 epilogue.
#include <cuda.h>

#include "qg_common.cuh"

namespace qg {

bool make_tmap_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols,
                  int64_t rows, int64_t pitch, uint32_t box_cols, uint32_t box_rows,
                  CUtensorMapSwizzle swizzle);

struct Fp8SmallArgs {
  const float* scale;    // [KB][lds]
  const float* w_scale;  // [ceil(N/128)][KB]
  void* out;
  int64_t lds, ldo;
  int M, N, KB, stages;
  int out_f32, pdl;
  uint32_t* err;
};

constexpr int kFp8SmallMaxStages = 32;

template <int R, int BM>
struct Fp8SmallCfg {
  static constexpr uint32_t kW = R * 128, kQ = BM * 128, kS = BM * 4;
  static constexpr uint32_t kStage = kW + kQ + kS;
  static constexpr int kBufs = 256 / BM < 8 ? 256 / BM : 8;
  static constexpr uint32_t kCols = kBufs * BM < 32 ? 32 : kBufs * BM;  // a power of two
  static constexpr int kChunk = BM < 32 ? 16 : 32;                      // columns per load
};

struct Fp8SmallBars {
  uint64_t full[kFp8SmallMaxStages], empty[kFp8SmallMaxStages];
  uint64_t tfull[8], tempty[8];
  uint64_t mdrain;
  uint32_t tmem_base, tmem_busy;
};

template <int R, int BM>
__global__ void __launch_bounds__(192) gemm_fp8_small_kernel(const __grid_constant__ CUtensorMap tmW,
                                                             const __grid_constant__ CUtensorMap tmQ,
                                                             const Fp8SmallArgs a) {
  using C = Fp8SmallCfg<R, BM>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Fp8SmallBars S;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int stages = a.stages, KB = a.KB;
  uint8_t* sw = base;                       // weight tiles
  uint8_t* sq = sw + stages * C::kW;        // token tiles
  uint8_t* ss = sq + stages * C::kQ;        // token scales
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * R, m0 = blockIdx.y * BM;

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 5);  // the MMAs' commit and the four epilogue warps (scales)
    }
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(&S.tfull[i], 1);
      mbar_init(&S.tempty[i], 4);
    }
    mbar_init(&S.mdrain, 1);
    S.tmem_busy = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmQ);
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
    if (lane == 0) {
      // scales of this tile's tokens: whole quads, within the row's lds
      const uint32_t sbytes = (uint32_t)min(BM, (a.M - m0 + 3) & ~3) * 4;
      const float* sc = a.scale + m0;
      auto load_w = [&](int b, int s) {
        mbar_arrive_expect_tx(&S.full[s], C::kW + C::kQ + sbytes);
        tma_load_2d(sw + s * C::kW, &tmW, &S.full[s], b * 128, n0);
      };
      auto load_q = [&](int b, int s) {
        tma_load_2d(sq + s * C::kQ, &tmQ, &S.full[s], b * 128, m0);
        bulk_copy_g2s(ss + s * C::kS, sc + (int64_t)b * a.lds, sbytes, &S.full[s]);
      };
      // the first round of the ring: as a programmatic dependent of the
      // quantize kernel, the weights are requested before the wait for its grid
      const int P = min(KB, stages);
      for (int b = 0; b < P; ++b) {
        load_w(b, b);
        if (!a.pdl) load_q(b, b);
      }
      if (a.pdl) {
        griddep_wait();
        for (int b = 0; b < P; ++b) load_q(b, b);
      }
      bool ok = true;
      int s = 0;
      uint32_t phase = 0;
      int last = P;  // loads issued
      for (int b = P; b < KB; ++b) {
        ok = mbar_wait(&S.empty[s], phase, a.err);
        if (!ok) break;
        load_w(b, s);
        load_q(b, s);
        ++last;
        if (++s == stages) { s = 0; phase ^= 1; }
      }
      // every load has landed and (unless a wait gave up) every stage has been
      // released before the CTA exits
      for (int i = max(0, last - stages); i < last; ++i) {
        mbar_wait(&S.full[i % stages], (uint32_t)(i / stages) & 1u, a.err);
        if (ok) mbar_wait(&S.empty[i % stages], (uint32_t)(i / stages) & 1u, a.err);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(R, BM);
      int s = 0, t = 0;
      uint32_t phase = 0, tphase = 1;
      bool ok = true;
      for (int b = 0; b < KB; ++b) {
        ok = mbar_wait(&S.full[s], phase, a.err) && mbar_wait(&S.tempty[t], tphase, a.err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t wa = smem_u32(sw + s * C::kW), qa = smem_u32(sq + s * C::kQ);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_e4m3_ss(tmem + t * BM, smem_desc_sw128(wa + k * 32), smem_desc_sw128(qa + k * 32),
                      idesc, k);
        mma_commit(&S.tfull[t]);
        mma_commit(&S.empty[s]);
        if (++s == stages) { s = 0; phase ^= 1; }
        if (++t == C::kBufs) { t = 0; tphase ^= 1; }
      }
      if (!ok) {
        mma_commit(&S.mdrain);
        if (!mbar_wait(&S.mdrain, 0, a.err)) atomicExch(&S.tmem_busy, 1u);
      }
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3;
    // M = 128: row i in lane i; M = 64: rows 16w.. in the first lanes of quarter w
    const int n = n0 + quarter * (R / 4) + lane;
    const bool nvalid = lane < R / 4 && n < a.N;
    const float* wsp = a.w_scale + (int64_t)(n0 >> 7) * KB;  // a tile lies inside one block of rows
    if (a.pdl) griddep_wait();  // the output may be what an earlier kernel still reads
    float acc[BM];
#pragma unroll
    for (int j = 0; j < BM; ++j) acc[j] = 0.0f;
    int s = 0, t = 0;
    uint32_t phase = 0, tphase = 0;
    bool ok = true;
    float w_next = __ldg(wsp);
    for (int b = 0; b < KB; ++b) {
      const float wsc = w_next;
      if (b + 1 < KB) w_next = __ldg(wsp + b + 1);
      ok = mbar_wait(&S.tfull[t], tphase, a.err) && mbar_wait(&S.full[s], phase, a.err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + t * BM;
      const float* sc = reinterpret_cast<const float*>(ss + s * C::kS);
      const float2 w2 = make_float2(wsc, wsc);
#pragma unroll
      for (int c = 0; c < BM; c += C::kChunk) {
        uint32_t v[C::kChunk];
        if constexpr (C::kChunk == 32) tmem_ld32(taddr + c, v);
        else tmem_ld16(taddr + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < C::kChunk; ++i) asm volatile("" : "+r"(v[i]));
        if (c + C::kChunk == BM) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.tempty[t]);
        }
#pragma unroll
        for (int i = 0; i < C::kChunk; i += 4) {
          const float4 f4 = *reinterpret_cast<const float4*>(sc + c + i);
          const float2 f0 = __fmul2_rn(make_float2(f4.x, f4.y), w2);
          const float2 f1 = __fmul2_rn(make_float2(f4.z, f4.w), w2);
          float* ac = acc + c + i;
          float2 r0 = __ffma2_rn(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), f0,
                                 make_float2(ac[0], ac[1]));
          float2 r1 = __ffma2_rn(make_float2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])), f1,
                                 make_float2(ac[2], ac[3]));
          ac[0] = r0.x; ac[1] = r0.y; ac[2] = r1.x; ac[3] = r1.y;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.empty[s]);  // this warp has read the stage's scales
      if (++s == stages) { s = 0; phase ^= 1; }
      if (++t == C::kBufs) { t = 0; tphase ^= 1; }
    }
    if (ok && nvalid) {
      const int64_t o = (int64_t)m0 * a.ldo + n;
      const int mc = a.M - m0;
#pragma unroll
      for (int j = 0; j < BM; ++j) {
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
static cudaError_t launch_small(const CUtensorMap& tw, const uint8_t* q, int64_t K, Fp8SmallArgs a,
                                bool pdl, cudaStream_t st) {
  using C = Fp8SmallCfg<R, BM>;
  CUtensorMap tq;
  if (!make_tmap_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, K, a.M, K, 128, BM,
                    CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorNotSupported;
  const dim3 grid((unsigned)ceil_div(a.N, R), (unsigned)ceil_div(a.M, BM));
  // one CTA per SM takes the whole shared memory for its ring; two share it
  const int64_t ctas = (int64_t)grid.x * grid.y;
  const int budget = (ctas <= num_sms() ? 224 : 110) * 1024 - 1024;
  int stages = budget / (int)C::kStage;
  stages = stages > kFp8SmallMaxStages ? kFp8SmallMaxStages : stages;
  stages = stages > a.KB ? a.KB : stages;
  a.stages = stages;
  const size_t smem = (size_t)stages * C::kStage + 1024;
  auto kern = gemm_fp8_small_kernel<R, BM>;
  static std::atomic<uint64_t> attr_set{0};
  const cudaError_t e = smem_attr_once_per_device(kern, 224 * 1024, attr_set);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, grid, dim3(192), smem, st, pdl, tw, tq, a);
}

cudaError_t launch_gemm_fp8_small(const uint8_t* q, const float* scale, int64_t lds, int64_t M,
                                  int64_t K, const uint8_t* w, int64_t ldw, const float* w_scale,
                                  int64_t N, void* out, bool out_f32, int64_t ldo, uint32_t* err,
                                  bool pdl, cudaStream_t st) {
  const int bm = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  // 128-row tiles read the tokens half as often; 64-row tiles fill the SMs
  const int r = ceil_div(N, 128) * ceil_div(M, bm) * 4 >= 3 * num_sms() ? 128 : 64;
  CUtensorMap tw;
  if (!make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, K, N, ldw, 128, r,
                    CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorNotSupported;
  Fp8SmallArgs a{scale, w_scale, out, lds, ldo, (int)M, (int)N, (int)ceil_div(K, 128), 0,
                 out_f32, pdl, err};
  if (r == 64) switch (bm) {
    case 16: return launch_small<64, 16>(tw, q, K, a, pdl, st);
    case 32: return launch_small<64, 32>(tw, q, K, a, pdl, st);
    case 64: return launch_small<64, 64>(tw, q, K, a, pdl, st);
    default: return launch_small<64, 128>(tw, q, K, a, pdl, st);
  }
  switch (bm) {
    case 16: return launch_small<128, 16>(tw, q, K, a, pdl, st);
    case 32: return launch_small<128, 32>(tw, q, K, a, pdl, st);
    case 64: return launch_small<128, 64>(tw, q, K, a, pdl, st);
    default: return launch_small<128, 128>(tw, q, K, a, pdl, st);
  }
}

}  // namespace qg
