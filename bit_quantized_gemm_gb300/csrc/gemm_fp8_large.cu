// gemm_fp8_large.cu -- block-scaled e4m3 product for many tokens (prefill).
//
//   out[m][n] = chain over blocks b of 128, ascending:
//               acc = fmaf(sum_{k in b} q[m][k] * w[n][k], s[b][m] * ws[n/128][b], acc)
//
// Bound by the tensor cores: a 128 x 256 x 128 block is 512 tensor cycles of
// an SM. Each block accumulates from zero in its own tensor-memory buffer
// (two buffers of up to 256 columns: all 512), and while the next block's MMAs
// run, the epilogue warps add the finished one to their fp32 accumulators in
// registers. Tokens lie in tensor-memory lanes, so that a thread owns one
// token and a span of columns inside one or two blocks of 128 weight rows: the
// scale s * ws is one number per thread and block, and the chain is one FMA
// per output and block (half the MMA's cycles).
//
// A tile is 128 tokens x W columns for one CTA, or 256 x W for a pair of CTAs
// of one cluster (kPair): each CTA of the pair loads its own 128 tokens and
// half of the W weight rows, and holds the accumulators of its own tokens, so
// that per MMA a pair brings in W/2 instead of W weight rows per SM.
//
// Warps (384 threads, one CTA per SM, persistent): 0 TMA producer, 1 and 2 MMA
// issuers (of a pair's leader CTA; even and odd blocks: an MMA's issue blocks
// while the tensor core is busy, so one issuer's barrier waits have to overlap
// the other's MMAs), 3 idle, 4..11 epilogue: warp w reads lanes 32*(w%4).. and half (w-4)/4 of the columns. Outputs are
// staged per warp in shared memory (32 rows of 128 bytes, swizzled) and leave
// by TMA, or by coalesced element stores where the row length or the pitch is
// not a multiple of 16 bytes.
#include <cuda.h>

#include <cstring>

#include "qg_common.cuh"

namespace qg {

bool make_tmap_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols,
                  int64_t rows, int64_t pitch, uint32_t box_cols, uint32_t box_rows,
                  CUtensorMapSwizzle swizzle);
cudaError_t launch_gemm_fp8_small(const uint8_t* q, const float* scale, int64_t lds, int64_t M,
                                  int64_t K, const uint8_t* w, int64_t ldw, const float* w_scale,
                                  int64_t N, void* out, bool out_f32, int64_t ldo, uint32_t* err,
                                  bool pdl, cudaStream_t st);

struct Fp8LargeArgs {
  const float* scale;    // [KB][lds]
  const float* w_scale;  // [NB][KB]
  void* out;
  int64_t lds, ldo;
  int M, N, KB, NB;
  int tile_group;        // token tiles per group of the persistent tile order
  int tma_out, pdl;
  uint32_t* err;
};

constexpr int kFp8Epi = 8;    // epilogue warps
// The epilogue's 128 accumulators and two 32-column loads do not fit the 168
// registers of an even split: 208 for its warps and 88 for the other four
// (together no more than the 384 * 168 of the launch).
constexpr int kFp8EpiRegs = 208, kFp8RestRegs = 88;
static_assert(32 * (kFp8Epi * kFp8EpiRegs + 4 * kFp8RestRegs) <= (128 + 32 * kFp8Epi) * 168, "registers");
constexpr int kFp8LargeThreads = 128 + 32 * kFp8Epi;

template <bool kPair, int W, bool kF32>
struct Fp8LargeCfg {
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kTileM = 128 * kCtas;
  static constexpr int kWRows = W / kCtas;       // weight rows loaded by a CTA
  static constexpr uint32_t kABytes = 128 * 128, kBBytes = kWRows * 128;
  static constexpr int kCols = W / (kFp8Epi / 4);  // columns per epilogue thread
  static constexpr int kRowBytes = 512 / kFp8Epi;  // staging rows: 64 (or 32) bytes
  static constexpr int kRound = kRowBytes / (kF32 ? 4 : 2);  // columns per staging round
  static constexpr int kStaging = kFp8Epi * 32 * kRowBytes;
  static constexpr int kScales = 2 * 2 * 128 * 4;  // s * ws: two buffers, two blocks of rows, 128 tokens
  static constexpr int kFixed = kStaging + kScales + 1024;
  // an even ring: each of the two issuers owns half of its stages
  static constexpr int kFit = (226 * 1024 - kFixed) / (int)(kABytes + kBBytes) & ~1;
  static constexpr int kStages = kFit > 12 ? 12 : kFit;
  static constexpr size_t kSmem = (size_t)kStages * (kABytes + kBBytes) + kFixed;
  static_assert(W % 64 == 0 && W <= 256 && kCols % kRound == 0 && kStages >= 4, "tile");
};

__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[16]) { tmem_ld16(taddr, v); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[32]) { tmem_ld32(taddr, v); }

template <bool kPair, int W, bool kF32>
__global__ void __launch_bounds__(kFp8LargeThreads, 1)
    gemm_fp8_large_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmW,
                          const __grid_constant__ CUtensorMap tmO, const Fp8LargeArgs a) {
  using C = Fp8LargeCfg<kPair, W, kF32>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[C::kStages], empty[C::kStages], tfull[2], tempty[2], sempty[2], mdrain[2];
  __shared__ uint32_t tmem_slot, tmem_busy;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sa = base;                              // token tiles
  uint8_t* sb = sa + C::kStages * C::kABytes;      // weight tiles
  uint8_t* so = sb + C::kStages * C::kBBytes;      // output staging, kRowBytes x 32 per warp
  float* sf = reinterpret_cast<float*>(so + C::kStaging);  // s * ws [buffer][row block][token]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0;
  const int KB = a.KB;
  const int MT = (a.M + C::kTileM - 1) / C::kTileM, NT = (a.N + W - 1) / W;
  const int tiles = MT * NT;
  const int first = (int)blockIdx.x / C::kCtas, step = (int)gridDim.x / C::kCtas;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 2);                    // the MMAs' commit and the scale warp
      mbar_init(&tempty[i], kFp8Epi * C::kCtas);  // epilogue warps of both CTAs
      mbar_init(&sempty[i], kFp8Epi);
      mbar_init(&mdrain[i], 1);
    }
    tmem_busy = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(&tmem_slot, 512);
    } else {
      tmem_alloc(&tmem_slot, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (kPair) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  auto coords = [&](int tile, int& mt, int& nt) {
    // groups of tile_group token tiles, the token tile fastest: the tiles in
    // flight share weight rows and a bounded set of tokens in L2
    const int per = a.tile_group * NT, g = tile / per;
    const int gm = min(a.tile_group, MT - g * a.tile_group);
    const int idx = tile - g * per;
    mt = g * a.tile_group + idx % gm;
    nt = idx / gm;
  };

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFp8RestRegs));
  if (warp == 0) {
    if (lane == 0) {
      // as a programmatic dependent of the quantize kernel: nothing of the
      // first blocks hides its wait here (the tiles are long)
      if (a.pdl) griddep_wait();
      bool ok = true;
      int s = 0, loads = 0;
      uint32_t phase = 1;
      for (int tile = first; tile < tiles && ok; tile += step) {
        int mt, nt;
        coords(tile, mt, nt);
        const int m = mt * C::kTileM + (int)rank * 128, n = nt * W + (int)rank * C::kWRows;
        for (int b = 0; b < KB; ++b) {
          ok = mbar_wait(&empty[s], phase, a.err);
          if (!ok) break;
          // both CTAs' bytes complete on the leader's barrier
          if (rank == 0) mbar_arrive_expect_tx(&full[s], C::kCtas * (C::kABytes + C::kBBytes));
          if constexpr (kPair) {
            const uint32_t bar = map_to_cta(&full[s], 0);
            tma_load_2d_pair(sa + s * C::kABytes, &tmQ, bar, b * 128, m);
            tma_load_2d_pair(sb + s * C::kBBytes, &tmW, bar, b * 128, n);
          } else {
            tma_load_2d(sa + s * C::kABytes, &tmQ, &full[s], b * 128, m);
            tma_load_2d(sb + s * C::kBBytes, &tmW, &full[s], b * 128, n);
          }
          ++loads;
          if (++s == C::kStages) { s = 0; phase ^= 1; }
        }
      }
      // Every load has landed before the CTA exits: the MMAs that read a stage
      // release it, so the last round's releases cover their loads. After a
      // wait gave up, the leader waits for the loads themselves.
      for (int i = max(0, loads - C::kStages); i < loads; ++i) {
        const int r = i % C::kStages;
        const uint32_t par = (uint32_t)(i / C::kStages) & 1u;
        if (ok) ok = mbar_wait(&empty[r], par, a.err);
        if (!ok && rank == 0) mbar_wait(&full[r], par, a.err);
      }
    }
    __syncwarp();
  } else if (warp <= 2) {
    // issuer `par` takes the blocks g = par, par + 2, ... of this CTA's tiles,
    // into buffer par; the even ring depth gives it the same stages each round
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(C::kTileM, W);
      const int par = warp - 1;
      const int total = first < tiles ? (tiles - first + step - 1) / step * KB : 0;
      int s = par;
      uint32_t phase = 0, tphase = 1;
      bool ok = true;
      for (int g = par; g < total; g += 2) {
        ok = mbar_wait(&full[s], phase, a.err) && mbar_wait(&tempty[par], tphase, a.err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t aa = smem_u32(sa + s * C::kABytes), ba = smem_u32(sb + s * C::kBBytes);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (kPair)
              mma_e4m3_ss_pair(tmem + par * 256, smem_desc_sw128(aa + k * 32),
                               smem_desc_sw128(ba + k * 32), idesc, k);
            else
              mma_e4m3_ss(tmem + par * 256, smem_desc_sw128(aa + k * 32),
                          smem_desc_sw128(ba + k * 32), idesc, k);
          }
          if constexpr (kPair) {
            mma_commit_pair(&tfull[par]);
            mma_commit_pair(&empty[s]);
          } else {
            mma_commit(&tfull[par]);
            mma_commit(&empty[s]);
          }
        }
        __syncwarp();
        s += 2;
        if (s >= C::kStages) { s = par; phase ^= 1; }
        tphase ^= 1;
      }
      if (!ok) {
        // the MMAs issued so far may still run: wait (bounded) before tensor
        // memory is freed; if that gives up too, it stays allocated
        if (elect_one()) {
          if constexpr (kPair) mma_commit_pair(&mdrain[par]);
          else mma_commit(&mdrain[par]);
        }
        __syncwarp();
        if (!mbar_wait(&mdrain[par], 0, a.err)) atomicExch(&tmem_busy, 1u);
      }
    }
  } else if (warp == 3) {
    // scale warp: s * ws of block g for this CTA's 128 tokens and the (at most
    // two) blocks of weight rows of the tile, into buffer g % 2. Four blocks
    // are loaded ahead, across tiles: a load from L2 takes about as long as
    // two blocks of MMAs.
    if (a.pdl) griddep_wait();  // the scales come from the quantize kernel
    const int total = first < tiles ? (tiles - first + step - 1) / step * KB : 0;
    int lt = first, lb = 0;  // the next block to load
    const float *lp = nullptr, *lw0 = nullptr, *lw1 = nullptr;
    bool valid = false;
    float4 s_cur[4], s_nxt[4];
    float2 w_cur[4], w_nxt[4];
    auto load = [&](float4& s4, float2& w2) {
      if (lt >= tiles) return;
      if (lb == 0) {
        int mt, nt;
        coords(lt, mt, nt);
        const int m = mt * C::kTileM + (int)rank * 128 + lane * 4;
        valid = m < a.M;  // whole quads: lds is a multiple of 4
        lp = a.scale + m;
        const int nb = (nt * W) >> 7;
        lw0 = a.w_scale + (int64_t)nb * KB;
        lw1 = a.w_scale + (int64_t)min(nb + 1, a.NB - 1) * KB;
      }
      s4 = valid ? ldg_f32x4_pinned(lp + (int64_t)lb * a.lds) : make_float4(0.f, 0.f, 0.f, 0.f);
      w2.x = ldg_f32_pinned(lw0 + lb);
      w2.y = W > 128 ? ldg_f32_pinned(lw1 + lb) : 0.0f;
      if (++lb == KB) {
        lb = 0;
        lt += step;
      }
    };
#pragma unroll
    for (int j = 0; j < 4; ++j) load(s_nxt[j], w_nxt[j]);
    bool ok = true;
    uint32_t phase = 1;
    for (int g0 = 0; g0 < total && ok; g0 += 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s_cur[j] = s_nxt[j];
        w_cur[j] = w_nxt[j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) load(s_nxt[j], w_nxt[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (g0 + j >= total) break;
        constexpr int kT[4] = {0, 1, 0, 1};
        const int t = kT[j];
        ok = mbar_wait(&sempty[t], phase, a.err);
        if (!ok) break;
        float* f = sf + t * 256 + lane * 4;
        const float4 v = s_cur[j];
        const float2 w = w_cur[j];
        *reinterpret_cast<float4*>(f) = make_float4(v.x * w.x, v.y * w.x, v.z * w.x, v.w * w.x);
        if (W > 128)
          *reinterpret_cast<float4*>(f + 128) =
              make_float4(v.x * w.y, v.y * w.y, v.z * w.y, v.w * w.y);
        __syncwarp();
        if (lane == 0) mbar_arrive(&tfull[t]);
        if (t == 1) phase ^= 1;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFp8EpiRegs));
    const int quarter = warp & 3, part = (warp - 4) >> 2;
    if (a.pdl) griddep_wait();  // the output may be what an earlier kernel still reads
    uint8_t* stage = so + (warp - 4) * 32 * C::kRowBytes;
    uint32_t tempty_addr[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      tempty_addr[i] = kPair ? map_to_cta(&tempty[i], 0) : smem_u32(&tempty[i]);
    int t = 0;
    uint32_t tphase = 0;
    bool ok = true;
    for (int tile = first; tile < tiles && ok; tile += step) {
      int mt, nt;
      coords(tile, mt, nt);
      const int mrow0 = mt * C::kTileM + (int)rank * 128 + quarter * 32;  // this warp's first token
      const int nc0 = nt * W + part * C::kCols;                          // and first column
      // column c of this thread uses the scale of the tile's row block
      // (coff + c) / 128; a span that is a power of two lies in one
      constexpr bool kCross = (C::kCols & (C::kCols - 1)) != 0;
      const int coff = ((nt * W) & 127) + part * C::kCols;
      float acc[C::kCols];
#pragma unroll
      for (int j = 0; j < C::kCols; ++j) acc[j] = 0.0f;
      // kChunk columns per load, the next load in flight during the FMAs, also
      // across blocks: the next block's barrier is looked at a few chunks
      // early, so that its first load can follow this block's last one
      constexpr int kChunk = C::kCols % 64 == 0 ? 32 : 16;
      constexpr int kN = C::kCols / kChunk;
      static_assert(kN % 2 == 0, "a block's first load goes to v[0]");
      uint32_t v[2][kChunk];
      float f0 = 0.0f, f1 = 0.0f;
      uint32_t taddr = 0;
      auto begin = [&]() {  // buffer t is complete: its first load and its scales
        tc_fence_after();
        taddr = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(t * 256 + part * C::kCols);
        tmem_ld(taddr, v[0]);
        const float* fp = sf + t * 256 + quarter * 32 + lane;
        f0 = kCross ? fp[0] : fp[(coff >> 7) * 128];
        f1 = kCross ? fp[128] : 0.0f;
      };
      ok = mbar_wait(&tfull[t], tphase, a.err);
      if (!ok) break;
      begin();
      for (int b = 0; b < KB; ++b) {
        const int tc = t;
        t ^= 1;  // the next block's buffer and phase
        if (t == 0) tphase ^= 1;
        bool ready = false;
#pragma unroll
        for (int c = 0; c < kN; ++c) {
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < kChunk; ++i) asm volatile("" : "+r"(v[c & 1][i]));
          const float g0 = f0, g1 = f1;
          if (c + 1 < kN) {
            tmem_ld(taddr + (c + 1) * kChunk, v[(c + 1) & 1]);
            if (c == (kN > 4 ? kN - 4 : 0)) ready = mbar_test(&tfull[t], tphase);
          } else {
            tc_fence_before();
            ready = __all_sync(0xffffffffu, ready) && b + 1 < KB;
            if (lane == 0) {
              if constexpr (kPair) mbar_arrive_cluster(tempty_addr[tc]);
              else mbar_arrive(&tempty[tc]);
              mbar_arrive(&sempty[tc]);
            }
            __syncwarp();
            if (ready) begin();
          }
#pragma unroll
          for (int i = 0; i < kChunk; i += 2) {
            const float f = kCross && coff + c * kChunk + (i & ~15) >= 128 ? g1 : g0;
            float* ac = acc + c * kChunk + i;
            const float2 r = __ffma2_rn(make_float2(__uint_as_float(v[c & 1][i]),
                                                    __uint_as_float(v[c & 1][i + 1])),
                                        make_float2(f, f), make_float2(ac[0], ac[1]));
            ac[0] = r.x;
            ac[1] = r.y;
          }
        }
        if (!ready && b + 1 < KB) {
          ok = mbar_wait(&tfull[t], tphase, a.err);
          if (!ok) break;
          begin();
        }
      }
      if (!ok) break;
      // outputs: kRound columns of this warp's 32 tokens at a time through its
      // staging rows; a 16-byte chunk lands at chunk ^ (row / 2 % 4), for
      // 32-byte rows chunk ^ (row / 4 % 2), the TMA swizzles
#pragma unroll
      for (int c = 0; c < C::kCols; c += C::kRound) {
        if (a.tma_out) {
          if (lane == 0) bulk_wait_read_all();  // the previous store has read the rows
        }
        __syncwarp();
        const uint32_t sw = C::kRowBytes == 64 ? ((lane >> 1) & 3) : ((lane >> 2) & 1);
#pragma unroll
        for (int i = 0; i < C::kRowBytes / 16; ++i) {
          uint4 o;
          if constexpr (kF32) {
            const float* p = acc + c + 4 * i;
            o = make_uint4(__float_as_uint(p[0]), __float_as_uint(p[1]), __float_as_uint(p[2]),
                           __float_as_uint(p[3]));
          } else {
            const float* p = acc + c + 8 * i;
            uint32_t* w4 = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(p[2 * j], p[2 * j + 1]);
              w4[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
          }
          *reinterpret_cast<uint4*>(stage + lane * C::kRowBytes + ((i ^ sw) * 16)) = o;
        }
        if (a.tma_out) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && mrow0 < a.M && nc0 + c < a.N) {
            tma_store_2d(&tmO, stage, nc0 + c, mrow0);
            bulk_commit_group();
          }
        } else {
          __syncwarp();
          const int rows = min(32, a.M - mrow0);
          for (int r = 0; r < rows; ++r) {
            const uint32_t rsw = C::kRowBytes == 64 ? ((r >> 1) & 3) : ((r >> 2) & 1);
            const int j = lane;
            if (j < C::kRound && nc0 + c + j < a.N) {
              const int n = nc0 + c + j;
              const int byte = j * (kF32 ? 4 : 2);
              const uint8_t* p =
                  stage + r * C::kRowBytes + (((byte >> 4) ^ rsw) << 4) + (byte & 15);
              const int64_t o = (int64_t)(mrow0 + r) * a.ldo + n;
              if constexpr (kF32)
                reinterpret_cast<float*>(a.out)[o] = *reinterpret_cast<const float*>(p);
              else
                reinterpret_cast<uint16_t*>(a.out)[o] = *reinterpret_cast<const uint16_t*>(p);
            }
          }
          __syncwarp();
        }
      }
    }
    if (a.tma_out && lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  // the pair's barriers and tensor memory outlive both CTAs' use of them; the
  // leader's note that MMAs may still run keeps both CTAs' allocations
  bool busy = tmem_busy != 0;
  if constexpr (kPair) {
    cluster_sync();
    if (rank != 0) {
      uint32_t v;
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_cta(&tmem_busy, 0)));
      busy = v != 0;
    }
    cluster_sync();
  }
  if (warp == 1 && !busy) {
    tc_fence_after();
    if constexpr (kPair) tmem_dealloc_pair(tmem, 512);
    else tmem_dealloc(tmem, 512);
  }
}

template <bool kPair, int W, bool kF32>
static cudaError_t launch_large(const uint8_t* q, int64_t K, const uint8_t* w, int64_t ldw,
                                Fp8LargeArgs a, cudaStream_t st) {
  using C = Fp8LargeCfg<kPair, W, kF32>;
  static_assert(C::kSmem <= 226 * 1024, "shared memory per CTA");
  CUtensorMap tq, tw, to;
  if (!make_tmap_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, K, a.M, K, 128, 128,
                    CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, K, a.N, ldw, 128, C::kWRows,
                    CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorNotSupported;
  memset(&to, 0, sizeof(to));
  // the store clips a row at 16-byte granularity: a row whose end is not on
  // such a boundary would overwrite what lies behind it
  a.tma_out = a.N * (kF32 ? 4 : 2) % 16 == 0 &&
              make_tmap_2d(&to, kF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                           a.out, a.N, a.M, a.ldo * (kF32 ? 4 : 2), C::kRound, 32,
                           C::kRowBytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
  a.tile_group = 2048 / C::kTileM;
  auto kern = gemm_fp8_large_kernel<kPair, W, kF32>;
  static std::atomic<uint64_t> attr_set{0};
  cudaError_t e = smem_attr_once_per_device(kern, (int)C::kSmem, attr_set);
  if (e != cudaSuccess) return e;
  // the register split takes from what the block was launched with
  static const int regs = [&] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : 0;
  }();
  if (regs * kFp8LargeThreads < 32 * (kFp8Epi * kFp8EpiRegs + 4 * kFp8RestRegs))
    return cudaErrorInvalidConfiguration;
  const int64_t tiles = ceil_div(a.M, C::kTileM) * ceil_div(a.N, W);
  const int64_t slots = num_sms() / C::kCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((tiles < slots ? tiles : slots) * C::kCtas));
  cfg.blockDim = dim3(kFp8LargeThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C::kCtas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, tq, tw, to, a);
}

template <bool kF32>
static cudaError_t launch_large_any(const uint8_t* q, int64_t K, const uint8_t* w, int64_t ldw,
                                    const Fp8LargeArgs& a, cudaStream_t st) {
  // the tile of the smallest estimated time: waves x cycles per block of K
  struct Choice {
    bool pair;
    int w;
    double step;
  };
  static const Choice kChoices[] = {{true, 256, 512}, {true, 192, 400}, {true, 128, 290},
                                    {false, 128, 400}, {false, 64, 300}};
  const int sms = num_sms();
  int best = 0;
  double best_t = 1e300;
  for (int i = 0; i < 5; ++i) {
    const Choice& c = kChoices[i];
    const int ctas = c.pair ? 2 : 1;
    const int64_t tiles = ceil_div(a.M, 128 * ctas) * ceil_div(a.N, c.w);
    const double t = (double)ceil_div(tiles, sms / ctas) * c.step;
    if (t < best_t) { best_t = t; best = i; }
  }
  switch (best) {
    case 0: return launch_large<true, 256, kF32>(q, K, w, ldw, a, st);
    case 1: return launch_large<true, 192, kF32>(q, K, w, ldw, a, st);
    case 2: return launch_large<true, 128, kF32>(q, K, w, ldw, a, st);
    case 3: return launch_large<false, 128, kF32>(q, K, w, ldw, a, st);
    default: return launch_large<false, 64, kF32>(q, K, w, ldw, a, st);
  }
}

cudaError_t launch_gemm_fp8(const uint8_t* q, const float* scale, int64_t lds, int64_t M, int64_t K,
                            const uint8_t* w, int64_t ldw, const float* w_scale, int64_t N,
                            void* out, bool out_f32, int64_t ldo, uint32_t* err, bool pdl,
                            cudaStream_t st) {
  if (M <= 128)
    return launch_gemm_fp8_small(q, scale, lds, M, K, w, ldw, w_scale, N, out, out_f32, ldo, err,
                                 pdl, st);
  Fp8LargeArgs a{scale, w_scale, out, lds, ldo, (int)M, (int)N, (int)ceil_div(K, 128),
                 (int)ceil_div(N, 128), 0, 0, pdl, err};
  return out_f32 ? launch_large_any<true>(q, K, w, ldw, a, st)
                 : launch_large_any<false>(q, K, w, ldw, a, st);
}

}  // namespace qg
