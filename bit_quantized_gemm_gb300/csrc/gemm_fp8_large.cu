// gemm_fp8_large.cu -- block-scaled e4m3 product for many tokens (prefill).
//
//   out[m][n] = chain over blocks b of 128, ascending:
//               acc = fmaf(sum_{k in b} q[m][k] * w[n][k], s[b][m] * ws[n/128][b], acc)
//
// Bound by the tensor cores (a 128 x 256 x 128 block is 512 tensor cycles of an
// SM) and, before they saturate, by the epilogue: each block accumulates from
// zero in its own tensor-memory buffer (two of 256 columns, four of 128 or 64),
// and while the next block's MMAs run, the epilogue warps add the finished one
// to their fp32 accumulators in registers. Tokens lie in tensor-memory lanes, so
// that a thread owns one token and a span of columns inside one block of 128
// weight rows: s * ws is one number per thread and block, the chain one FMA per
// output and block (256 cycles of the FMA pipe for a block of 512 MMA cycles).
// Measured at 8192 x 5120 x 17408: 550-556 us from a graph, 2.6 PFLOP/s. In loops of
// two seconds, with the SM clock sampled (median): 588 us at 1916 MHz, the power
// limit, 971 cycles a block; without the epilogue's FMAs 551 us at 1980, 940 cycles;
// without its loads too 547, 940; without the operand loads too 504 at 2070, 899. So
// what bounds it is neither the epilogue's work nor the clock: with nothing left but
// MMAs (512 cycles) and barriers a block still takes 900. What is left is the way of
// a buffer from the commit over the epilogue and the scale warp back to its issuer.
//
// A tile is 128 tokens x W columns for one CTA, or 256 x W for a pair of CTAs
// of one cluster (kPair): each CTA of the pair loads its own 128 tokens and
// half of the W weight rows, and holds the accumulators of its own tokens, so
// that per MMA a pair brings in W/2 instead of W weight rows per SM.
//
// Warps (384 threads, one CTA per SM, persistent): 0 TMA producer; 1 and 2 MMA
// issuers (of a pair's leader CTA; even and odd blocks: an MMA's issue blocks
// while the tensor core is busy, so one issuer's barrier waits have to overlap
// the other's MMAs; one issuer 692 us); 3 scales; 4..11 epilogue: warp w reads
// lanes 32*(w%4).. and half (w-4)/4 of the columns. Sixteen epilogue warps were
// no faster (570 us), nor were half blocks of 128 columns in four buffers (599; both
// when this form took 545 to 560).
// Outputs are staged per warp in shared memory (32 rows of 64 bytes, swizzled)
// and leave by TMA, or by coalesced element stores where the row length or the
// pitch is not a multiple of 16 bytes.
//
// Grouped by expert (kGrouped), the tiles are those of each expert's rows, listed by
// every CTA for itself, the weights a third dimension of their tensor map. An
// expert's last rows leave in 16-byte stores (straight from the registers, all of
// them: 161 us where it was 147). 16384 rows of 64 experts, 2560 -> 2432: 138 us. A
// fifth of the tiles' rows lies behind an expert's last; of 6.6 us a tile of 128 x 128
// the blocks take 5.0 (250 ns each: L2 delivers 13 TB/s then), the stores 1.3.
#include <cuda.h>

#include <cstring>
#include <type_traits>

#include "gemm_grouped.cuh"

namespace qg {

bool make_tmap_3d(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols,
                  int64_t rows, int64_t mats, int64_t pitch, int64_t mat_pitch, uint32_t box_cols,
                  uint32_t box_rows, CUtensorMapSwizzle swizzle);
bool make_tmap_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols,
                  int64_t rows, int64_t pitch, uint32_t box_cols, uint32_t box_rows,
                  CUtensorMapSwizzle swizzle);
cudaError_t launch_gemm_fp8_small(const uint8_t* q, const float* scale, int64_t lds, int64_t M,
                                  int64_t K, const uint8_t* w, int64_t ldw, const float* w_scale,
                                  int64_t N, void* out, bool out_f32, int64_t ldo, uint32_t* err,
                                  bool pdl, cudaStream_t st);
void fp8_small_tile(int64_t M, int64_t N, int sms, int* tokens, int* rows);

// up to 64 tokens stream the weights (64 x 5120 x 17408: 18.4 us, 19.0 here; 64 x
// 17408 x 5120: 26.1 us, 35.5 here; 40 x 4096 x 131072: 84.0, 88.8)
constexpr int64_t kFp8SmallM = 64;

struct Fp8LargeArgs {
  const float* scale;    // [KB][lds]
  const float* w_scale;  // [NB][KB]
  void* out;
  int64_t lds, ldo;
  int M, N, KB, NB;
  int tile_group;        // token tiles per group of the persistent tile order
  int tma_out, pdl;
  uint32_t* err;
  // grouped by expert
  const int64_t* offsets;  // [E + 1]
  int E;
};

// Geometry of a tile
template <bool kPair, int W, bool kF32, bool kGrouped>
struct Fp8LargeCfg {
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kTileM = 128 * kCtas;
  static constexpr int kWRows = W / kCtas;  // weight rows loaded by a CTA
  static constexpr uint32_t kABytes = 128 * 128, kBBytes = kWRows * 128;
  // block accumulators in tensor memory: each of the two issuers owns kSlots
  // (not more than two: the unrolled loops outgrow the instruction cache)
  static constexpr int kSlots = W == 256 ? 1 : 2;
  static constexpr int kEpi = 8;        // epilogue warps; a thread owns one token and kCols columns
  static constexpr int kThreads = 128 + 32 * kEpi;
  static constexpr int kCols = W / 2;
  // 128 accumulators and two 32-column loads take more than an even share of
  // the registers: 208, which the other four warps make up for
  static constexpr int kLaunchRegs = 168;
  static constexpr int kEpiRegs = W == 256 ? 208 : 168, kRestRegs = W == 256 ? 88 : 168;
  static_assert(32 * (kEpi * kEpiRegs + 4 * kRestRegs) <= kThreads * kLaunchRegs, "registers");
  // output staging of a warp: 32 rows of 64 bytes, kRound columns
  static constexpr int kEsize = kF32 ? 4 : 2;
  static constexpr int kRowBytes = 64;
  static constexpr int kRound = kRowBytes / kEsize;
  static constexpr int kWarpStaging = 32 * kRowBytes;
  // ring stages of G blocks of K share their barriers; a stage also brings the
  // token scales of its blocks
  static constexpr int G = 2;
  // a row of scales has to start on a multiple of four tokens: where an expert's
  // first row decides, four more are loaded
  static constexpr int kScaleRow = kGrouped ? 132 : 128, kScaleLoad = G * kScaleRow * 4;
  static constexpr int kScaleBytes = (kScaleLoad + 127) / 128 * 128;
  static constexpr uint32_t kStage = G * (kABytes + kBBytes);
  // s * ws of a block: [buffer][row block of the tile][token]
  static constexpr int kScaleRows = W > 128 ? 2 : 1;
  static constexpr int kProducts = 2 * kSlots * kScaleRows * 512;
  static constexpr int kFixed = kEpi * kWarpStaging + kProducts + 1024;
  static constexpr int kFit = (226 * 1024 - kFixed) / ((int)kStage + kScaleBytes);
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static constexpr size_t kSmem = (size_t)kStages * (kStage + kScaleBytes) + kFixed;
  static_assert(W % 64 == 0 && W <= 256 && kCols % kRound == 0 && kStages >= (kGrouped ? 2 : 3), "tile");
};

template <bool kPair, int W, bool kF32, bool kGrouped>
__global__ void __launch_bounds__(Fp8LargeCfg<kPair, W, kF32, kGrouped>::kThreads, 1)
    gemm_fp8_large_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmW,
                          const __grid_constant__ CUtensorMap tmS,
                          const __grid_constant__ CUtensorMap tmO, const Fp8LargeArgs a) {
  using C = Fp8LargeCfg<kPair, W, kF32, kGrouped>;
  constexpr int kSlots = C::kSlots, G = C::G;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[C::kStages], empty[C::kStages], sfull[C::kStages];
  __shared__ uint64_t tfull[2 * kSlots], tempty[2 * kSlots];  // [issuer][slot]
  __shared__ uint64_t sempty[2 * kSlots], mdrain[2];
  __shared__ uint32_t tmem_slot, tmem_busy;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sa = base;                                // token tiles [stage][G]
  uint8_t* sb = sa + C::kStages * G * C::kABytes;    // weight tiles [stage][G]
  uint8_t* so = sb + C::kStages * G * C::kBBytes;    // output staging [warp]
  uint8_t* ss = so + C::kEpi * C::kWarpStaging;      // token scales [stage][G][128]
  float* sf = reinterpret_cast<float*>(ss + C::kStages * C::kScaleBytes);  // s * ws [buffer][row block][token]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0;
  const int KB = a.KB, NS = (KB + G - 1) / G;
  const int MT = (a.M + C::kTileM - 1) / C::kTileM, NT = (a.N + W - 1) / W;
  int tiles = MT * NT;
  int* const lists = reinterpret_cast<int*>(sf + C::kProducts / 4);  // grouped: the experts' rows and tiles
  const GroupedTiles T{lists, lists + a.E + 1, a.E, NT};
  const int first = (int)blockIdx.x / C::kCtas, step = (int)gridDim.x / C::kCtas;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&sfull[i], 1);
      mbar_init(&empty[i], 3);  // a commit of each issuer, and the scale warp
    }
    for (int i = 0; i < 2 * kSlots; ++i) {
      mbar_init(&tfull[i], 2);  // the MMAs' commit and the scale warp
      mbar_init(&tempty[i], C::kEpi * C::kCtas);  // epilogue warps of both CTAs
      mbar_init(&sempty[i], C::kEpi);
    }
    mbar_init(&mdrain[0], 1);
    mbar_init(&mdrain[1], 1);
    tmem_busy = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmS);
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(&tmem_slot, 512);
    } else {
      tmem_alloc(&tmem_slot, 512);
      tmem_relinquish();
    }
  }
  if constexpr (kGrouped) {
    if (warp == 2) GroupedTiles::fill(a.offsets, a.E, a.M, C::kTileM, lists, lists + a.E + 1);
  }
  tc_fence_before();
  if constexpr (kPair) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if constexpr (kGrouped) tiles = T.total();

  // a tile's expert (grouped), its first token and the token after its last, its
  // number among the tiles of weight rows
  struct Place {
    int e, m, end, nt;
  };
  auto place = [&](int tile) {
    Place p;
    if constexpr (kGrouped) {
      int mi;
      T.at(tile, p.e, mi, p.nt);
      p.m = T.first[p.e] + mi * C::kTileM;
      p.end = T.first[p.e + 1];
      return p;
    }
    // groups of tile_group token tiles, the token tile fastest: the tiles in
    // flight share weight rows and a bounded set of tokens in L2
    const int per = a.tile_group * NT, g = tile / per;
    const int gm = min(a.tile_group, MT - g * a.tile_group);
    const int idx = tile - g * per;
    p.e = 0;
    p.m = (g * a.tile_group + idx % gm) * C::kTileM;
    p.end = a.M;
    p.nt = idx / gm;
    return p;
  };

  if (C::kEpiRegs != C::kRestRegs && warp < 4)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRestRegs));
  if (warp == 0) {
    // as a programmatic dependent of the quantize kernel: nothing of the
    // first blocks hides its wait here (the tiles are long)
    if (a.pdl) griddep_wait();
    bool ok = true;
    int s = 0, loads = 0;
    uint32_t phase = 1;
    for (int tile = first; tile < tiles && ok; tile += step) {
      const Place p = place(tile);
      const int m = p.m + (int)rank * 128, n = p.nt * W + (int)rank * C::kWRows;
      for (int i = 0; i < NS; ++i) {
        ok = mbar_wait_warp(&empty[s], phase, a.err);
        if (!ok) break;
        if (elect_one()) {
          // the scale warp reads the slot's scales through the generic proxy
          // (ld.shared); the load below rewrites them through the async proxy,
          // ordered after those reads only by this fence
          fence_proxy_async_smem();
          const int blocks = min(G, KB - G * i);
          // both CTAs' bytes complete on the leader's barrier
          if (rank == 0)
            mbar_arrive_expect_tx(&full[s], blocks * C::kCtas * (C::kABytes + C::kBBytes));
          mbar_arrive_expect_tx(&sfull[s], C::kScaleLoad);
          tma_load_2d(ss + s * C::kScaleBytes, &tmS, &sfull[s], kGrouped ? m & ~3 : m, G * i);
          const uint32_t bar = kPair ? map_to_cta(&full[s], 0) : 0;
          for (int j = 0; j < blocks; ++j) {
            const int k = (G * i + j) * 128;
            if constexpr (kPair) {
              tma_load_2d_pair(sa + (G * s + j) * C::kABytes, &tmQ, bar, k, m);
              if constexpr (kGrouped)
                tma_load_3d_pair(sb + (G * s + j) * C::kBBytes, &tmW, bar, k, n, p.e);
              else
                tma_load_2d_pair(sb + (G * s + j) * C::kBBytes, &tmW, bar, k, n);
            } else {
              tma_load_2d(sa + (G * s + j) * C::kABytes, &tmQ, &full[s], k, m);
              if constexpr (kGrouped)
                tma_load_3d(sb + (G * s + j) * C::kBBytes, &tmW, &full[s], k, n, p.e);
              else
                tma_load_2d(sb + (G * s + j) * C::kBBytes, &tmW, &full[s], k, n);
            }
          }
        }
        __syncwarp();
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
      if (ok) ok = mbar_wait_warp(&empty[r], par, a.err);
      if (!ok && rank == 0) mbar_wait_warp(&full[r], par, a.err);
      if (!ok) mbar_wait_warp(&sfull[r], par, a.err);
    }
  } else if (warp <= 2) {
    // Block b of every tile goes to buffer b / 2 % kSlots of issuer b % 2: each
    // buffer belongs to one issuer.
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(C::kTileM, W);
      const int me = warp - 1;
      const int tiles_here = first < tiles ? (tiles - first + step - 1) / step : 0;
      const uint32_t dbase = tmem + me * kSlots * W;
      int s = 0;
      uint32_t phase = 0, used = ~0u;  // used: bit per buffer, phase of the next wait
      bool ok = true;
      for (int tile = 0; tile < tiles_here && ok; ++tile) {
#pragma unroll kSlots
        for (int i = 0; i < NS; ++i) {
          const int t = i & (kSlots - 1);
          if (2 * i + me < KB) {  // block `me` of the stage
            ok = mbar_wait_warp2(&tempty[me * kSlots + t], (used >> t) & 1u, &full[s], phase, a.err);
            if (!ok) break;
            tc_fence_after();
            const uint32_t aa = smem_u32(sa + (G * s + me) * C::kABytes);
            const uint32_t ba = smem_u32(sb + (G * s + me) * C::kBBytes);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if constexpr (kPair)
                  mma_e4m3_ss_pair(dbase + t * W, smem_desc_sw128(aa + k * 32),
                                   smem_desc_sw128(ba + k * 32), idesc, k);
                else
                  mma_e4m3_ss(dbase + t * W, smem_desc_sw128(aa + k * 32),
                              smem_desc_sw128(ba + k * 32), idesc, k);
              }
              if constexpr (kPair) {
                mma_commit_pair(&tfull[me * kSlots + t]);
                mma_commit_pair(&empty[s]);
              } else {
                mma_commit(&tfull[me * kSlots + t]);
                mma_commit(&empty[s]);
              }
            }
            __syncwarp();
            used ^= 1u << t;
          } else {
            // no block of its own in an odd tail: the stage's other user is
            // waited for all the same, then released
            ok = mbar_wait_warp(&full[s], phase, a.err);
            if (!ok) break;
            if (elect_one()) {
              if constexpr (kPair) mma_commit_pair(&empty[s]);
              else mma_commit(&empty[s]);
            }
            __syncwarp();
          }
          if (++s == C::kStages) { s = 0; phase ^= 1; }
        }
      }
      if (!ok) {
        // the MMAs issued so far may still run: wait (bounded) before tensor
        // memory is freed; if that gives up too, it stays allocated
        if (elect_one()) {
          if constexpr (kPair) mma_commit_pair(&mdrain[me]);
          else mma_commit(&mdrain[me]);
        }
        __syncwarp();
        if (!mbar_wait_warp(&mdrain[me], 0, a.err)) atomicExch(&tmem_busy, 1u);
      }
    }
  } else if (warp == 3) {
    // scale warp: s * ws of each block for this CTA's 128 tokens and the (at
    // most two) blocks of weight rows of the tile, so that the epilogue, whose
    // loop bounds the kernel, reads one number per block. Of the weight scales
    // a lane holds one of 32 blocks, and the next 32 are on their way. The
    // products are formed before the wait for their buffer; with two buffers an
    // issuer, both blocks of a stage go through one round of waits (single waits,
    // products after them: 4096 x 5120 x 4864 in pair tiles of 128 columns 95 us,
    // 83 here).
    constexpr int U = kSlots == 1 ? 1 : G;
    const int tiles_here = first < tiles ? (tiles - first + step - 1) / step : 0;
    bool ok = true;
    int s = 0;
    uint32_t phase = 0, used = ~0u;  // used: bit per buffer, phase of the next wait
    float w_first[C::kScaleRows];    // the weight scales of a tile's first 32 blocks
    auto w_row = [&](const Place& p, int r) {
      return a.w_scale + (kGrouped ? (int64_t)p.e * a.NB * KB : 0) + (int64_t)min((p.nt * W >> 7) + r, a.NB - 1) * KB;
    };
    // (Grouped, the search for a tile's place is made a tile ahead. Dense, it is formed anew:
    // kept over the loop it shows there; with the rolled stores below 128 x 17408 x 5120 takes
    // 35.2 us in place of 36.5, 4096 x 2560 x 5120 fp32 61.3 in place of 64.4.)
    Place here{}, after{};
    if (tiles_here) after = place(first);
#pragma unroll
    for (int r = 0; r < C::kScaleRows; ++r)
      w_first[r] = tiles_here && lane < KB ? ldg_f32_pinned(w_row(after, r) + lane) : 0.0f;
    for (int ti = 0; ti < tiles_here && ok; ++ti) {
      here = kGrouped ? after : place(first + ti * step);
      if (ti + 1 < tiles_here) after = place(first + (ti + 1) * step);
      const int odd = kGrouped ? here.m & 3 : 0;  // (of either CTA: its tokens are 128 apart)
      const float* wp[C::kScaleRows];
      float w_cur[C::kScaleRows], w_nxt[C::kScaleRows];
#pragma unroll
      for (int r = 0; r < C::kScaleRows; ++r) {
        wp[r] = w_row(here, r);
        w_cur[r] = w_first[r];
        w_nxt[r] = 32 + lane < KB ? ldg_f32_pinned(wp[r] + 32 + lane) : 0.0f;
        if (ti + 1 < tiles_here)
          w_first[r] = lane < KB ? ldg_f32_pinned(w_row(after, r) + lane) : 0.0f;
      }
#pragma unroll (2 * kSlots / U)
      for (int b = 0; b < KB; b += U) {
        const int own = U == 1 ? b & 1 : 0, t = b >> 1 & (kSlots - 1);
        const int buf = own * kSlots + t, buf1 = buf + kSlots;
        const bool two = U == 2 && b + 1 < KB, last_of_stage = U == 2 || own || b + 1 == KB;
        if (!own) ok = mbar_wait_warp(&sfull[s], phase, a.err);
        if (!ok) break;
        float4 p[U][C::kScaleRows];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float* ps =
              reinterpret_cast<const float*>(ss + s * C::kScaleBytes + (own + u) * C::kScaleRow * 4) + lane * 4;
          float4 v;
          if constexpr (kGrouped)
            v = make_float4(ps[odd], ps[odd + 1], ps[odd + 2], ps[odd + 3]);
          else
            v = *reinterpret_cast<const float4*>(ps);
#pragma unroll
          for (int r = 0; r < C::kScaleRows; ++r) {
            const float w = __shfl_sync(0xffffffffu, w_cur[r], (b + u) & 31);
            p[u][r] = make_float4(v.x * w, v.y * w, v.z * w, v.w * w);
            // (done before the wait below)
            asm volatile("" : "+f"(p[u][r].x), "+f"(p[u][r].y), "+f"(p[u][r].z), "+f"(p[u][r].w));
          }
        }
        const int mine = two && (lane & 1) ? buf1 : buf;
        ok = mbar_wait_warp(&sempty[mine], (used >> mine) & 1u, a.err);
        if (!ok) break;
        __syncwarp();  // each lane has seen one of the two buffers released
        float* f = sf + lane * 4;
#pragma unroll
        for (int r = 0; r < C::kScaleRows; ++r) {
          *reinterpret_cast<float4*>(f + (buf * C::kScaleRows + r) * 128) = p[0][r];
          if (two) *reinterpret_cast<float4*>(f + (buf1 * C::kScaleRows + r) * 128) = p[U - 1][r];
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&tfull[buf]);
          if (two) mbar_arrive(&tfull[buf1]);
          if (last_of_stage) mbar_arrive(&empty[s]);  // its scales are read
        }
        if (last_of_stage && ++s == C::kStages) { s = 0; phase ^= 1; }
        used ^= 1u << buf;
        if (two) used ^= 1u << buf1;
        if (((b + U) & 31) == 0) {
#pragma unroll
          for (int r = 0; r < C::kScaleRows; ++r) {
            w_cur[r] = w_nxt[r];
            w_nxt[r] = b + U + 32 + lane < KB ? ldg_f32_pinned(wp[r] + b + U + 32 + lane) : 0.0f;
          }
        }
      }
    }
  } else {
    if (C::kEpiRegs != C::kRestRegs)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kEpiRegs));
    const int quarter = warp & 3, part = (warp - 4) >> 2;
    if (a.pdl) griddep_wait();  // the output may be what an earlier kernel still reads
    uint8_t* stage = so + (warp - 4) * C::kWarpStaging;
    const uint32_t tempty_leader = kPair ? map_to_cta(tempty, 0) : 0;
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(part * C::kCols);
    // its columns lie in one block of weight rows: spans of 32, 64 or 128
    const float* fp = sf + (C::kScaleRows == 2 ? part * 128 : 0) + quarter * 32 + lane;
    uint32_t used = 0;  // bit per buffer: phase of its next wait
    bool ok = true;
    for (int tile = first; tile < tiles && ok; tile += step) {
      const Place p = place(tile);
      const int mrow0 = p.m + (int)rank * 128 + quarter * 32;  // this warp's first token
      const int nc0 = p.nt * W + part * C::kCols;              // and first column
      // (a store of 32 rows stops at the last of all rows, not at the expert's)
      const bool tma_out = a.tma_out && (!kGrouped || mrow0 + 32 <= p.end);
      float acc[C::kCols];
#pragma unroll
      for (int j = 0; j < C::kCols; ++j) acc[j] = 0.0f;
      // kChunk columns per load, the next load in flight during the FMAs, also
      // across blocks: the next block's barrier is looked at early, so that its
      // first load can follow this block's last
      constexpr int kChunk = C::kCols == 32 ? 16 : 32;
      constexpr int kN = C::kCols / kChunk;
      static_assert(kN % 2 == 0, "a block's first load goes to v[0]");
      uint32_t v[2][kChunk];
      float f = 0.0f;
      int buf = 0;
      uint32_t par = 0;
      auto locate = [&](int b) {  // block b's buffer and phase
        buf = (b & 1) * kSlots + (b >> 1 & (kSlots - 1));
        par = (used >> buf) & 1u;
        used ^= 1u << buf;
      };
      auto begin = [&]() {  // the buffer is complete: its first load and its scales
        tc_fence_after();
        tmem_ld(lane_base + (uint32_t)(buf * W), v[0]);
        f = fp[buf * (C::kScaleRows * 128)];
      };
      locate(0);
      ok = mbar_wait_warp(&tfull[buf], par, a.err);
      if (!ok) break;
      begin();
      // (one round of the buffers a trip: their numbers are constants. This loop
      // bounds the kernel, and a few integer operations per block show: 579 us
      // rolled, 548 unrolled at 8192 x 5120 x 17408)
#pragma unroll (2 * kSlots)
      for (int b = 0; b < KB; ++b) {
        const int here = buf;
        const bool more = b + 1 < KB;
        if (more) locate(b + 1);
        bool ready = false;
#pragma unroll
        for (int c = 0; c < kN; ++c) {
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < kChunk; ++i) asm volatile("" : "+r"(v[c & 1][i]));
          const float2 f2 = make_float2(f, f);
          if (c + 1 < kN) {
            tmem_ld(lane_base + (uint32_t)(here * W + (c + 1) * kChunk), v[(c + 1) & 1]);
            if (c == (kN > 4 ? kN - 4 : 0) && more) ready = mbar_test(&tfull[buf], par);
          } else {
            tc_fence_before();
            ready = __all_sync(0xffffffffu, ready);
            __syncwarp();  // (a vote orders no memory: the lanes' reads of f)
            if (lane == 0) {
              if constexpr (kPair) mbar_arrive_cluster(tempty_leader + here * 8);
              else mbar_arrive(&tempty[here]);
              mbar_arrive(&sempty[here]);
            }
            __syncwarp();
            if (ready) begin();
          }
#pragma unroll
          for (int i = 0; i < kChunk; i += 2) {
            float* ac = acc + c * kChunk + i;
            const float2 r = __ffma2_rn(make_float2(__uint_as_float(v[c & 1][i]),
                                                    __uint_as_float(v[c & 1][i + 1])),
                                        f2, make_float2(ac[0], ac[1]));
            ac[0] = r.x;
            ac[1] = r.y;
          }
        }
        if (!ready && more) {
          ok = mbar_wait_warp(&tfull[buf], par, a.err);
          if (!ok) break;
          begin();
        }
      }
      if (!ok) break;
      // outputs: kRound columns x this warp's 32 tokens at a time through its
      // staging rows; a 16-byte chunk lands at chunk ^ (row / 2 % 4), the TMA
      // swizzle
      const uint32_t sw = (lane >> 1) & 3;
#pragma unroll
      for (int c0 = 0; c0 < C::kCols; c0 += C::kRound) {
        if (a.tma_out) {
          if (lane == 0) bulk_wait_read_all();  // the previous store has read the rows
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 o;
          if constexpr (kF32) {
            const float* f = acc + c0 + 4 * i;
            o = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                           __float_as_uint(f[3]));
          } else {
            const float* f = acc + c0 + 8 * i;
            uint32_t* w4 = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
              w4[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
          }
          *reinterpret_cast<uint4*>(stage + lane * C::kRowBytes + ((i ^ sw) * 16)) = o;
        }
        if (tma_out) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && mrow0 < a.M && nc0 + c0 < a.N) {
            tma_store_2d(&tmO, stage, nc0 + c0, mrow0);
            bulk_commit_group();
          }
        } else if (kGrouped && a.tma_out) {
          // an expert's last rows: 16 bytes a lane, eight rows at a time
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + (lane >> 2), col = (lane & 3) * (16 / C::kEsize);
            if (mrow0 + r >= p.end || nc0 + c0 + col >= a.N) continue;
            const uint4 o = *reinterpret_cast<const uint4*>(stage + r * C::kRowBytes + (((lane & 3) ^ ((r >> 1) & 3)) << 4));
            *reinterpret_cast<uint4*>(reinterpret_cast<char*>(a.out) +
                                      ((int64_t)(mrow0 + r) * a.ldo + nc0 + c0 + col) * C::kEsize) = o;
          }
          __syncwarp();
        } else {
          __syncwarp();
          // 32 columns of a row at a time, or 16 of two rows, eight reads ahead of
          // their stores (1777 rows of 7 experts, 1216 -> 2563, fp32: 23.3 us; a
          // read and its store after one another 28.3). A loop where the
          // accumulators fill the registers: unrolled, 16384 rows of 64 experts 169
          // us in place of 138. A loop in the dense kernels, too (see the scale warp).
          using Element = std::conditional_t<kF32, uint32_t, uint16_t>;
          constexpr int kRows = 32 / C::kRound;
          const int row = lane / C::kRound, rows = min(32, p.end - mrow0) - row;
          const int col = lane % C::kRound, byte = col * C::kEsize;
          Element* to = reinterpret_cast<Element*>(a.out) + (int64_t)(mrow0 + row) * a.ldo + nc0 + c0 + col;
          const bool in = nc0 + c0 + col < a.N;
#pragma unroll (W == 256 || !kGrouped ? 1 : 4)
          for (int i0 = 0; i0 < C::kRound; i0 += 8) {
            Element o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = (i0 + i) * kRows + row;
              o[i] = *reinterpret_cast<const Element*>(stage + r * C::kRowBytes +
                                                       (((byte >> 4) ^ (i * kRows >> 1 & 3)) << 4) + (byte & 15));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i, to += kRows * a.ldo)
              if (in && (i0 + i) * kRows < rows) *to = o[i];
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

// (experts' weights lie lde bytes apart where the product is grouped)
template <bool kPair, int W, bool kF32, bool kGrouped>
static cudaError_t launch_large(const uint8_t* q, int64_t K, const uint8_t* w, int64_t ldw, int64_t lde,
                                Fp8LargeArgs a, cudaStream_t st) {
  using C = Fp8LargeCfg<kPair, W, kF32, kGrouped>;
  static_assert(C::kSmem + (kGrouped ? GroupedTiles::bytes(1024) : 0) <= 226 * 1024, "shared memory per CTA");
  CUtensorMap tq, tw, ts, to;
  if (!make_tmap_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, K, a.M, K, 128, 128,
                    CU_TENSOR_MAP_SWIZZLE_128B) ||
      !(kGrouped ? make_tmap_3d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, K, a.N, a.E, ldw, lde, 128, C::kWRows,
                                CU_TENSOR_MAP_SWIZZLE_128B)
                 : make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, K, a.N, ldw, 128, C::kWRows,
                                CU_TENSOR_MAP_SWIZZLE_128B)) ||
      !make_tmap_2d(&ts, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.scale, a.M, a.KB, a.lds * 4, C::kScaleRow,
                    C::G, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorNotSupported;
  memset(&to, 0, sizeof(to));
  // the store clips a row at 16-byte granularity: a row whose end is not on
  // such a boundary would overwrite what lies behind it
  a.tma_out = a.N * (kF32 ? 4 : 2) % 16 == 0 &&
              make_tmap_2d(&to, kF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                           a.out, a.N, a.M, a.ldo * (kF32 ? 4 : 2), C::kRound, 32,
                           CU_TENSOR_MAP_SWIZZLE_64B);
  a.tile_group = 2048 / C::kTileM;
  // (grouped: the list of tiles behind everything else)
  const size_t smem = C::kSmem + (kGrouped ? GroupedTiles::bytes(a.E) : 0);
  auto kern = gemm_fp8_large_kernel<kPair, W, kF32, kGrouped>;
  static std::atomic<uint64_t> attr_set{0};
  cudaError_t e = smem_attr_once_per_device(kern, (int)C::kSmem + (kGrouped ? GroupedTiles::bytes(1024) : 0), attr_set);
  if (e != cudaSuccess) return e;
  // the register split takes from what the block was launched with
  static const int regs = [&] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : 0;
  }();
  if (C::kEpiRegs != C::kRestRegs && regs < C::kLaunchRegs)
    return cudaErrorInvalidConfiguration;
  // (grouped: at most; the device knows the number)
  const int64_t tiles = (kGrouped ? a.M / C::kTileM + (a.M < a.E ? a.M : a.E) : ceil_div(a.M, C::kTileM)) *
                        ceil_div(a.N, W);
  const int64_t slots = num_sms() / C::kCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((tiles < slots ? tiles : slots) * C::kCtas));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C::kCtas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, tq, tw, ts, to, a);
}

// The tiles, and their ns per block of K (measured with forced choices at
// 8192 x 5120 x 17408). Of fourteen other sizes the choice is the fastest or within
// 1 % at eleven; a tile's stores and first loads, which are not in it, show at the
// rest: 1024 x 512 x 2560 8.8 us (128 x 128: 7.7), 128 x 17408 x 5120 36.2 (256 x 128:
// 34.1), 2048 x 512 x 9728 20.1 (19.8). In us, 256 x 256 / 256 x 128 / 128 x 128 / 128
// x 64: 777 x 2576 x 5003 fp32 (its rows element by element after one another then;
// 23.6 now) 37.1 / 29.8 / 24.5 / 30.5; 2048 x 2560 x 9728 47.7 / 48.1
// / 52.1 / 82.2; 4096 x 2560 x 5120 fp32 63.8 / 61.0 / 65.7 / 91.9; 256 x 17408 x 5120
// 62.2 / 34.4 / 42.4 / 69.3.
struct Fp8LargeChoice {
  bool pair;
  int w;
  double step;
};
// Grouped by expert there is a fifth, 128 x 256: as much of the weights a token as a
// pair has, in tiles of half the tokens (a ring of two stages: of no use in the
// other). us, 128 x 128 and 128 x 256: 16384 rows of 64 experts, 2560 -> 2432 143.6,
// 138.1; of 32, 2560 -> 4864 225, 216; 1024 rows of 8, 2560 -> 2432 20.6, 18.2; 4096 rows
// of 32 50.2, 57.2.
static const Fp8LargeChoice kChoices[] = {
    {true, 256, 481}, {true, 128, 252}, {false, 128, 276}, {false, 64, 236}, {false, 256, 482}};

// the tile of the smallest estimated time: waves x ns per block. (Rows of `experts`:
// the last tile of each is taken as half full, and each has one.)
static int fp8_large_choice(int64_t M, int64_t N, int sms, int64_t experts) {
  int best = 3;
  double best_t = 1e300;
  for (int i = 0; i < (experts ? 5 : 4); ++i) {
    const Fp8LargeChoice& c = kChoices[i];
    const int ctas = c.pair ? 2 : 1;
    if (sms < ctas) continue;
    const int64_t full = ceil_div(M, 128 * ctas) + experts / 2, least = M < experts ? M : experts;
    const int64_t tiles = (full > least ? full : least) * ceil_div(N, c.w);
    const double t = (double)ceil_div(tiles, sms / ctas) * c.step;
    if (t < best_t) { best_t = t; best = i; }
  }
  return best;
}

// (experts: 0 where the product is not grouped)
void fp8_grouped_large_tile(int64_t M, int64_t N, int64_t experts, int sms, int* tokens, int* rows) {
  const Fp8LargeChoice& c = kChoices[fp8_large_choice(M, N, sms, experts)];
  *tokens = c.pair ? 256 : 128;
  *rows = c.w;
}

void fp8_tile(int64_t M, int64_t N, int sms, int* tokens, int* rows) {
  if (M <= kFp8SmallM) return fp8_small_tile(M, N, sms, tokens, rows);
  fp8_grouped_large_tile(M, N, 0, sms, tokens, rows);
}

template <bool kF32, bool kGrouped>
static cudaError_t launch_large_any(const uint8_t* q, int64_t K, const uint8_t* w, int64_t ldw, int64_t lde,
                                    const Fp8LargeArgs& a, cudaStream_t st) {
  switch (fp8_large_choice(a.M, a.N, num_sms(), kGrouped ? a.E : 0)) {
    case 0: return launch_large<true, 256, kF32, kGrouped>(q, K, w, ldw, lde, a, st);
    case 1: return launch_large<true, 128, kF32, kGrouped>(q, K, w, ldw, lde, a, st);
    case 2: return launch_large<false, 128, kF32, kGrouped>(q, K, w, ldw, lde, a, st);
    case 4:
      if constexpr (kGrouped) return launch_large<false, 256, kF32, kGrouped>(q, K, w, ldw, lde, a, st);
      return cudaErrorInvalidValue;
    default: return launch_large<false, 64, kF32, kGrouped>(q, K, w, ldw, lde, a, st);
  }
}

// gemm_fp8_grouped for many rows an expert
cudaError_t launch_gemm_fp8_grouped_large(const uint8_t* q, const float* scale, int64_t lds, int64_t M, int64_t K,
                                          const int64_t* offsets, int64_t E, const uint8_t* w, int64_t ldw,
                                          int64_t lde, const float* w_scale, int64_t N, void* out, bool out_f32,
                                          int64_t ldo, uint32_t* err, cudaStream_t st) {
  const Fp8LargeArgs a{scale, w_scale, out, lds, ldo, (int)M, (int)N, (int)ceil_div(K, 128),
                       (int)ceil_div(N, 128), 0, 0, 0, err, offsets, (int)E};
  return out_f32 ? launch_large_any<true, true>(q, K, w, ldw, lde, a, st)
                 : launch_large_any<false, true>(q, K, w, ldw, lde, a, st);
}

cudaError_t launch_gemm_fp8(const uint8_t* q, const float* scale, int64_t lds, int64_t M, int64_t K,
                            const uint8_t* w, int64_t ldw, const float* w_scale, int64_t N,
                            void* out, bool out_f32, int64_t ldo, uint32_t* err, bool pdl,
                            cudaStream_t st) {
  if (M <= kFp8SmallM)
    return launch_gemm_fp8_small(q, scale, lds, M, K, w, ldw, w_scale, N, out, out_f32, ldo, err,
                                 pdl, st);
  Fp8LargeArgs a{scale, w_scale, out, lds, ldo, (int)M, (int)N, (int)ceil_div(K, 128),
                 (int)ceil_div(N, 128), 0, 0, pdl, err, nullptr, 0};
  return out_f32 ? launch_large_any<true, false>(q, K, w, ldw, 0, a, st)
                 : launch_large_any<false, false>(q, K, w, ldw, 0, a, st);
}

}  // namespace qg
