// lora.cu -- low-rank adapters of many requests beside a shared projection.
//
//   h[m][r]   = sum_k x[m][k] * A[id][r][k]        id = ids[m]
//   out[m][n] = base[m][n] + sum_r (scaling[id] * h[m][r]) * B[id][n][r]
// A row whose id is not one of the adapters keeps base's bits.
//
// `shrink` sums h over parts of K, which are added up in order and scaled; `expand`
// adds the second product to base. The parts are cut by K alone,
// so a row's bits do not depend on the other rows, but for the choice of the kernels:
//   few rows (decode), bound by reading the adapters that the rows use: a row at a
//   time on the fp32 units, a few products for every value read;
//   more rows, bound by x, base and out: products on the tensor cores, where
//   scaling * h goes in as the sum of two bf16 numbers (off by 2^-17 of itself, far
//   less than a bf16 output's rounding) or, for fp32 outputs, of three (2^-24),
//   everything by TMA.
// Each kernel is a programmatic dependent of the one before it. Rows may come in
// any order. Many rows are taken in tiles of 128, in which the different ids are
// found by votes; each costs a pass over the tile.
#include <cuda.h>

#include <cstring>

#include "qg_common.cuh"

namespace qg {

bool make_tmap_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols,
                  int64_t rows, int64_t pitch, uint32_t box_cols, uint32_t box_rows,
                  CUtensorMapSwizzle swizzle);
bool make_tmap_3d(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols,
                  int64_t rows, int64_t mats, int64_t pitch, int64_t mat_pitch, uint32_t box_cols,
                  uint32_t box_rows, CUtensorMapSwizzle swizzle);

// Rows that are taken one at a time. GPU us of a call with one adapter and with one of 16
// each row, one at a time | by tensor cores: 5120 -> 5120, rank 32, 96 rows 13.0, 17.1 |
// 12.7, 27.7, 128 rows 14.6, 17.6 | 13.6, 28.2; rank 64, 32 rows 11.1, 13.6 | 13.3, 25.8,
// 64 rows 16.9, 20.5 | 13.6, 28.1; 5120 -> 17408, 32 rows 21.0, 28.3 | 14.6, 28.3, 64
// rows 35, 42 | 16, 31; 2560 -> 9728, rank 128, 16 rows 14.4, 17.7 | 15.1, 23.0, 32 rows
// 26, 31 | 16, 27.
static int64_t few_rows(int64_t rank) { return rank <= 32 ? 128 : rank <= 64 ? 32 : 16; }
constexpr int kManyParts = 8;                      // parts of K of many rows

struct LoraArgs {
  const void* x;
  const uint16_t *a, *b;  // bf16 [count][rank][K], [count][N][rank]
  const int64_t* ids;
  const float* scaling;   // [count] or null
  const void* base;
  void* out;
  float* h;               // sums [part of K][M][rp], rp ranks a row (many rows: up to 16, 32, 64 or 128)
  uint32_t* parts;        // many rows: scaling * h as [large to small numbers][M][rp / 2] pairs of bf16
  int64_t ldx, ldb, ldo, M;
  int K, N, rank, count, rp;
  int numbers;            // many rows: bf16 numbers that scaling * h is the sum of
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// the same, rounded towards zero
__device__ __forceinline__ uint32_t bf16x2_rz(float lo, float hi) {
  uint32_t r;
  asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// the id of row m as an adapter's number, -1 for none
__device__ __forceinline__ int adapter_of(const LoraArgs& a, int64_t m) {
  if (m >= a.M) return -1;
  const int64_t id = __ldg(a.ids + m);
  return id >= 0 && id < a.count ? (int)id : -1;
}

// one value of base or out
template <bool kBf16>
__device__ __forceinline__ uint32_t load_raw(const void* p, int64_t i) {
  if (kBf16) return reinterpret_cast<const uint16_t*>(p)[i];
  return reinterpret_cast<const uint32_t*>(p)[i];
}
template <bool kBf16>
__device__ __forceinline__ void store_raw(void* p, int64_t i, uint32_t v) {
  if (kBf16) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)v;
  else reinterpret_cast<uint32_t*>(p)[i] = v;
}
template <bool kBf16>
__device__ __forceinline__ uint32_t add_raw(uint32_t v, float y) {
  if (kBf16) return f32_to_bf16_rne(__uint_as_float(v << 16) + y);
  return __float_as_uint(__uint_as_float(v) + y);
}

// -------------------------------------------------------------------- few rows
// A CTA sums one part of K (up to 1024 values) of one row for 8 R ranks, a warp the
// ranks warp and warp + 8: 8 values a lane at a time, up to kU times, all loads ahead of
// the first product.
constexpr int kFewWarps = 8, kFewPart = 128;  // eights of a part
__host__ __device__ inline int few_parts(int K) { return (K / 8 + kFewPart - 1) / kFewPart; }

template <bool kBf16, int R>
__global__ void __launch_bounds__(32 * kFewWarps) lora_shrink_few_kernel(const LoraArgs a) {
  griddep_launch_dependents();
  constexpr int kU = 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = blockIdx.x, parts = gridDim.x;
  const int r0 = (int)blockIdx.z * R * kFewWarps + warp;  // its first rank
  const int64_t m = blockIdx.y;
  const int id = adapter_of(a, m);
  if (id < 0) return;
  const int eights = a.K / 8;
  const int e0 = eights * part / parts, e1 = eights * (part + 1) / parts;
  const char* px = reinterpret_cast<const char*>(a.x) + m * a.ldx * (kBf16 ? 2 : 4);
  const uint16_t* pa = a.a + (int64_t)id * a.rank * a.K;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  float acc[R];
#pragma unroll
  for (int i = 0; i < R; ++i) acc[i] = 0.0f;
  for (int base = e0 + lane; base - lane < e1; base += 32 * kU) {
    uint4 x[kU][kBf16 ? 1 : 2], w[kU][R];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int e = base + 32 * u;
#pragma unroll
      for (int j = 0; j < (kBf16 ? 1 : 2); ++j)
        x[u][j] = e < e1 ? __ldg(reinterpret_cast<const uint4*>(px) + (kBf16 ? 1 : 2) * e + j) : zero;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int r = r0 + i * kFewWarps;
        w[u][i] = e < e1 && r < a.rank ? __ldg(reinterpret_cast<const uint4*>(pa + (int64_t)r * a.K) + e) : zero;
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float f[8];
      if (kBf16) {
        const uint32_t v[4] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[2 * j] = bf16_lo(v[j]);
          f[2 * j + 1] = bf16_hi(v[j]);
        }
      } else {
        const uint4 lo = x[u][0], hi = x[u][kBf16 ? 0 : 1];
        const uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(v[j]);
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint32_t v[4] = {w[u][i].x, w[u][i].y, w[u][i].z, w[u][i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i] = fmaf(f[2 * j], bf16_lo(v[j]), acc[i]);
          acc[i] = fmaf(f[2 * j + 1], bf16_hi(v[j]), acc[i]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = r0 + i * kFewWarps;
    if (r >= a.rank) break;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (lane == 0) a.h[((int64_t)part * a.M + m) * a.rp + r] = acc[i];
  }
}

// A warp adds to 32 C columns of up to kFewRows rows (`group`), one after another, a
// lane to column lane (+ 32). B's part for a row (contiguous: columns x rank) comes
// through a ring of the warp's own by bulk copies, once for rows that follow one
// another with one id. A lane reads its column's ranks eight at a time, starting
// with another eight than its neighbours, so that their reads do not conflict.
constexpr int kExpandWarps = 4, kExpandRing = 4, kFewRows = 8;
template <bool kBf16, int C>
__global__ void __launch_bounds__(32 * kExpandWarps) lora_expand_few_kernel(const LoraArgs a, int group, uint32_t* err) {
  extern __shared__ __align__(128) uint8_t smem[];  // [warp][slot][column][rank], then h [row][rank]
  __shared__ uint64_t full[kExpandWarps][kExpandRing];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = a.rank;
  const int slot_bytes = 32 * C * rank * 2;
  uint8_t* const ring = smem + warp * kExpandRing * slot_bytes;
  float* const h = reinterpret_cast<float*>(smem + kExpandWarps * kExpandRing * slot_bytes);
  const int col0 = ((int)blockIdx.x * kExpandWarps + warp) * 32 * C;
  const int cols = min(32 * C, a.N - col0);  // (none: a warp behind the last column)
  const int64_t m0 = (int64_t)blockIdx.y * group;
  const int rows = (int)min((int64_t)group, a.M - m0);
  const bool keep = a.base == a.out && a.ldb == a.ldo;  // rows without an adapter are in place
  const int mine = lane < rows ? adapter_of(a, m0 + lane) : -1;
  // a row brings B unless the last row before it that has an adapter has the same
  const uint32_t with = __ballot_sync(0xffffffffu, mine >= 0);
  const uint32_t before = with & ((1u << lane) - 1);
  const int last = __shfl_sync(0xffffffffu, mine, before ? 31 - __clz(before) : 0);
  const uint32_t brings = cols > 0 ? __ballot_sync(0xffffffffu, mine >= 0 && (!before || last != mine)) : 0;
  if (lane == 0) {
    for (int i = 0; i < kExpandRing; ++i) mbar_init(&full[warp][i], 1);
    fence_barrier_init();
  }
  __syncwarp();
  uint32_t left = brings;  // rows whose B has not been asked for
  int asked = 0;
  auto ask = [&] {
    if (!left) return;
    const int id = __shfl_sync(0xffffffffu, mine, __ffs(left) - 1), s = asked % kExpandRing;
    left &= left - 1;
    ++asked;
    if (lane == 0) {
      fence_proxy_async_smem();  // (the slot's reads come before its refill)
      mbar_arrive_expect_tx(&full[warp][s], cols * rank * 2);
      bulk_copy_g2s(ring + s * slot_bytes, a.b + ((int64_t)id * a.N + col0) * rank, cols * rank * 2, &full[warp][s]);
    }
    __syncwarp();
  };
#pragma unroll
  for (int i = 0; i < kExpandRing; ++i) ask();
  uint32_t raw[C], raw_next[C];
  auto load_base = [&](int row, uint32_t (&v)[C]) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      v[c] = row < rows && lane + 32 * c < cols ? load_raw<kBf16>(a.base, (m0 + row) * a.ldb + col0 + lane + 32 * c) : 0;
  };
  load_base(0, raw);
  // nothing above is shrink's work; out may be what a kernel before it reads
  griddep_wait();
  const int parts = few_parts(a.K);
  for (int e = threadIdx.x; e < rows * (rank / 4); e += 32 * kExpandWarps) {
    const int row = e / (rank / 4), r = e % (rank / 4) * 4;
    const int id = adapter_of(a, m0 + row);
    if (id < 0) continue;
    float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 8
    for (int i = 0; i < parts; ++i) {
      const float4 p = *reinterpret_cast<const float4*>(a.h + ((int64_t)i * a.M + m0 + row) * a.rp + r);
      v.x += p.x;
      v.y += p.y;
      v.z += p.z;
      v.w += p.w;
    }
    const float scale = a.scaling ? __ldg(a.scaling + id) : 1.0f;
    *reinterpret_cast<float4*>(h + row * rank + r) = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
  }
  __syncthreads();
  int used = -1;  // the slot in use, counted from the first
  for (int row = 0; row < rows && cols > 0; ++row) {
    load_base(row + 1, raw_next);
    if (with >> row & 1) {
      if (brings >> row & 1) {
        if (used >= 0) {
          __syncwarp();  // every lane has read the slot that is asked for again
          ask();
        }
        ++used;
        mbar_wait_warp(&full[warp][used % kExpandRing], (uint32_t)(used / kExpandRing) & 1u, err);
      }
      const uint8_t* from = ring + (used % kExpandRing) * slot_bytes;
      const int eights = rank >> 3;
      float acc[C];
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] = 0.0f;
      int e = lane % eights;
#pragma unroll 2
      for (int i = 0; i < eights; ++i) {
        const float4 h0 = *reinterpret_cast<const float4*>(h + row * rank + e * 8);
        const float4 h1 = *reinterpret_cast<const float4*>(h + row * rank + e * 8 + 4);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint4 v = *reinterpret_cast<const uint4*>(from + (lane + 32 * c) * rank * 2 + e * 16);
          acc[c] = fmaf(h0.x, bf16_lo(v.x), acc[c]);
          acc[c] = fmaf(h0.y, bf16_hi(v.x), acc[c]);
          acc[c] = fmaf(h0.z, bf16_lo(v.y), acc[c]);
          acc[c] = fmaf(h0.w, bf16_hi(v.y), acc[c]);
          acc[c] = fmaf(h1.x, bf16_lo(v.z), acc[c]);
          acc[c] = fmaf(h1.y, bf16_hi(v.z), acc[c]);
          acc[c] = fmaf(h1.z, bf16_lo(v.w), acc[c]);
          acc[c] = fmaf(h1.w, bf16_hi(v.w), acc[c]);
        }
        if (++e == eights) e = 0;
      }
#pragma unroll
      for (int c = 0; c < C; ++c) raw[c] = add_raw<kBf16>(raw[c], acc[c]);
    }
    if ((with >> row & 1) || !keep) {  // (a row without an adapter keeps base's bits)
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (lane + 32 * c < cols) store_raw<kBf16>(a.out, (m0 + row) * a.ldo + col0 + lane + 32 * c, raw[c]);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) raw[c] = raw_next[c];
  }
  // (every copy asked for has been waited for: each is some row's)
}

// ------------------------------------------------------------------- many rows
// D (16 x 8) += A (16 x 16) * B (16 x 8), bf16 operands, fp32 sums
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// position of set bit number n (from 0) of a mask that has more than n
__device__ __forceinline__ int nth_bit(uint32_t mask, int n) {
  int pos = 0;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1)
    if (__popc(mask & ((1u << (pos + s)) - 1)) <= n) pos += s;
  return pos;
}

// The pieces of a window's rows: piece j has those of the j-th different id
// (rows without an adapter are a piece, too, id -1).
struct LoraPieces {
  int mine;          // this lane's row's adapter
  uint32_t same;     // the rows that share it
  uint32_t leaders;  // one row of each piece that is left
  __device__ LoraPieces(const LoraArgs& a, int64_t m0, int rows) {
    const int lane = threadIdx.x & 31;
    const bool row = lane < rows && m0 + lane < a.M;
    mine = row ? adapter_of(a, m0 + lane) : -2;
    same = __match_any_sync(0xffffffffu, mine);
    leaders = __ballot_sync(0xffffffffu, row && lane == __ffs(same) - 1);
  }
  // the next piece that is `z` modulo `step`: its id and rows; false when there is none
  __device__ bool next(int& j, int z, int step, int& id, uint32_t& rows) {
    while (leaders) {
      const int first = __ffs(leaders) - 1;
      leaders &= leaders - 1;
      if (j++ % step != z) continue;
      id = __shfl_sync(0xffffffffu, mine, first);
      rows = __shfl_sync(0xffffffffu, same, first);
      return true;
    }
    return false;
  }
};

// One step of 32 values of K: A's rows are the MMA's 16, 8 rows of x its columns. A
// lane has 8 consecutive k of a row of each: k 8t.. of 32, t = lane % 4, in
// whatever order the MMA sums them. A value of x goes in as the sum of three bf16
// numbers (24 bits), each rounded towards zero: to the nearest, values above 2^128 -
// 2^119 would become infinite.
template <int RT>
struct ShrinkStep {
  uint4 w[RT][2], x[2];
  __device__ __forceinline__ void multiply(float (&acc)[RT][4]) const {
    const uint32_t u[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    float f[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) f[c] = __uint_as_float(u[c]);
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      uint32_t v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[c] = bf16x2_rz(f[2 * c], f[2 * c + 1]);
        // (an infinity's rest would be NaN)
        f[2 * c] = isfinite(bf16_lo(v[c])) ? f[2 * c] - bf16_lo(v[c]) : 0.0f;
        f[2 * c + 1] = isfinite(bf16_hi(v[c])) ? f[2 * c + 1] - bf16_hi(v[c]) : 0.0f;
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const uint32_t f0[4] = {w[r][0].x, w[r][1].x, w[r][0].y, w[r][1].y};
        const uint32_t f1[4] = {w[r][0].z, w[r][1].z, w[r][0].w, w[r][1].w};
        mma_bf16_16816(acc[r], f0, v[0], v[1]);
        mma_bf16_16816(acc[r], f1, v[2], v[3]);
      }
    }
  }
};

// asynchronous 16-byte global -> shared copy; `in` false: zeros
__device__ __forceinline__ void cp_async_16(void* to, const void* from, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(in ? 16 : 0)
               : "memory");
}

// Many rows of fp32 x, which tcgen05 has no type of enough bits for: windows of 32
// rows; a CTA a part of K, whose steps (32 values of every row of x and of A) it
// brings through a ring in shared memory; warp w multiplies rows 8w.. of the
// piece. A step's rows of A lie 64 bytes apart, which a lane's 16-byte reads of row
// lane / 4, piece lane % 4, take without conflicts. Two steps are fetched at once.
// A part is cut into eight shares, whose sums are added in order (chains of MMAs of
// bounded length).
constexpr int kManyWarps = 4, kManyRing = 4, kShares = 8;
template <int RT>
struct ManyCfg {
  static constexpr int kX = 32 * 128, kA = RT * 16 * 64, kStep = kX + kA;
  static constexpr int kSmem = kManyRing * 2 * kStep;
};

template <int RT>
__global__ void __launch_bounds__(32 * kManyWarps) lora_shrink_f32_kernel(const LoraArgs a) {
  griddep_launch_dependents();
  using C = ManyCfg<RT>;
  constexpr int RP = RT * 16, kThreads = 32 * kManyWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int kg = blockIdx.x;
  const int64_t m0 = (int64_t)blockIdx.y * 32;
  const int units = (a.K + 31) >> 5;
  const int u0 = units * kg / kManyParts, u1 = units * (kg + 1) / kManyParts;  // this group's steps
  LoraPieces pieces(a, m0, 32);
  int id, j = 0;
  uint32_t rows;
  while (pieces.next(j, blockIdx.z, gridDim.z, id, rows)) {
    if (id < 0) continue;
    const int count = __popc(rows);
    const uint16_t* pa = a.a + (int64_t)id * a.rank * a.K;
    // x: eight threads a row, 16 rows a round
    constexpr int kPer = 8, kRounds = 32 * kPer / kThreads;
    const char* px[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      px[i] = reinterpret_cast<const char*>(a.x) +
              (m0 + nth_bit(rows, min(i * (kThreads / kPer) + (int)threadIdx.x / kPer, count - 1))) * a.ldx *
                  4;
    auto fetch = [&](int u) {  // steps u and u + 1
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        uint8_t* to = smem + (((u - u0) / 2 % kManyRing) * 2 + d) * C::kStep;
        const bool in = u + d < u1;
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
          const int c = threadIdx.x % kPer, row = i * (kThreads / kPer) + (int)threadIdx.x / kPer;
          const int k = (u + d) * 32 + c * 4;
          const bool ok = in && row < count && k < a.K;
          cp_async_16(to + row * 128 + c * 16, px[i] + (ok ? (int64_t)k * 4 : 0), ok);
        }
#pragma unroll
        for (int i = 0; i < (RP * 4 + kThreads - 1) / kThreads; ++i) {
          const int e = i * kThreads + threadIdx.x, row = e >> 2, c = e & 3, k = (u + d) * 32 + c * 8;
          if (RP * 4 % kThreads && row >= RP) break;
          const bool ok = in && row < a.rank && k < a.K;
          cp_async_16(to + C::kX + row * 64 + c * 16, ok ? pa + (int64_t)row * a.K + k : pa, ok);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kManyRing - 1; ++i) fetch(u0 + 2 * i);
    float group[RT][4], acc[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) group[r][c] = acc[r][c] = 0.0f;
    int share = kg * kShares;
    int end = units * (share + 1) / (kShares * kManyParts);  // of the share
    auto fold = [&](int u) {                              // shares that end at step u
      while (u == end && share < (kg + 1) * kShares) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            group[r][c] += acc[r][c];
            acc[r][c] = 0.0f;
          }
        ++share;
        end = units * (share + 1) / (kShares * kManyParts);
      }
    };
    fold(u0);
    for (int u = u0; u < u1; u += 2) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kManyRing - 2) : "memory");
      __syncthreads();
      fetch(u + 2 * (kManyRing - 1));  // (into the slot that the last round read)
      if (warp * 8 < count) {
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          if (u + d >= u1) break;
          const uint8_t* from = smem + (((u - u0) / 2 % kManyRing) * 2 + d) * C::kStep;
          ShrinkStep<RT> s;
          const uint8_t* fx = from + (warp * 8 + g) * 128 + t * 32;
#pragma unroll
          for (int i = 0; i < 2; ++i) s.x[i] = *(reinterpret_cast<const uint4*>(fx) + i);
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              s.w[r][h] = *reinterpret_cast<const uint4*>(from + C::kX + (r * 16 + h * 8 + g) * 64 + t * 16);
          s.multiply(acc);
          fold(u + d + 1);
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // group[r]: ranks 16r + g (c 0, 1) and + 8 (c 2, 3) of rows 2t and + 1 of the warp's eight
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int n = warp * 8 + 2 * t + c;
      if (n >= count) continue;
      float* to = a.h + ((int64_t)kg * a.M + m0 + nth_bit(rows, n)) * RP + g;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        to[r * 16] = group[r][c];
        to[r * 16 + 8] = group[r][2 + c];
      }
    }
    __syncthreads();  // the ring has been read
  }
}

// The different adapters of 128 rows, in the order of their first rows of a lane:
// number k in lane k % 32 (every warp that asks finds them by itself).
struct TileIds {
  int list[4], count;
  int v[4];  // the ids of rows lane, lane + 32, ...
  __device__ __forceinline__ void load(const LoraArgs& a, int64_t m0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = adapter_of(a, m0 + j * 32 + (threadIdx.x & 31));
  }
  __device__ __forceinline__ void find() {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) list[j] = -1;
    count = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t left;
      while ((left = __ballot_sync(0xffffffffu, v[j] >= 0)) != 0) {
        const int id = __shfl_sync(0xffffffffu, v[j], __ffs(left) - 1);
#pragma unroll
        for (int i = j; i < 4; ++i)
          if (v[i] == id) v[i] = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (count == i * 32 + lane) list[i] = id;
        ++count;
      }
    }
  }
  __device__ __forceinline__ int at(int k) const {
    const int v = k < 32 ? list[0] : k < 64 ? list[1] : k < 96 ? list[2] : list[3];
    return __shfl_sync(0xffffffffu, v, k & 31);
  }
};

// Instruction descriptor, kind::f16: D fp32, A and B bf16, both K-major
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// four ranks of a row of scaling * h as two or three bf16 numbers each. (Ranks that
// only pad: 0, also where x is infinite.)
__device__ __forceinline__ void put_parts(const LoraArgs& a, int64_t m, int r, float4 v, float scale) {
  v = r < a.rank ? make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale) : make_float4(0, 0, 0, 0);
  auto rest = [](float f, float h) { return isfinite(h) ? f - h : 0.0f; };  // (an infinity's would be NaN)
  uint2* to = reinterpret_cast<uint2*>(a.parts) + (m * a.rp + r) / 4;
  // (a finite number's nearest is finite, too: bf16's largest for those above 2^128 - 2^119)
  auto near = [](float f) { return isfinite(f) ? fminf(fmaxf(f, -0x1.FEp127f), 0x1.FEp127f) : f; };
  for (int i = 0; i < a.numbers; ++i, to += a.M * (a.rp / 4)) {
    const uint2 n = make_uint2(bf16x2(near(v.x), near(v.y)), bf16x2(near(v.z), near(v.w)));
    *to = n;
    v = make_float4(rest(v.x, bf16_lo(n.x)), rest(v.y, bf16_hi(n.x)), rest(v.z, bf16_lo(n.y)), rest(v.w, bf16_hi(n.y)));
  }
}

// Many rows of bf16 x. A cluster of eight CTAs, one a part of K, multiplies 128 rows
// with the A of each of their adapters: D, 128 rows x RP ranks in tensor memory, of
// 64 values of K a step (x 16 KB and A by TMA), for up to four adapters at once. The
// parts' sums meet in shared memory, where every CTA adds up 16 rows, in order. Two
// CTAs an SM (one for ranks above 64). Of 10.5 us (4096 x 5120, rank 64) the steps
// are 3.6; the CTAs of a launch of this size start over 3 us, the ids take 0.9 and the
// meeting of the cluster 2.7.
// Warps: 0 producer, 1 MMA issuer, 2..5 epilogue (32 rows each: a row a thread).
template <int RP>
struct ShrinkTc {
  static constexpr int kX = 128 * 128, kA = RP * 128, kRing = 3, kARing = RP == 128 ? 4 : 3, kPitch = RP + 4;
  static constexpr int kBatch = 4, kCols = kBatch * RP;
  static constexpr size_t kSmem = kRing * kX + kARing * kA + 128 * kPitch * 4 + 1024;
};

template <int RP>
__global__ void __cluster_dims__(kManyParts, 1, 1) __launch_bounds__(192, RP == 128 ? 1 : 2)
    lora_shrink_tc_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmA,
                          const LoraArgs a, uint32_t* err) {
  using C = ShrinkTc<RP>;
  griddep_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t x_full[C::kRing], x_empty[C::kRing], a_full[C::kARing], a_empty[C::kARing], d_full, drain;
  __shared__ uint32_t tmem_slot, tmem_busy;
  __shared__ int ids[128];  // the adapters of the rows
  uint8_t* sx = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sa = sx + C::kRing * C::kX;
  float* sum = reinterpret_cast<float*>(sa + C::kARing * C::kA);  // [row][rank], kPitch apart
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = (int)cluster_ctarank();
  const int64_t m0 = (int64_t)blockIdx.y * 128;
  const int all = (a.K + 63) / 64, k0 = all * part / kManyParts, k1 = all * (part + 1) / kManyParts;  // steps
  TileIds T;
  T.load(a, m0);
  const int q = warp & 3, mine = q == 0 ? T.v[0] : q == 1 ? T.v[1] : q == 2 ? T.v[2] : T.v[3];  // of row 32 q + lane
  T.find();
  const int per = (T.count + (int)gridDim.z - 1) / (int)gridDim.z;  // adapters of this cluster
  const int i0 = per * (int)blockIdx.z, i1 = min(T.count, i0 + per);
  if (i0 >= i1) return;  // (every thread of the cluster)
  if (warp == 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) ids[j * 32 + lane] = T.list[j];
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(&x_full[i], 1);
      mbar_init(&x_empty[i], 1);
    }
    for (int i = 0; i < C::kARing; ++i) {
      mbar_init(&a_full[i], 1);
      mbar_init(&a_empty[i], 1);
    }
    mbar_init(&d_full, 1);
    mbar_init(&drain, 1);
    tmem_busy = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    if (elect_one()) {
      tma_prefetch_desc(&tmX);
      tma_prefetch_desc(&tmA);
    }
    __syncwarp();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  bool ok = true;
  // of the producer and of the issuer: slots, phases (a fresh slot is free), loads so far
  int s = 0, sA = 0, loads = 0, loadsA = 0;
  uint32_t phase = warp == 0, phaseA = warp == 0, phaseD = 0;
  for (int first = i0; first < i1; first += C::kBatch) {
    const int batch = min(C::kBatch, i1 - first);
    if (warp == 0) {
      for (int k = k0; k < k1 && ok; ++k) {
        ok = mbar_wait_warp(&x_empty[s], phase, err);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&x_full[s], C::kX);
          tma_load_2d(sx + s * C::kX, &tmX, &x_full[s], k * 64, (int)m0);
        }
        __syncwarp();
        ++loads;
        if (++s == C::kRing) { s = 0; phase ^= 1; }
        for (int i = 0; i < batch; ++i) {
          const int id = T.at(first + i);
          ok = mbar_wait_warp(&a_empty[sA], phaseA, err);
          if (!ok) break;
          if (elect_one()) {
            mbar_arrive_expect_tx(&a_full[sA], C::kA);
            tma_load_3d(sa + sA * C::kA, &tmA, &a_full[sA], k * 64, 0, id);
          }
          __syncwarp();
          ++loadsA;
          if (++sA == C::kARing) { sA = 0; phaseA ^= 1; }
        }
      }
    } else if (warp == 1) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, RP);
      for (int k = k0; k < k1 && ok; ++k) {
        const uint64_t xa = smem_desc_sw128(smem_u32(sx + s * C::kX));
        ok = mbar_wait_warp(&x_full[s], phase, err);
        for (int i = 0; i < batch && ok; ++i) {
          const uint64_t aa = smem_desc_sw128(smem_u32(sa + sA * C::kA));
          ok = mbar_wait_warp(&a_full[sA], phaseA, err);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_f16_ss(tmem + i * RP, xa + j * 2, aa + j * 2, idesc, k > k0 || j > 0);
            mma_commit(&a_empty[sA]);
            if (i + 1 == batch) mma_commit(&x_empty[s]);
            if (i + 1 == batch && k + 1 == k1) mma_commit(&d_full);
          }
          __syncwarp();
          if (++sA == C::kARing) { sA = 0; phaseA ^= 1; }
        }
        if (++s == C::kRing) { s = 0; phase ^= 1; }
      }
    } else {
      if (k0 < k1) {
        if (ok) ok = mbar_wait_warp(&d_full, phaseD, err);
        phaseD ^= 1;
        tc_fence_after();
      }
      for (int i = 0; i < batch; ++i) {
        const int id = T.at(first + i);
        if (!__any_sync(0xffffffffu, mine == id)) continue;
#pragma unroll
        for (int c = 0; c < RP; c += 16) {
          uint32_t v[16];
          tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + i * RP + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) asm volatile("" : "+r"(v[j]));
          if (mine == id) {
#pragma unroll
            for (int j = 0; j < 4; ++j)  // (a part without steps: nothing has been summed)
              *reinterpret_cast<uint4*>(sum + (q * 32 + lane) * C::kPitch + c + 4 * j) =
                  k0 < k1 ? make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]) : make_uint4(0, 0, 0, 0);
          }
        }
      }
      tc_fence_before();
    }
    cluster_sync();  // the sums are there, the accumulators have been read
    tc_fence_after();
    for (int e = threadIdx.x; e < 16 * (RP / 4); e += 192) {
      const int row = part * 16 + e / (RP / 4), r = e % (RP / 4) * 4, id = adapter_of(a, m0 + row);
      bool here = false;  // whether its sums are of this batch
      for (int i = 0; i < batch; ++i) here |= id == ids[first + i];
      if (id < 0 || !here) continue;
      float4 v = make_float4(0, 0, 0, 0), p[kManyParts];
#pragma unroll
      for (int c = 0; c < kManyParts; ++c)
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(p[c].x), "=f"(p[c].y), "=f"(p[c].z), "=f"(p[c].w)
                     : "r"(map_to_cta(sum + row * C::kPitch + r, c))
                     : "memory");
#pragma unroll
      for (int c = 0; c < kManyParts; ++c) {
        v.x += p[c].x;
        v.y += p[c].y;
        v.z += p[c].z;
        v.w += p[c].w;
      }
      put_parts(a, m0 + row, r, v, a.scaling ? __ldg(a.scaling + id) : 1.0f);
    }
    cluster_sync();  // the sums have been read
  }
  if (warp == 0) {
    // every load has landed before the CTA exits
    for (int i = max(0, loads - C::kRing); i < loads; ++i)
      mbar_wait_warp(&x_full[i % C::kRing], (uint32_t)(i / C::kRing) & 1u, err);
    for (int i = max(0, loadsA - C::kARing); i < loadsA; ++i)
      mbar_wait_warp(&a_full[i % C::kARing], (uint32_t)(i / C::kARing) & 1u, err);
  } else if (warp == 1 && !ok) {
    // (after a wait that gave up, MMAs issued so far may still run; bounded)
    if (elect_one()) mma_commit(&drain);
    __syncwarp();
    if (!mbar_wait_warp(&drain, 0, err)) atomicExch(&tmem_busy, 1u);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1 && tmem_busy == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

// The same end for the parts' sums that lora_shrink_f32_kernel leaves; a thread
// four ranks of a row. Rows without an adapter are left: nothing reads their products.
__global__ void __launch_bounds__(256) lora_join_kernel(const LoraArgs a) {
  griddep_launch_dependents();
  const int fours = a.rp / 4;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x, m = e / fours;
  const int r = (int)(e - m * fours) * 4, id = adapter_of(a, m);
  const float scale = id >= 0 && a.scaling ? __ldg(a.scaling + id) : 1.0f;
  griddep_wait();
  if (id < 0) return;
  float4 v = make_float4(0, 0, 0, 0), p[kManyParts];
#pragma unroll
  for (int i = 0; i < kManyParts; ++i)
    p[i] = *reinterpret_cast<const float4*>(a.h + ((int64_t)i * a.M + m) * a.rp + r);
#pragma unroll
  for (int i = 0; i < kManyParts; ++i) {
    v.x += p[i].x;
    v.y += p[i].y;
    v.z += p[i].z;
    v.w += p[i].w;
  }
  put_parts(a, m, r, v, scale);
}

// Many rows. Bound by reading base and writing out, so both go by TMA, tile by
// tile (128 rows x 128 bytes), through one ring: the epilogue adds to a tile where
// it lies in shared memory and stores it from there. A tile's second product is a
// tcgen05 MMA of 128 rows x kN columns: A operand h (its two or three numbers, in
// shared memory as long as the CTA stays with its 128 rows), B operand kN rows of
// B, into an accumulator in tensor memory. Where a tile's rows have
// several adapters, it is multiplied with each, and every row (a lane of tensor
// memory, a thread) adds the one that is its own. The tiles, columns fastest, are
// cut into `sections`, and each of them evenly over the CTAs: shares of some dozen
// tiles of the same rows, from different places, so that rows of several adapters
// are everybody's. Rows of base or out that do not lie on
// 16-byte pieces (`aligned` false) are read and written element by element.
// Warps: 0 producer, 1 and 10 issuers of MMAs, 2..5 and 6..9 epilogue (32 rows each): a
// tile's waits, loads, additions and store follow one another, so the two sets take
// turns, each with an issuer, accumulators and slots of B of its own. A product
// takes its issuer 700 to 900 cycles, waits among them, so that two of them are what
// tiles of several adapters need: 64 runs in 4096 rows, 5120 -> 17408, rank 64: 108 us,
// 119 with one. A product alone in its tile takes the epilogue 1150 cycles, under the
// time that the tile's bytes take. 4096 rows, 11 runs: 76.5 us, of one adapter 73.5: the
// first kernel 10.5, a start and an end of 10, and base and out at 5.7 TB/s (a copy of
// theirs through the same ring 48.8 us in all, through plain loads and stores 43.7).
template <bool kBf16, int kHalves>  // 64 ranks each
struct ExpandMany {
  static constexpr int kN = kBf16 ? 64 : 32;  // columns of a tile: 128 bytes of a row
  static constexpr int kBase = 128 * 128, kB = kN * 128 * kHalves, kH = 128 * 128;
  static constexpr int kNumbers = kBf16 ? 2 : 3;  // of h
  static constexpr int kBaseRing = kHalves == 2 || !kBf16 ? 6 : 8, kBRing = 2, kSlots = 4;  // (B: of a set)
  static constexpr int kHBytes = kNumbers * kHalves * kH, kHRing = kHalves == 2 ? 1 : 2;
  static constexpr int kThreads = 96 + 32 * 8;
  // A set waits for its own tiles alone, and a wait on a barrier tells a phase from
  // the next one only: every slot of base and every accumulator is one set's (even
  // rings; two accumulators each).
  static_assert(kBaseRing % 2 == 0 && kSlots == 4, "slots of one set");
  static constexpr size_t kSmem = kBaseRing * kBase + 2 * kBRing * kB + kHRing * kHBytes + 1024;
};

// how the tiles are dealt out: `sections` times the number of CTAs cells of `tiles`
// tiles, the first `rest` cells one more
struct ExpandShares {
  int sections;
  uint32_t tiles, rest;
};

template <bool kBf16, int kHalves>
__global__ void __launch_bounds__(ExpandMany<kBf16, kHalves>::kThreads, 1)
    lora_expand_many_kernel(const __grid_constant__ CUtensorMap tmBase, const __grid_constant__ CUtensorMap tmB,
                            const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmH, const LoraArgs a,
                            const int aligned, const ExpandShares share, uint32_t* err) {
  using C = ExpandMany<kBf16, kHalves>;
  constexpr int kN = C::kN;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t base_full[C::kBaseRing], base_empty[C::kBaseRing];
  __shared__ uint64_t b_full[2 * C::kBRing], b_empty[2 * C::kBRing], d_full[C::kSlots], d_empty[C::kSlots], drain[2];
  __shared__ uint64_t h_full[C::kHRing], h_empty[C::kHRing];
  __shared__ uint32_t tmem_slot, tmem_busy;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sx = base;                                  // tiles of base [slot]
  uint8_t* sb = sx + C::kBaseRing * C::kBase;          // B [set][slot][half]
  uint8_t* sh = sb + 2 * C::kBRing * C::kB;                // h [slot][number][half]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t CT = (a.N + kN - 1) / kN;
  const bool keep = a.base == a.out && a.ldb == a.ldo;  // rows without an adapter are in place

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kBaseRing; ++i) {
      mbar_init(&base_full[i], 1);
      mbar_init(&base_empty[i], 4);
    }
    for (int i = 0; i < 2 * C::kBRing; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 1);
    }
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], 4);
    }
    for (int i = 0; i < C::kHRing; ++i) {
      mbar_init(&h_full[i], 1);
      mbar_init(&h_empty[i], 2);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    tmem_busy = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    if (elect_one()) {
      tma_prefetch_desc(&tmB);
      tma_prefetch_desc(&tmH);
      if (aligned) {
        tma_prefetch_desc(&tmBase);
        tma_prefetch_desc(&tmOut);
      }
    }
    __syncwarp();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, C::kSlots * kN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  // the CTA's tiles, those of the same rows together: their first row, their
  // adapters, the tiles of columns c0 up to c1. Rows that have no adapter and are in
  // place are passed over. (The next rows' ids are on their way.)
  TileIds T, ahead;
  int section = 0, c0 = 0, c1 = 0, mine = -1;  // mine: of row 32 (warp % 4) + lane
  uint32_t next = 0, end = 0;
  int64_t m0 = 0;
  // (a CTA's place in a section moves on by a quarter from one to the next: rows of
  // several adapters often lie at regular distances)
  auto enter = [&]() {
    const uint32_t place = (blockIdx.x + section * (gridDim.x / 4 + 1)) % gridDim.x;
    const uint32_t cell = section * gridDim.x + place;
    next = cell * share.tiles + min(cell, share.rest);
    end = next + share.tiles + (cell < share.rest);
  };
  enter();
  auto skip_empty = [&]() {  // to the next section while this one is done
    while (next >= end && section + 1 < share.sections) {
      ++section;
      enter();
    }
    return next < end;
  };
  if (skip_empty()) ahead.load(a, (int64_t)(next / CT) * 128);
  auto advance = [&]() {
    while (skip_empty()) {
      const uint32_t rt = next / CT, stop = min(end, (rt + 1) * CT);
      m0 = (int64_t)rt * 128;
      c0 = (int)(next - rt * CT);
      c1 = (int)(stop - rt * CT);
      next = stop;
      T = ahead;
      if (skip_empty()) ahead.load(a, (int64_t)(next / CT) * 128);
      mine = (warp & 3) == 0 ? T.v[0] : (warp & 3) == 1 ? T.v[1] : (warp & 3) == 2 ? T.v[2] : T.v[3];
      T.find();
      if (T.count || !keep) return true;
    }
    return false;
  };

  if (warp == 0) {
    bool ok = true;
    int s = 0, sH = 0, loads = 0, loadsH = 0;
    uint32_t phase = 1, phaseH = 1, n = 0;  // n: tiles so far
    int loads0 = 0, loads1 = 0;  // of B, for either set
    auto load_base = [&](int c) {
      ok = mbar_wait_warp(&base_empty[s], phase, err);
      if (!ok) return;
      if (elect_one()) {
        mbar_arrive_expect_tx(&base_full[s], C::kBase);
        tma_load_2d(sx + s * C::kBase, &tmBase, &base_full[s], c * kN, (int)m0);
      }
      __syncwarp();
      ++loads;
      if (++s == C::kBaseRing) { s = 0; phase ^= 1; }
    };
    bool waited = false;
    while (ok && advance()) {
      int from = c0;  // the tile of base that is next
      if (!waited) {
        // base is no work of the kernels before (and the slots are all free)
        for (; aligned && ok && from < min(c1, c0 + C::kBaseRing); ++from) load_base(from);
        griddep_wait();
        waited = true;
        if (!ok) break;
      }
      if (T.count) {
        ok = mbar_wait_warp(&h_empty[sH], phaseH, err);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&h_full[sH], C::kHBytes);
#pragma unroll
          for (int o = 0; o < C::kNumbers; ++o)
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              tma_load_3d(sh + sH * C::kHBytes + (o * kHalves + h) * C::kH, &tmH, &h_full[sH], h * 64, (int)m0, o);
        }
        __syncwarp();
        ++loadsH;
        if (++sH == C::kHRing) { sH = 0; phaseH ^= 1; }
      }
      for (int c = c0; c < c1 && ok; c += 2) {
        const int both = min(2, c1 - c);
        for (; aligned && ok && from < c + both; ++from) load_base(from);
        for (int k = 0; k < T.count && ok; ++k) {
          const int id = T.at(k);
          for (int i = 0; i < both; ++i) {
            const int set = (n + i) & 1, u = set ? loads1 : loads0, sB = set * C::kBRing + u % C::kBRing;
            ok = mbar_wait_warp(&b_empty[sB], (u / C::kBRing & 1) ^ 1, err);
            if (!ok) break;
            if (elect_one()) {
              mbar_arrive_expect_tx(&b_full[sB], C::kB);
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                tma_load_3d(sb + sB * C::kB + h * kN * 128, &tmB, &b_full[sB], h * 64, (c + i) * kN, id);
            }
            __syncwarp();
            if (set) ++loads1;
            else ++loads0;
          }
        }
        n += both;
      }
    }
    if (!waited) griddep_wait();  // (this kernel's end is that of those before, too)
    // every load has landed before the CTA exits
    for (int i = max(0, loadsH - C::kHRing); i < loadsH; ++i)
      mbar_wait_warp(&h_full[i % C::kHRing], (uint32_t)(i / C::kHRing) & 1u, err);
    for (int i = max(0, loads - C::kBaseRing); i < loads; ++i)
      mbar_wait_warp(&base_full[i % C::kBaseRing], (uint32_t)(i / C::kBaseRing) & 1u, err);
    for (int i = max(0, loads0 - C::kBRing); i < loads0; ++i)
      mbar_wait_warp(&b_full[i % C::kBRing], (uint32_t)(i / C::kBRing) & 1u, err);
    for (int i = max(0, loads1 - C::kBRing); i < loads1; ++i)
      mbar_wait_warp(&b_full[C::kBRing + i % C::kBRing], (uint32_t)(i / C::kBRing) & 1u, err);
  } else if (warp == 1 || warp == 10) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, kN);
    const int steps = (a.rank + 15) / 16;
    const uint32_t set = warp == 10;
    bool ok = true;
    int sH = 0;
    uint32_t phaseH = 0;
    uint32_t n = 0, units = 0;  // tiles; products for the set so far
    while (ok && advance()) {
      if (!T.count) {
        n += c1 - c0;
        continue;
      }
      ok = mbar_wait_warp(&h_full[sH], phaseH, err);
      const uint64_t da = smem_desc_sw128(smem_u32(sh + sH * C::kHBytes));
      const uint32_t mine = (uint32_t)(c1 - c0 + ((n & 1) == set)) / 2 * T.count;  // products of these tiles
      n += c1 - c0;
      for (uint32_t i = 0; i < mine && ok; ++i, ++units) {
        const uint32_t d = 2 * set + (units & 1), sB = set * C::kBRing + units % C::kBRing;
        const uint64_t db = smem_desc_sw128(smem_u32(sb + sB * C::kB));
        ok = mbar_wait_warp2(&b_full[sB], units / C::kBRing & 1, &d_empty[d], (units >> 1 & 1) ^ 1, err);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int o = C::kNumbers - 1; o >= 0; --o)  // the small numbers first
#pragma unroll
            for (int k = 0; k < 4 * kHalves; ++k)
              if (k < steps)
                mma_f16_ss(tmem + d * kN, da + (((o * kHalves + (k >> 2)) * C::kH + (k & 3) * 32) >> 4),
                           db + (((k >> 2) * kN * 128 + (k & 3) * 32) >> 4), idesc, o + 1 < C::kNumbers || k > 0);
          mma_commit(&d_full[d]);
        }
        __syncwarp();
      }
      if (elect_one()) mma_commit(&h_empty[sH]);
      __syncwarp();
      if (++sH == C::kHRing) { sH = 0; phaseH ^= 1; }
    }
    // (after a wait that gave up, MMAs issued so far may still run; bounded)
    if (!ok) {
      if (elect_one()) mma_commit(&drain[set]);
      __syncwarp();
      if (!mbar_wait_warp(&drain[set], 0, err)) atomicExch(&tmem_busy, 1u);
    }
  } else {
    const int quarter = warp & 3;
    const uint32_t set = (warp - 2) >> 2;
    bool ok = true;
    int last = -1;
    uint32_t* const stage = reinterpret_cast<uint32_t*>(sx) + set * 128 * (kN + 1);  // (not `aligned`)
    uint32_t n = 0, units = 0;  // tiles, and products for this set, so far
    bool waited = false;
    while (ok && advance()) {
      if (!waited) griddep_wait();  // (out may be what a kernel before reads, too)
      waited = true;
      const int64_t w0 = m0 + quarter * 32;
      for (int c = c0; c < c1 && ok; ++c, ++n) {
        if ((n & 1) != set) continue;
        const uint32_t s = n % C::kBaseRing;
        if (aligned) ok = mbar_wait_warp(&base_full[s], n / C::kBaseRing & 1, err);
        if (!ok) break;
        uint8_t* const row = sx + s * C::kBase + (quarter * 32 + lane) * 128;
        for (int k = 0; k < T.count; ++k, ++units) {
          const int id = T.at(k);
          const uint32_t d = 2 * set + (units & 1);
          ok = mbar_wait_warp(&d_full[d], units >> 1 & 1, err);
          if (!ok) break;
          // its part of B has been read
          if (quarter == 0 && lane == 0) mbar_arrive(&b_empty[set * C::kBRing + units % C::kBRing]);
          if (__any_sync(0xffffffffu, mine == id)) {
            tc_fence_after();
            uint32_t v[kN / 32][32];
#pragma unroll
            for (int i = 0; i < kN / 32; ++i)
              tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + d * kN + i * 32, v[i]);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < kN / 32; ++i)
#pragma unroll
              for (int j = 0; j < 32; ++j) asm volatile("" : "+r"(v[i][j]));
            tc_fence_before();
            if (mine == id && !aligned) {
              // the products alone, as they will be read: row after row, a word on
              // from row to row
#pragma unroll
              for (int i = 0; i < kN; ++i)
                stage[(quarter * 32 + lane) * (kN + 1) + i] = v[i / 32][i % 32];
            } else if (mine == id) {  // (a row without an adapter keeps base's bits)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                uint4* p = reinterpret_cast<uint4*>(row + ((i ^ (lane & 7)) * 16));
                uint4 x = *p;
                if constexpr (kBf16) {
                  auto add = [&](uint32_t u, int j) {
                    return bf16x2(bf16_lo(u) + __uint_as_float(v[j / 32][j % 32]),
                                  bf16_hi(u) + __uint_as_float(v[(j + 1) / 32][(j + 1) % 32]));
                  };
                  x = make_uint4(add(x.x, 8 * i), add(x.y, 8 * i + 2), add(x.z, 8 * i + 4), add(x.w, 8 * i + 6));
                } else {
                  auto add = [&](uint32_t u, int j) {
                    return __float_as_uint(__uint_as_float(u) + __uint_as_float(v[0][j]));
                  };
                  x = make_uint4(add(x.x, 4 * i), add(x.y, 4 * i + 1), add(x.z, 4 * i + 2), add(x.w, 4 * i + 3));
                }
                *p = x;
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&d_empty[d]);
        }
        if (!ok) break;
        if (!aligned) {
          // base and out in whole rows of the tile, element by element, all 32 rows' loads ahead
          // of the first store (4096 rows of 16 runs, 1024 -> 4099, rank 64: fp32 85 us, bf16
          // 71; with eight rows' loads ahead of their stores 110 and 79, with all of them ahead
          // of the products 137 and 71). The loop has one trip at most; without it the compiler
          // forms every row's address ahead of the loads (in turn, buffers in L2: fp32 84.2 us in
          // place of 77.8, bf16 62.6 and 60.4)
          __syncwarp();
          const uint32_t with = __ballot_sync(0xffffffffu, mine >= 0);
          const int rows = (int)min((int64_t)32, a.M - w0);
#pragma unroll 1
          for (int r0 = 0; r0 < rows; r0 += 32) {
            uint32_t x[32][kN / 32];
#pragma unroll
            for (int i = 0; i < 32; ++i)
#pragma unroll
              for (int j = 0; j < kN / 32; ++j) {
                const int n = c * kN + j * 32 + lane;
                x[i][j] = r0 + i < rows && n < a.N ? load_raw<kBf16>(a.base, (w0 + r0 + i) * a.ldb + n) : 0;
              }
#pragma unroll
            for (int i = 0; i < 32; ++i)
#pragma unroll
              for (int j = 0; j < kN / 32; ++j) {
                const int n = c * kN + j * 32 + lane;
                if (r0 + i >= rows || n >= a.N) continue;
                const bool has = with >> (r0 + i) & 1;
                if (has)
                  x[i][j] = add_raw<kBf16>(
                      x[i][j], __uint_as_float(stage[(quarter * 32 + r0 + i) * (kN + 1) + j * 32 + lane]));
                if (has || !keep) store_raw<kBf16>(a.out, (w0 + r0 + i) * a.ldo + n, x[i][j]);
              }
          }
          __syncwarp();
          continue;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (w0 < a.M) tma_store_2d(&tmOut, sx + s * C::kBase + quarter * 4096, c * kN, (int)w0);
          bulk_commit_group();
          // the slot before this one goes back when its store has read it
          asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          if (last >= 0) mbar_arrive(&base_empty[last]);
        }
        last = (int)s;
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1 && tmem_busy == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kSlots * kN);
  }
}

template <int RT>
static cudaError_t launch_shrink_many(const LoraArgs& a, bool x_bf16, uint32_t* err, cudaStream_t st) {
  if (x_bf16) {
    constexpr int RP = RT * 16;
    using C = ShrinkTc<RP>;
    static_assert(C::kSmem <= (RP == 128 ? 227 : 113) * 1024, "shared memory");
    CUtensorMap tx, ta;
    if (!make_tmap_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, a.K, a.M, a.ldx * 2, 64, 128,
                      CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tmap_3d(&ta, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.a, a.K, a.rank, a.count, (int64_t)a.K * 2,
                      (int64_t)a.rank * a.K * 2, 64, RP, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorNotSupported;
    auto kern = lora_shrink_tc_kernel<RP>;
    static std::atomic<uint64_t> attr_set{0};
    const cudaError_t e = smem_attr_once_per_device(kern, (int)C::kSmem, attr_set);
    if (e != cudaSuccess) return e;
    // with few rows several clusters share their adapters (129 rows of 64 adapters,
    // 5120 -> 5120, rank 16: the call 50 us, 187 with one cluster a tile; 300 rows of 11
    // runs, 5120 -> 17408, rank 64: 30, 43; of one adapter 20.4, 21)
    const int64_t tiles = ceil_div(a.M, 128);
    int64_t z = num_sms() * (RP == 128 ? 1 : 2) / (tiles * kManyParts);
    z = z < 1 ? 1 : z > 16 ? 16 : z;
    kern<<<dim3(kManyParts, (unsigned)tiles, (unsigned)z), 192, C::kSmem, st>>>(tx, ta, a, err);
    return cudaGetLastError();
  }
  const int64_t windows = ceil_div(a.M, 32);
  // with few windows several CTAs share the pieces of one
  int64_t z = 4 * num_sms() / (windows * kManyParts);
  z = z < 1 ? 1 : z > 32 ? 32 : z;
  auto kern = lora_shrink_f32_kernel<RT>;
  static std::atomic<uint64_t> attr_set{0};
  const cudaError_t e = smem_attr_once_per_device(kern, ManyCfg<RT>::kSmem, attr_set);
  if (e != cudaSuccess) return e;
  kern<<<dim3(kManyParts, (unsigned)windows, (unsigned)z), 32 * kManyWarps, ManyCfg<RT>::kSmem, st>>>(a);
  return cudaGetLastError();
}

template <bool kBf16, int kHalves>
static cudaError_t launch_expand_many(const LoraArgs& a, uint32_t* err, cudaStream_t st) {
  using C = ExpandMany<kBf16, kHalves>;
  static_assert(C::kSmem <= 227 * 1024 && C::kBaseRing * C::kBase >= 2 * 128 * (C::kN + 1) * 4, "shared memory per CTA");
  constexpr int es = kBf16 ? 2 : 4;
  const auto type = kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  auto at16 = [](const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * es)) % 16 == 0; };
  // (a TMA store clips a row at 16-byte granularity: where a row does not end on
  // such a boundary it would overwrite what lies behind it)
  const bool aligned = at16(a.base, a.ldb) && at16(a.out, a.ldo) && (int64_t)a.N * es % 16 == 0;
  CUtensorMap tx, tb, to, th;
  memset(&tx, 0, sizeof(tx));
  memset(&to, 0, sizeof(to));
  if ((aligned &&
       (!make_tmap_2d(&tx, type, a.base, a.N, a.M, a.ldb * es, C::kN, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tmap_2d(&to, type, a.out, a.N, a.M, a.ldo * es, C::kN, 32, CU_TENSOR_MAP_SWIZZLE_128B))) ||
      !make_tmap_3d(&tb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.b, a.rank, a.N, a.count, (int64_t)a.rank * 2,
                    (int64_t)a.N * a.rank * 2, 64, C::kN, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_3d(&th, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.parts, a.rp, a.M, C::kNumbers, (int64_t)a.rp * 2,
                    a.M * a.rp * 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorNotSupported;
  auto kern = lora_expand_many_kernel<kBf16, kHalves>;
  static std::atomic<uint64_t> attr_set{0};
  const cudaError_t e = smem_attr_once_per_device(kern, (int)C::kSmem, attr_set);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ceil_div(a.M, 128) * ceil_div(a.N, C::kN), ctas = tiles < num_sms() ? tiles : num_sms();
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  // (a change of rows costs about as much as two tiles)
  int64_t sections = tiles / (ctas * 12);
  sections = sections < 1 ? 1 : sections > 8 ? 8 : sections;
  const ExpandShares share{(int)sections, (uint32_t)(tiles / (ctas * sections)), (uint32_t)(tiles % (ctas * sections))};
  return launch_kernel(kern, dim3((unsigned)ctas), dim3(C::kThreads), C::kSmem, st, true, tx, tb, to, th, a,
                       (int)aligned, share, err);
}

template <bool kBf16, int C>
static cudaError_t launch_expand_few(const LoraArgs& a, uint32_t* err, cudaStream_t st) {
  const size_t smem = (size_t)(kExpandWarps * kExpandRing * 32 * C * 2 + kFewRows * 4) * a.rank;
  auto kern = lora_expand_few_kernel<kBf16, C>;
  static std::atomic<uint64_t> attr_set{0};
  const cudaError_t e = smem_attr_once_per_device(kern, (kExpandWarps * kExpandRing * 64 + kFewRows * 4) * 128, attr_set);
  if (e != cudaSuccess) return e;
  // fewer rows a CTA while all of them still run at once (GPU us of a call: 16 rows of 16
  // adapters, 17408 -> 5120, rank 16, eight a CTA 15.5, one 9.0; beyond that 16 rows, 5120
  // -> 17408, rank 32, two a CTA 13.1, four 11.5)
  const int64_t columns = ceil_div(a.N, kExpandWarps * 32 * C);
  const int64_t fit = num_sms() * (int64_t)(227 * 1024 / (smem + 2048));
  int group = kFewRows;
  while (group > 1 && columns * ceil_div(a.M, group / 2) <= fit) group /= 2;
  return launch_kernel(kern, dim3((unsigned)columns, (unsigned)ceil_div(a.M, group)), dim3(32 * kExpandWarps), smem, st,
                       true, a, group, err);
}

template <bool kBf16>
static cudaError_t launch_shrink_few(const LoraArgs& a, cudaStream_t st) {
  auto launch = [&](auto kern, int R) {
    const dim3 grid((unsigned)few_parts(a.K), (unsigned)a.M, (unsigned)ceil_div(a.rank, R * kFewWarps));
    kern<<<grid, 32 * kFewWarps, 0, st>>>(a);
  };
  // (two ranks a warp: the loads of four go out in two turns, 4 rows, 5120 -> 5120, rank
  // 64 11.3 us in place of 7.8)
  if (a.rank <= kFewWarps) launch(lora_shrink_few_kernel<kBf16, 1>, 1);
  else launch(lora_shrink_few_kernel<kBf16, 2>, 2);
  return cudaGetLastError();
}

static int64_t padded(int64_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// bytes of the parts' sums of M rows; with many rows, of up to three bf16 numbers of
// each sum before them (and never less than fewer rows need)
int64_t lora_workspace(int64_t M, int64_t K, int64_t rank) {
  const int64_t few = few_rows(rank), sums = few_parts((int)K) * (M < few ? M : few) * rank * 4;
  if (M <= few) return sums;
  const int64_t many = (kManyParts * 4 + 6) * M * padded(rank);
  return many > sums ? many : sums;
}

cudaError_t launch_add_lora(const void* base, bool bf16, int64_t ldb, const void* x, bool x_bf16, int64_t M,
                            int64_t K, int64_t ldx, const void* A, const void* B, int64_t count, int64_t rank,
                            int64_t N, const int64_t* ids, const float* scaling, void* out, int64_t ldo, void* ws,
                            uint32_t* err, cudaStream_t st) {
  LoraArgs a{x, reinterpret_cast<const uint16_t*>(A), reinterpret_cast<const uint16_t*>(B), ids, scaling, base,
             out, reinterpret_cast<float*>(ws), reinterpret_cast<uint32_t*>(ws), ldx, ldb, ldo, M, (int)K, (int)N,
             (int)rank, (int)count, (int)rank, 0};
  if (M <= few_rows(rank)) {
    const cudaError_t e = x_bf16 ? launch_shrink_few<true>(a, st) : launch_shrink_few<false>(a, st);
    if (e != cudaSuccess) return e;
    if (rank <= 32) return bf16 ? launch_expand_few<true, 2>(a, err, st) : launch_expand_few<false, 2>(a, err, st);
    return bf16 ? launch_expand_few<true, 1>(a, err, st) : launch_expand_few<false, 1>(a, err, st);
  }
  a.rp = (int)padded(rank);
  a.numbers = bf16 ? 2 : 3;
  a.h = reinterpret_cast<float*>(a.parts + a.numbers * M * (a.rp / 2));  // (behind the numbers)
  cudaError_t e = a.rp == 16   ? launch_shrink_many<1>(a, x_bf16, err, st)
                  : a.rp == 32 ? launch_shrink_many<2>(a, x_bf16, err, st)
                  : a.rp == 64 ? launch_shrink_many<4>(a, x_bf16, err, st)
                               : launch_shrink_many<8>(a, x_bf16, err, st);
  if (e != cudaSuccess) return e;
  if (!x_bf16)
    e = launch_kernel(lora_join_kernel, dim3((unsigned)ceil_div(M * (a.rp / 4), 256)), dim3(256), 0, st, true, a);
  if (e != cudaSuccess) return e;
  if (rank <= 64) return bf16 ? launch_expand_many<true, 1>(a, err, st) : launch_expand_many<false, 1>(a, err, st);
  return bf16 ? launch_expand_many<true, 2>(a, err, st) : launch_expand_many<false, 2>(a, err, st);
}

}  // namespace qg
