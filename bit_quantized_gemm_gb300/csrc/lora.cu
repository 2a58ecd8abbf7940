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
// Rows may come in any order. In a window of consecutive rows the different ids
// are found by votes, and the rows of each, wherever they lie in it, are one
// piece of work: rows of one request that follow one another cost one pass, the
// rows of 32 requests 32, which are dealt out over CTAs when there are few rows.
#include "qg_common.cuh"

namespace qg {

struct LoraArgs {
  const void* x;
  const uint16_t *a, *b;  // bf16 [count][rank][K], [count][N][rank]
  const int64_t* ids;
  const float* scaling;   // [count] or null
  const void* base;
  void* out;
  uint32_t* h;            // [M][2][padded rank / 2] pairs of bf16: of each row the large parts, the small parts
  int64_t ldx, ldb, ldo, M;
  int K, N, rank, count;
};

// D (16 x 8) += A (16 x 16) * B (16 x 8), bf16 operands, fp32 sums
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
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

// ---------------------------------------------------------------------- shrink
// K is cut into 64 shares, eight groups of eight. A share's sum is a chain of
// MMAs; the eight shares of a group are added in order, then the eight groups.
// Where shares lie on different warps or CTAs does not change that order, and it
// depends on K alone: a row's bits do not depend on the other rows of its call.
constexpr int kShares = 8, kGroups = 8;

// A's rows are the MMA's 16, NT times 8 rows of x its columns. A lane loads 8
// consecutive k of a row (16 bytes): they are k 8t.. of 32, t = lane % 4, of
// both operands, in whatever order the MMA sums them.
template <bool kBf16, int RT, int NT>
struct ShrinkStep {
  static constexpr int P = kBf16 ? 1 : 3;  // bf16 numbers a value of x: fp32 as the sum of three (24 bits)
  uint4 w[RT][2];
  uint4 x[NT][kBf16 ? 1 : 2];
  __device__ __forceinline__ void load(const uint16_t* pa, const char* const (&px)[NT], int k, int K, int rank) {
    const int g = (threadIdx.x & 31) >> 2;
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < (kBf16 ? 1 : 2); ++j)
        x[i][j] = k < K ? __ldg(reinterpret_cast<const uint4*>(px[i] + (int64_t)k * (kBf16 ? 2 : 4)) + j) : zero;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = r * 16 + h * 8 + g;
        w[r][h] = k < K && row < rank ? __ldg(reinterpret_cast<const uint4*>(pa + (int64_t)row * K + k)) : zero;
      }
  }
  __device__ __forceinline__ void multiply(float (&acc)[RT][NT][4]) const {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      uint32_t v[P][4];
      if (kBf16) {
        v[0][0] = x[i][0].x;
        v[0][1] = x[i][0].y;
        v[0][2] = x[i][0].z;
        v[0][3] = x[i][0].w;
      } else {
        const uint4 lo = x[i][0], hi = x[i][kBf16 ? 0 : 1];
        const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        float f[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) f[c] = __uint_as_float(u[c]);
#pragma unroll
        for (int q = 0; q < P; ++q)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t b = bf16x2(f[2 * c], f[2 * c + 1]);
            v[q][c] = b;
            // (an infinity's rest would be NaN)
            f[2 * c] = isfinite(bf16_lo(b)) ? f[2 * c] - bf16_lo(b) : 0.0f;
            f[2 * c + 1] = isfinite(bf16_hi(b)) ? f[2 * c + 1] - bf16_hi(b) : 0.0f;
          }
      }
#pragma unroll
      for (int q = 0; q < P; ++q)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const uint32_t f0[4] = {w[r][0].x, w[r][1].x, w[r][0].y, w[r][1].y};
          const uint32_t f1[4] = {w[r][0].z, w[r][1].z, w[r][0].w, w[r][1].w};
          mma_bf16_16816(acc[r][i], f0, v[q][0], v[q][1]);
          mma_bf16_16816(acc[r][i], f1, v[q][2], v[q][3]);
        }
    }
  }
};

template <int RT, int NT>
__device__ __forceinline__ void zero(float (&acc)[RT][NT][4]) {
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[r][i][c] = 0.0f;
}

// kU steps loaded before the first is worked on
template <bool kBf16, int RT, int NT, int kU>
__device__ __forceinline__ void add_share(float (&acc)[RT][NT][4], const LoraArgs& a, const uint16_t* pa,
                                          const char* const (&px)[NT], int share) {
  const int units = (a.K + 31) >> 5, t = threadIdx.x & 3;
  const int u0 = units * share / (kShares * kGroups), u1 = units * (share + 1) / (kShares * kGroups);
  for (int u = u0; u < u1; u += kU) {
    ShrinkStep<kBf16, RT, NT> s[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i)
      if (u + i < u1) s[i].load(pa, px, (u + i) * 32 + t * 8, a.K, a.rank);
#pragma unroll
    for (int i = 0; i < kU; ++i)
      if (u + i < u1) s[i].multiply(acc);
  }
}

// acc[r][i]: ranks 16r + g (c 0, 1) and + 8 (c 2, 3) of rows 8i + 2t and + 1
template <int RT, int NT>
__device__ __forceinline__ void put(float* part, const float (&acc)[RT][NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        part[(8 * i + 2 * t + (c & 1)) * (RT * 16 + 4) + r * 16 + g + 8 * (c >> 1)] = acc[r][i][c];
}

// ranks r and r + 1 of a row's sum v, scaled, as two bf16 numbers each
__device__ __forceinline__ void put_h(const LoraArgs& a, int64_t m, int rp, int r, float scale, float v0, float v1) {
  // (ranks that only pad: 0, also where x is infinite)
  v0 = r < a.rank ? v0 * scale : 0.0f;
  v1 = r < a.rank ? v1 * scale : 0.0f;
  const uint32_t hi = bf16x2(v0, v1);
  const uint32_t lo = bf16x2(isfinite(bf16_lo(hi)) ? v0 - bf16_lo(hi) : 0.0f,
                             isfinite(bf16_hi(hi)) ? v1 - bf16_hi(hi) : 0.0f);
  uint32_t* h = a.h + m * rp + r / 2;
  h[0] = hi;
  h[rp / 2] = lo;
}

// The groups' sums of a piece's rows, added in order by the cluster's threads
template <int RP>
__device__ __forceinline__ void join_groups(const LoraArgs& a, const float* sum, int64_t m0, int id, uint32_t rows,
                                            int rank) {
  const int count = __popc(rows);
  const float scale = a.scaling ? __ldg(a.scaling + id) : 1.0f;
  for (int e = ((int)threadIdx.x * kGroups + rank) * 2; e < count * RP; e += 2 * (int)blockDim.x * kGroups) {
    float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
    for (int c = 0; c < kGroups; ++c) {
      const uint32_t p = map_to_cta(sum + e, c);
      v0 += ld_cluster_f32(p);
      v1 += ld_cluster_f32(p + 4);
    }
    put_h(a, m0 + nth_bit(rows, e / RP), RP, e % RP, scale, v0, v1);
  }
}

// Few rows: windows of 8 rows; a cluster of eight CTAs, one a group of K, one
// warp a share. gridDim.z CTAs share a window's pieces.
template <bool kBf16, int RT>
__global__ void __cluster_dims__(kGroups, 1, 1) __launch_bounds__(32 * kShares)
    lora_shrink_few_kernel(const LoraArgs a) {
  griddep_launch_dependents();
  constexpr int RP = RT * 16, kPitch = RP + 4;
  __shared__ float part[kShares][8 * kPitch], sum[8 * RP];
  const int warp = threadIdx.x >> 5, g = (threadIdx.x & 31) >> 2;
  const uint32_t rank = cluster_ctarank();
  const int64_t m0 = (int64_t)blockIdx.y * 8;
  LoraPieces pieces(a, m0, 8);
  int id, j = 0;
  uint32_t rows;
  while (pieces.next(j, blockIdx.z, gridDim.z, id, rows)) {
    if (id < 0) continue;
    const int count = __popc(rows);
    // this lane's row of x, the g-th (past the last: the last)
    const char* px[1] = {reinterpret_cast<const char*>(a.x) +
                         (m0 + nth_bit(rows, min(g, count - 1))) * a.ldx * (kBf16 ? 2 : 4)};
    float acc[RT][1][4];
    zero(acc);
    add_share<kBf16, RT, 1, RT == 1 ? 5 : RT == 2 ? 3 : RT == 4 ? 2 : 1>(
        acc, a, a.a + (int64_t)id * a.rank * a.K, px, (int)rank * kShares + warp);
    put(part[warp], acc);
    __syncthreads();
    for (int e = threadIdx.x; e < count * RP; e += 32 * kShares) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kShares; ++w) s += part[w][e / RP * kPitch + e % RP];
      sum[e] = s;
    }
    cluster_sync();
    join_groups<RP>(a, sum, m0, id, rows, (int)rank);
    cluster_sync();  // the sums have been read
  }
}

// asynchronous 16-byte global -> shared copy; `in` false: zeros
__device__ __forceinline__ void cp_async_16(void* to, const void* from, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(in ? 16 : 0)
               : "memory");
}

// Many rows: windows of 32; a cluster of eight CTAs, one a group of K, that
// brings its steps of K (32 values of every row of x and of A) through a ring in
// shared memory; warp w multiplies rows 8w.. of the piece. A step's rows lie 64
// bytes apart (x in fp32: 128), which a lane's 16-byte reads of row lane / 4,
// piece lane % 4, take without conflicts. Two steps are fetched at once, whole
// 128-byte lines.
constexpr int kManyWarps = 4, kManyRing = 4;
template <bool kBf16, int RT>
struct ManyCfg {
  static constexpr int kX = 32 * (kBf16 ? 64 : 128), kA = RT * 16 * 64, kStep = kX + kA;
  static constexpr int kSum = 32 * RT * 16 * 4;
  static constexpr int kSmem = kManyRing * 2 * kStep + kSum;
};

template <bool kBf16, int RT>
__global__ void __cluster_dims__(kGroups, 1, 1) __launch_bounds__(32 * kManyWarps)
    lora_shrink_many_kernel(const LoraArgs a) {
  griddep_launch_dependents();
  using C = ManyCfg<kBf16, RT>;
  constexpr int RP = RT * 16, kThreads = 32 * kManyWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  float* const sum = reinterpret_cast<float*>(smem + kManyRing * 2 * C::kStep);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t rank = cluster_ctarank();
  const int64_t m0 = (int64_t)blockIdx.y * 32;
  const int units = (a.K + 31) >> 5;
  const int u0 = units * (int)rank / kGroups, u1 = units * ((int)rank + 1) / kGroups;  // this group's steps
  LoraPieces pieces(a, m0, 32);
  int id, j = 0;
  uint32_t rows;
  while (pieces.next(j, blockIdx.z, gridDim.z, id, rows)) {
    if (id < 0) continue;
    const int count = __popc(rows);
    const uint16_t* pa = a.a + (int64_t)id * a.rank * a.K;
    // x: four threads a row (eight of fp32), 32 or 16 rows a round
    constexpr int kPer = kBf16 ? 4 : 8, kRounds = 32 * kPer / kThreads;
    const char* px[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      px[i] = reinterpret_cast<const char*>(a.x) +
              (m0 + nth_bit(rows, min(i * (kThreads / kPer) + (int)threadIdx.x / kPer, count - 1))) * a.ldx *
                  (kBf16 ? 2 : 4);
    auto fetch = [&](int u) {  // steps u and u + 1
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        uint8_t* to = smem + (((u - u0) / 2 % kManyRing) * 2 + d) * C::kStep;
        const bool in = u + d < u1;
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
          const int c = threadIdx.x % kPer, row = i * (kThreads / kPer) + (int)threadIdx.x / kPer;
          const int k = (u + d) * 32 + c * (kBf16 ? 8 : 4);
          const bool ok = in && row < count && k < a.K;
          cp_async_16(to + row * (kBf16 ? 64 : 128) + c * 16, px[i] + (ok ? (int64_t)k * (kBf16 ? 2 : 4) : 0), ok);
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
    float group[RT][1][4], acc[RT][1][4];
    zero(group);
    zero(acc);
    int share = (int)rank * kShares;
    int end = units * (share + 1) / (kShares * kGroups);  // of the share
    auto fold = [&](int u) {                              // shares that end at step u
      while (u == end && share < ((int)rank + 1) * kShares) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            group[r][0][c] += acc[r][0][c];
            acc[r][0][c] = 0.0f;
          }
        ++share;
        end = units * (share + 1) / (kShares * kGroups);
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
          ShrinkStep<kBf16, RT, 1> s;
          const uint8_t* fx = from + (warp * 8 + g) * (kBf16 ? 64 : 128) + t * (kBf16 ? 16 : 32);
#pragma unroll
          for (int i = 0; i < (kBf16 ? 1 : 2); ++i) s.x[0][i] = *(reinterpret_cast<const uint4*>(fx) + i);
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
    if (warp * 8 < count) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sum[(warp * 8 + 2 * t + (c & 1)) * RP + r * 16 + g + 8 * (c >> 1)] = group[r][0][c];
    }
    cluster_sync();
    join_groups<RP>(a, sum, m0, id, rows, (int)rank);
    cluster_sync();  // the sums have been read
  }
}

// ---------------------------------------------------------------------- expand
constexpr int kExpandWarps = 4, kExpandCols = 64;

// eight consecutive columns of a row of base or out, as they lie in memory
template <bool kBf16>
struct Cols8 {
  static constexpr int kWords = kBf16 ? 4 : 8, kEs = kBf16 ? 2 : 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const char* p, int n, bool vec) {  // n of them
    if (vec && n >= 8) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = *(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if (kBf16)
          w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
        else
          w[i % kWords] = reinterpret_cast<const uint32_t*>(p)[i];
      }
  }
  __device__ __forceinline__ void add(int i, float y0, float y1) {  // to columns 2i and 2i + 1
    if (kBf16) {
      w[i] = bf16x2(bf16_lo(w[i]) + y0, bf16_hi(w[i]) + y1);
    } else {
      w[2 * i % kWords] = __float_as_uint(__uint_as_float(w[2 * i % kWords]) + y0);
      w[(2 * i + 1) % kWords] = __float_as_uint(__uint_as_float(w[(2 * i + 1) % kWords]) + y1);
    }
  }
  __device__ __forceinline__ void store(char* p, int n, bool vec) const {
    if (vec && n >= 8) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i)
        *(reinterpret_cast<uint4*>(p) + i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if (kBf16)
          reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
        else
          reinterpret_cast<uint32_t*>(p)[i] = w[i % kWords];
      }
  }
};

// A warp adds to kCols columns of a piece's rows, 16 rows an MMA. The MMA's
// columns are dealt out so that a lane's outputs of four MMAs are 8 consecutive
// columns of two rows: column 2t + i of MMA j is column 8t + 2j + i of 32. Ranks
// likewise: a lane's are 8t.. of 32 (two MMAs; 4t.. of 16 for ranks up to 16), so
// that it reads both operands in 16 bytes. A warp's part of B stays in registers
// from piece to piece while the id is the same; where it is small, the next
// piece's is on its way. Windows of 32 rows; a CTA takes `windows` of them,
// gridDim.z CTAs share a window's pieces.
template <bool kBf16, int RT>
struct ExpandCfg {
  static constexpr int kCols = RT == 8 || (RT == 4 && !kBf16) ? 32 : 64;
  static constexpr bool kAhead = RT <= 2;
  static constexpr int kQuads = kCols / 32, kPairs = RT == 1 ? 1 : RT / 2, kWords = RT == 1 ? 2 : 4;
};

template <bool kBf16, int RT>
struct ExpandB {
  using C = ExpandCfg<kBf16, RT>;
  uint32_t w[C::kQuads][4][C::kPairs][C::kWords];
  __device__ __forceinline__ void load(const LoraArgs& a, int id, int col0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint16_t* pb = a.b + (int64_t)id * a.N * a.rank;
#pragma unroll
    for (int q = 0; q < C::kQuads; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = col0 + q * 32 + 8 * (g >> 1) + 2 * i + (g & 1);
#pragma unroll
        for (int p = 0; p < C::kPairs; ++p) {
          const int r = p * 32 + t * (RT == 1 ? 4 : 8);
          const bool in = n < a.N && r < a.rank;
          const uint16_t* from = pb + (int64_t)n * a.rank + r;
          if constexpr (RT == 1) {
            const uint2 v = in ? __ldg(reinterpret_cast<const uint2*>(from)) : make_uint2(0, 0);
            w[q][i][p][0] = v.x;
            w[q][i][p][1] = v.y;
          } else {
            const uint4 v = in ? __ldg(reinterpret_cast<const uint4*>(from)) : make_uint4(0, 0, 0, 0);
            w[q][i][p][0] = v.x;
            w[q][i][p][1] = v.y;
            w[q][i][p][2] = v.z;
            w[q][i][p][3] = v.w;
          }
        }
      }
  }
};

// a lane's ranks of a row of h
template <int kWords>
__device__ __forceinline__ void load_h(const uint32_t* p, bool in, uint32_t (&v)[kWords]) {
  if constexpr (kWords == 2) {
    const uint2 x = in ? *reinterpret_cast<const uint2*>(p) : make_uint2(0, 0);
    v[0] = x.x;
    v[1] = x.y;
  } else {
    const uint4 x = in ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
    v[0] = x.x;
    v[1] = x.y;
    v[2] = x.z;
    v[3] = x.w;
  }
}

template <bool kBf16, int RT>
__global__ void __launch_bounds__(32 * kExpandWarps) lora_expand_kernel(const LoraArgs a, const int vec,
                                                                        const int windows) {
  using C = ExpandCfg<kBf16, RT>;
  constexpr int RP = RT * 16, kEs = kBf16 ? 2 : 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int col0 = ((int)blockIdx.x * kExpandWarps + warp) * C::kCols;
  const bool keep = a.base == a.out && a.ldb == a.ldo;  // rows without an adapter are in place
  bool waited = false;
  if (col0 < a.N) {
    int64_t m0 = (int64_t)blockIdx.y * windows * 32;
    const int64_t end = min(m0 + (int64_t)windows * 32, a.M);
    LoraPieces pieces(a, m0, 32);
    int number = 0;
    // the next piece, of this window or a later one
    auto advance = [&](int64_t& m, int& id, uint32_t& rows) {
      for (;;) {
        while (pieces.next(number, blockIdx.z, gridDim.z, id, rows))
          if (id >= 0 || !keep) {
            m = m0;
            return true;
          }
        m0 += 32;
        if (m0 >= end) return false;
        pieces = LoraPieces(a, m0, 32);
        number = 0;
      }
    };
    int id, id_next, held = -1;
    int64_t m, m_next;
    uint32_t rows, rows_next;
    ExpandB<kBf16, RT> b, b_next;
    bool more = advance(m, id, rows);
    if (more && id >= 0) {
      b.load(a, id, col0);
      held = id;
    }
    while (more) {
      more = advance(m_next, id_next, rows_next);
      if (C::kAhead && more && id_next >= 0 && id_next != held) b_next.load(a, id_next, col0);
      const int count = __popc(rows);
#pragma unroll
      for (int tile = 0; tile < 2; ++tile) {
        if (16 * tile >= count) break;
        int row[2];  // this lane's rows of the piece: numbers g and g + 8 of the tile
        Cols8<kBf16> raw[C::kQuads][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = 16 * tile + g + 8 * h;
          row[h] = n < count ? nth_bit(rows, n) : -1;
#pragma unroll
          for (int q = 0; q < C::kQuads; ++q) {
            const int n0 = col0 + q * 32 + 8 * t;
            if (row[h] >= 0)
              raw[q][h].load(reinterpret_cast<const char*>(a.base) + ((m + row[h]) * a.ldb + n0) * kEs, a.N - n0, vec);
          }
        }
        if (!waited) {  // (nothing above is shrink's work; out may be what a kernel before it reads)
          griddep_wait();
          waited = true;
        }
        if (id >= 0) {  // (a row without an adapter keeps base's bits)
          float acc[C::kQuads][4][4];
#pragma unroll
          for (int q = 0; q < C::kQuads; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int c = 0; c < 4; ++c) acc[q][i][c] = 0.0f;
#pragma unroll
          for (int p = 0; p < C::kPairs; ++p) {
            uint32_t h[2][2][C::kWords];  // [large, small parts][row]
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t* ph = a.h + (m + row[i]) * RP + (p * 32 + t * 2 * C::kWords) / 2;
              load_h(ph, row[i] >= 0, h[0][i]);
              load_h(ph + RP / 2, row[i] >= 0, h[1][i]);
            }
#pragma unroll
            for (int k = 0; k < C::kWords / 2; ++k)
#pragma unroll
              for (int o = 1; o >= 0; --o) {
                const uint32_t f[4] = {h[o][0][2 * k], h[o][1][2 * k], h[o][0][2 * k + 1], h[o][1][2 * k + 1]};
#pragma unroll
                for (int q = 0; q < C::kQuads; ++q)
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    mma_bf16_16816(acc[q][i], f, b.w[q][i][p][2 * k], b.w[q][i][p][2 * k + 1]);
              }
          }
#pragma unroll
          for (int q = 0; q < C::kQuads; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 4; ++i) raw[q][h].add(i, acc[q][i][2 * h], acc[q][i][2 * h + 1]);
        }
#pragma unroll
        for (int q = 0; q < C::kQuads; ++q)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int n0 = col0 + q * 32 + 8 * t;
            if (row[h] >= 0)
              raw[q][h].store(reinterpret_cast<char*>(a.out) + ((m + row[h]) * a.ldo + n0) * kEs, a.N - n0, vec);
          }
      }
      if (more && id_next >= 0 && id_next != held) {
        if (C::kAhead) b = b_next;
        else b.load(a, id_next, col0);
        held = id_next;
      }
      id = id_next;
      m = m_next;
      rows = rows_next;
    }
  }
  // (this kernel's end stands for shrink's, too)
  if (!waited) griddep_wait();
}

template <bool kBf16, int RT>
static cudaError_t launch_shrink(const LoraArgs& a, cudaStream_t st) {
  if (a.M > 128) {
    const int64_t windows = ceil_div(a.M, 32);
    // with few windows several clusters share the pieces of one
    int64_t z = 4 * num_sms() / (windows * kGroups);
    z = z < 1 ? 1 : z > 32 ? 32 : z;
    auto kern = lora_shrink_many_kernel<kBf16, RT>;
    static std::atomic<uint64_t> attr_set{0};
    const cudaError_t e = smem_attr_once_per_device(kern, ManyCfg<kBf16, RT>::kSmem, attr_set);
    if (e != cudaSuccess) return e;
    kern<<<dim3(kGroups, (unsigned)windows, (unsigned)z), 32 * kManyWarps, ManyCfg<kBf16, RT>::kSmem, st>>>(a);
    return cudaGetLastError();
  }
  const int windows = (int)ceil_div(a.M, 8), most = a.M < 8 ? (int)a.M : 8;
  lora_shrink_few_kernel<kBf16, RT><<<dim3(kGroups, windows, most), 32 * kShares, 0, st>>>(a);
  return cudaGetLastError();
}

template <bool kXBf16, bool kBf16, int RT>
static cudaError_t launch_lora(const LoraArgs& a, cudaStream_t st) {
  const cudaError_t e = launch_shrink<kXBf16, RT>(a, st);
  if (e != cudaSuccess) return e;
  constexpr int es = kBf16 ? 2 : 4;
  auto at16 = [](const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * es)) % 16 == 0; };
  const int vec = at16(a.base, a.ldb) && at16(a.out, a.ldo);
  const int64_t gx = ceil_div(a.N, ExpandCfg<kBf16, RT>::kCols * kExpandWarps), all = ceil_div(a.M, 32);
  // four windows to a CTA where that leaves enough CTAs (they read the same rows
  // of B); with few windows their pieces are dealt out
  const int windows = gx * all >= 32 * num_sms() ? 4 : 1;
  const int64_t gy = ceil_div(all, windows);
  int64_t gz = 4 * num_sms() / (gx * gy);
  gz = gz < 1 ? 1 : gz > 32 ? 32 : gz;
  gz = gz < a.M ? gz : a.M;
  return launch_kernel(lora_expand_kernel<kBf16, RT>, dim3((unsigned)gx, (unsigned)gy, (unsigned)gz),
                       dim3(32 * kExpandWarps), 0, st, true, a, vec, windows);
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
  const LoraArgs a{x, reinterpret_cast<const uint16_t*>(A), reinterpret_cast<const uint16_t*>(B), ids, scaling, base,
                   out, reinterpret_cast<uint32_t*>(ws), ldx, ldb, ldo, M, (int)K, (int)N, (int)rank, (int)count};
  if (x_bf16) return bf16 ? launch_lora_any<true, true>(a, st) : launch_lora_any<true, false>(a, st);
  return bf16 ? launch_lora_any<false, true>(a, st) : launch_lora_any<false, false>(a, st);
}

}  // namespace qg
