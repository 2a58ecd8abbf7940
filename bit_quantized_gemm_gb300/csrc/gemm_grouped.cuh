// gemm_grouped.cuh -- the tiles of a product grouped by expert, found on the device.
#pragma once

#include "qg_common.cuh"

namespace qg {

// Expert e owns rows first[e] up to first[e + 1] (the offsets, those outside 0..M
// taken as 0 or M; an expert that ends before it begins has none). It has ceil(rows
// / T) tiles of T rows (before[e] of them lie ahead of its own) times NT tiles of
// weight rows, the rows' tiles of one weight tile after one another: weights come
// from HBM once.
struct GroupedTiles {
  const int *first, *before;  // [E + 1] each, in shared memory
  int E, NT;
  // bytes of the two lists
  static __host__ __device__ constexpr int bytes(int E) { return 2 * (E + 1) * 4; }
  // filled by one warp, 128 experts' offsets a trip to memory (8 rows of 64 experts, 2560
  // -> 2432: 11.8 us; 32 a trip 12.4)
  static __device__ void fill(const int64_t* offsets, int E, int M, int T, int* first, int* before) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int e0 = 0; e0 <= E; e0 += 128) {
      auto row = [&](int i) { return (int)min(max(__ldg(offsets + min(i, E)), (int64_t)0), (int64_t)M); };
      int lo[4], hi[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo[j] = row(e0 + 32 * j + lane);
        hi[j] = row(e0 + 32 * j + lane + 1);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = e0 + 32 * j + lane, n = e < E ? max(hi[j] - lo[j], 0) : 0;
        const int t = (n + T - 1) / T;
        int s = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, s, o);
          if (lane >= o) s += v;
        }
        if (e <= E) {
          first[e] = lo[j];
          before[e] = base + s - t;
        }
        base += __shfl_sync(0xffffffffu, s, 31);
      }
    }
  }
  // (ascending offsets have less than 2^30 tiles in any memory; others may claim rows
  // hundreds of times over, and their tiles' numbers must not pass 2^31)
  __device__ int total() const { return (int)min((int64_t)before[E] * NT, (int64_t)1 << 30); }
  // the expert of tile t, the number of its tile of rows and of weight rows; by a
  // whole warp (a 32-way search)
  __device__ void at(int t, int& e, int& mi, int& ni) const {
    const int lane = threadIdx.x & 31, row = t / NT;  // row: the tiles of rows, counted over the experts
    int lo = 0;
    for (int span = 1024; span > 1; span >>= 5) {
      const int i = min(lo + lane * (span >> 5), E);
      lo += (__popc(__ballot_sync(0xffffffffu, before[i] <= row)) - 1) * (span >> 5);
      lo = min(lo, E - 1);
    }
    e = lo;
    const int k = before[e + 1] - before[e], idx = t - before[e] * NT;
    ni = idx / k;
    mi = idx - ni * k;
  }
};

}  // namespace qg
