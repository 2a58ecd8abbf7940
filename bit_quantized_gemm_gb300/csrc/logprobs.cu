// logprobs.cu -- log probabilities of given tokens, entropy and the largest
// alternatives of each row of logits.
//
// With m = max x, S = sum e^(x-m), T = sum e^(x-m) (x-m) over a row of V:
//   log p[i] = x[i] - m - log S,   H = -sum p log p = log S - T / S
// (both terms of H are >= 0: nothing cancels). The alternatives are the first
// `top` values in the order (value descending, index ascending). Statistics
// are held in fp32 relative to a running maximum: a thread adds up the terms of a
// chunk, the sums of up to 32 chunks, and these in a compensated sum, so that log S
// is off by no more than 2e-5 at any V (one chain of 4096 terms: 1.2e-4).
// The order of a row's sums depends on its pieces, so on the number of rows, and on
// its address modulo 16: so do its last bits. The alternatives' order is exact.
//
// Rows without a distribution: -inf everywhere (a mask that leaves nothing)
// gives log p = -inf, H = 0 and no alternatives (index -1, -inf); a row with a
// NaN or +inf gives NaN and no alternatives (index -1, NaN): either makes S a
// NaN, which is how it is told. An alternative of -inf is none: its index is
// -1. An id below 0 asks for nothing and gives 0; an id >= V gives NaN.
//
// Bound by reading the logits once: 2 (bf16) or 4 bytes a value. The rows are
// cut into `splits` pieces where there are too few of them for the SMs; a CTA
// reads its piece in chunks of 128 threads x 64 bytes, the next chunk in
// flight, and each thread keeps (m, S, T) of its own values. For the
// alternatives a CTA keeps its `top` best so far as 64-bit keys (value, then
// inverted index) and only looks at values above the last of them: the first
// chunk, where a threshold comes from the warps' maxima, is ranked at once, and
// from then on the few values that pass (about `top` for each doubling of the
// length) are collected without a barrier and ranked after 2, 4, 8, ... chunks.
// The pieces of a row are a cluster of CTAs, whose first one joins them.
//
// Measured (GB300, bf16, from a CUDA graph): 4096 x 131072 without alternatives
// 164-168 us, 6.4-6.5 TB/s (a copy: 6.69); with 1, 5, 20, 32 alternatives 182, 200,
// 243, 275 us: bound by issued instructions there (73 % of the slots; 8.7 a value
// without alternatives, 10.9 with five). 2048 x 131072 fp32, 5 alternatives 169 us; 1 x
// 131072 4.2 us, with 5 8.7, with 20 10.3.
#include <math_constants.h>

#include "qg_common.cuh"

namespace qg {

// Small CTAs, eight on an SM: one's barriers hide behind the others (4096 x 131072
// bf16, no alternatives, when it took 167 us: 175 with 256 threads, 209 with 512).
constexpr int kLpThreads = 128, kLpWarps = kLpThreads / 32, kLpCtas = 8;
constexpr int kLpVecs = 4;                   // 16-byte loads per thread and chunk
constexpr int kLpCap = 512;                  // candidates that are ranked at once
constexpr int kLpTop = QG_LOGPROBS_MAX_TOP;
constexpr int kLpFold = 32;                  // chunks whose sums are added in plain fp32
constexpr int kLpMaxSplits = 16;             // CTAs of a cluster
static_assert(kLpTop <= 32 && kLpTop % kLpWarps == 0, "a lane per alternative");

struct LpArgs {
  const void* logits;
  int64_t V, ldl;
  const int64_t* ids;
  float* logprobs;
  float* entropy;
  int64_t* top_ids;
  float* top_logprobs;
  int G, top, splits;
};

// Order of the alternatives as an unsigned key: larger value first (both zeros
// are equal), then smaller index. 0 is below every value.
__device__ __forceinline__ uint64_t lp_key(float x, uint32_t i) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  const uint32_t o = (u >> 31) ? ~u : u | 0x80000000u;
  return (uint64_t)o << 32 | (uint32_t)~i;
}
__device__ __forceinline__ float lp_value(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float((o >> 31) ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t warp_max_u64(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (uint64_t)hi << 32 | lo;
}

// (m, S, T) of two sets of values as one
__device__ __forceinline__ void lp_join(float& m, float& S, float& T, float m2, float S2, float T2) {
  const float mm = fmaxf(m, m2);
  // S = 0 marks an empty set (m = -inf); a NaN in S stays. A difference below
  // -200 (or one that overflows) stands for a factor of 0.
  const float c1 = S == 0.0f ? 0.0f : __expf(m - mm), c2 = S2 == 0.0f ? 0.0f : __expf(m2 - mm);
  const float d1 = S == 0.0f ? 0.0f : fmaxf(m - mm, -200.0f), d2 = S2 == 0.0f ? 0.0f : fmaxf(m2 - mm, -200.0f);
  T = c1 * fmaf(S, d1, T) + c2 * fmaf(S2, d2, T2);
  S = c1 * S + c2 * S2;
  m = mm;
}
__device__ __forceinline__ void lp_join_warp(float& m, float& S, float& T) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), S2 = __shfl_xor_sync(0xffffffffu, S, o),
                T2 = __shfl_xor_sync(0xffffffffu, T, o);
    lp_join(m, S, T, m2, S2, T2);
  }
}

// a + b with the rounding error of the sum added to `lost`
__device__ __forceinline__ float add_exact(float a, float b, float& lost) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  lost += __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
  return s;
}

// Adds the sums of kLpFold chunks (relative to m, the thread's maximum so far) to
// the thread's sums. These follow the maximum only once it is one above their
// reference, so that many small rises do not scale them, and round them, many
// times: the factors shrink what the earlier ones rounded. (Shared memory and a
// call of its own: rare, and the loop has no register to spare.)
__device__ __noinline__ void lp_fold(float (*fold)[kLpThreads], float m, float S, float T) {
  if (S == 0.0f) return;  // only -inf so far
  float* f = &fold[0][threadIdx.x];
  float ref = f[0], s = f[kLpThreads], s_lost = f[2 * kLpThreads], t = f[3 * kLpThreads], t_lost = f[4 * kLpThreads];
  if (!(m <= ref + 1.0f)) {
    const float c = __expf(ref - m), d = fmaxf(ref - m, -200.0f);  // c = 0 at first
    t = c * fmaf(s, d, t);
    t_lost = c * fmaf(s_lost, d, t_lost);
    s *= c;
    s_lost *= c;
    ref = m;
  } else {
    const float d = m - ref, c = __expf(d);
    T = c * fmaf(S, d, T);
    S *= c;
  }
  f[0] = ref;
  f[kLpThreads] = add_exact(s, S, s_lost);
  f[2 * kLpThreads] = s_lost;
  f[3 * kLpThreads] = add_exact(t, T, t_lost);
  f[4 * kLpThreads] = t_lost;
}

template <bool kBf16>
__device__ __forceinline__ float lp_load(const void* row, int64_t i) {
  if (kBf16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
  return reinterpret_cast<const float*>(row)[i];
}

// One row's outputs from its statistics and its keys (descending, 0: none), by
// the whole CTA: the given tokens, the entropy and the alternatives by warps of
// their own (each part is short and waits mostly for its own instructions).
// id0, x0: the thread's first given id and its logit, loaded ahead.
template <bool kBf16>
__device__ __forceinline__ void lp_outputs(const LpArgs& a, int64_t m, const void* row, float mx, float S,
                                           float T, const uint64_t* keys, int64_t id0, float x0) {
  const int tid = threadIdx.x;
  const bool empty = mx == -CUDART_INF_F && S == 0.0f, bad = !(S == S);
  const float shift = empty ? 0.0f : mx, lse = empty ? 0.0f : logf(S);
  auto logp = [&](float x) {
    if (bad) return CUDART_NAN_F;
    return x == -CUDART_INF_F ? x : (x - shift) - lse;
  };
  if (tid == kLpThreads - 33 && a.entropy)
    a.entropy[m] = bad ? CUDART_NAN_F : empty ? 0.0f : lse - T / S;
  for (int g = tid; g < a.G; g += kLpThreads) {
    const int64_t id = g == tid ? id0 : a.ids[m * a.G + g];
    const float x = g == tid || id < 0 || id >= a.V ? x0 : lp_load<kBf16>(row, id);
    a.logprobs[m * a.G + g] = id < 0 ? 0.0f : id >= a.V ? CUDART_NAN_F : logp(x);
  }
  const int t = tid - (kLpThreads - 32);  // the last warp
  if (t >= 0 && t < a.top) {
    const uint64_t k = keys[t];
    const bool none = bad || k == 0;
    a.top_ids[m * a.top + t] = none ? -1 : (int64_t)(uint32_t)~(uint32_t)k;
    a.top_logprobs[m * a.top + t] = logp(k == 0 ? -CUDART_INF_F : lp_value(k));
  }
}

template <bool kBf16>
struct LpChunk {
  static constexpr int kVec = kBf16 ? 8 : 4;           // values per 16-byte load
  static constexpr int kPer = kLpVecs * kVec;          // values per thread
  uint4 v[kLpVecs];

  static __device__ __forceinline__ float value(const uint4& q, int j) {  // value j (a constant) of a load
    if (kBf16) {
      const uint32_t w = j < 2 ? q.x : j < 4 ? q.y : j < 6 ? q.z : q.w;
      return __uint_as_float((j & 1) ? w & 0xFFFF0000u : w << 16);
    }
    return __uint_as_float(j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w);
  }
  __device__ __forceinline__ float at(int i) const { return value(v[i / kVec], i % kVec); }
  static __device__ __forceinline__ float max_of(const uint4& q) {  // largest value, NaNs aside
    if (kBf16) {
      const __nv_bfloat162 a = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&q.x),
                                       *reinterpret_cast<const __nv_bfloat162*>(&q.y));
      const __nv_bfloat162 b = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&q.z),
                                       *reinterpret_cast<const __nv_bfloat162*>(&q.w));
      const __nv_bfloat162 m = __hmax2(a, b);
      return fmaxf(__low2float(m), __high2float(m));
    }
    return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)),
                 fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
  }
  static constexpr uint32_t kNone = kBf16 ? 0xFF80FF80u : 0xFF800000u;  // -inf
  // the thread's vectors of a chunk of n (whole: n = 4 * 128)
  __device__ __forceinline__ void load(const uint4* chunk, int n) {
    if (n >= kLpVecs * kLpThreads) {
#pragma unroll
      for (int i = 0; i < kLpVecs; ++i) v[i] = __ldcs(chunk + i * kLpThreads + threadIdx.x);
    } else {
#pragma unroll
      for (int i = 0; i < kLpVecs; ++i) {
        const int q = i * kLpThreads + threadIdx.x;
        v[i] = q < n ? __ldcs(chunk + q) : make_uint4(kNone, kNone, kNone, kNone);
      }
    }
  }
  // one value, or none
  __device__ __forceinline__ void load_one(const void* row, int64_t e, bool valid) {
#pragma unroll
    for (int i = 0; i < kLpVecs; ++i) v[i] = make_uint4(kNone, kNone, kNone, kNone);
    if (!valid) return;
    if (kBf16) v[0].x = (kNone & 0xFFFF0000u) | reinterpret_cast<const uint16_t*>(row)[e];
    else v[0].x = reinterpret_cast<const uint32_t*>(row)[e];
  }
  // largest value (NaNs aside)
  __device__ __forceinline__ float max() const {
    if (kBf16) {
      __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&v[0].x);
#pragma unroll
      for (int i = 0; i < kLpVecs; ++i) {
        m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&v[i].x));
        m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&v[i].y));
        m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&v[i].z));
        m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&v[i].w));
      }
      return fmaxf(__low2float(m), __high2float(m));
    }
    float m = at(0);
#pragma unroll
    for (int i = 1; i < kPer; ++i) m = fmaxf(m, at(i));
    return m;
  }
};

struct LpShared {
  uint4 own[kLpVecs][kLpThreads];  // values of the threads that have candidates
  uint64_t cand[kLpCap];           // candidates
  uint64_t list[2][kLpTop];        // the best so far, descending, 0: none; the other one is 0
  uint64_t red[kLpWarps];
  float wm[kLpWarps], wS[kLpWarps], wT[kLpWarps];
  int count[2];                    // candidates, also those past the buffer's end
  // a thread's sums of whole groups of chunks: their reference, then S and T, each
  // with what its roundings lost
  float fold[5][kLpThreads];
  uint64_t final_list[kLpTop];     // what the row's first CTA reads of a piece
  float stats[3];
};

// value i of the thread, from S.own, and its row index (i0: that of value 0)
template <bool kBf16>
__device__ __forceinline__ float lp_own(const LpShared& S, int i) {
  return lp_load<kBf16>(&S.own[i / LpChunk<kBf16>::kVec][threadIdx.x], i % LpChunk<kBf16>::kVec);
}
template <bool kBf16>
__device__ __forceinline__ uint32_t lp_index(uint32_t i0, int i) {
  constexpr int kVec = LpChunk<kBf16>::kVec;
  return i0 + (uint32_t)((i / kVec) * kLpThreads * kVec + i % kVec);
}

// Appends this thread's values above `low` (with `ties`, at it as well) to the
// candidates, in no particular order: they are ranked by their keys. (Calls of
// their own from here on: rare, and inlined they took the main loop's registers.)
template <bool kBf16>
__device__ __noinline__ void lp_append(LpShared& S, int cur, float low, bool ties, uint32_t i0) {
  using C = LpChunk<kBf16>;
  uint32_t hits = 0;  // bit per value: one atomic per thread, not one per value
#pragma unroll
  for (int i = 0; i < kLpVecs; ++i) {
    const uint4 q = S.own[i][threadIdx.x];
    const float vm = C::max_of(q);
    if (!(vm > low || (ties && vm == low))) continue;
#pragma unroll
    for (int j = 0; j < C::kVec; ++j) {
      const float x = C::value(q, j);
      if (x > low || (ties && x == low)) hits |= 1u << (i * C::kVec + j);
    }
  }
  int p = atomicAdd(&S.count[cur], __popc(hits));
  for (; hits != 0; hits &= hits - 1, ++p) {
    const int i = __ffs(hits) - 1;
    if (p < kLpCap) S.cand[p] = lp_key(lp_own<kBf16>(S, i), lp_index<kBf16>(i0, i));
  }
}

__device__ __forceinline__ float lp_last(const LpShared& S, int cur, int top) {
  const uint64_t k = S.list[cur][top - 1];
  return k == 0 ? -CUDART_INF_F : lp_value(k);
}

// Ranks the candidates (no more than fit) and list `cur` into list 1 - cur and
// returns its last value, -inf while it is not full. List and count `cur` are
// left at 0 for the round after. Called by the whole CTA after a barrier that
// follows the last append.
__device__ __noinline__ float lp_rank(LpShared& S, int cur, int top) {
  const int tid = threadIdx.x, n = S.count[cur];
  // the rank of a key is the number of larger ones (keys differ, empty ones aside)
  for (int i = tid; i < n + top; i += kLpThreads) {
    const uint64_t k = i < n ? S.cand[i] : S.list[cur][i - n];
    if (k == 0) continue;
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) rank += S.cand[j] > k;
#pragma unroll 4
    for (int j = 0; j < top; ++j) rank += S.list[cur][j] > k;
    if (rank < top) S.list[1 - cur][rank] = k;
  }
  __syncthreads();
  if (tid < kLpTop) S.list[cur][tid] = 0;
  if (tid == 0) S.count[cur] = 0;
  return lp_last(S, 1 - cur, top);
}

// Takes a chunk's values above `tau` (the last of the list's values, -inf while
// it is not full; with `ties`, values at tau as well) into the list, whatever
// their number: list `cur` becomes list 1 - cur, whose last value is returned.
// Threads whose maximum mx qualifies have left their values in S.own. No
// candidates are pending. Called by the whole CTA.
template <bool kBf16>
__device__ __noinline__ float lp_take(LpShared& S, int cur, float mx, float tau, bool ties, uint32_t i0,
                                      int top) {
  using C = LpChunk<kBf16>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // While the list is not full, a lower bound of its last value: with r =
  // ceil(top / warps), the smallest over the warps of their r-th largest
  // thread maximum has at least `top` values at or above it.
  float low = tau;
  if (tau == -CUDART_INF_F) {
    // (as ordered integers, for the warp's maximum in one instruction)
    uint32_t x = mx == mx ? (uint32_t)(lp_key(mx, 0) >> 32) : 0u, r = 0;
    for (int i = 0; i < (top + kLpWarps - 1) / kLpWarps; ++i) {
      r = __reduce_max_sync(0xffffffffu, x);
      const uint32_t at = __ballot_sync(0xffffffffu, x == r);
      if (lane == __ffs(at) - 1) x = 0;
    }
    const float rv = r <= 0x007FFFFFu ? -CUDART_INF_F : lp_value((uint64_t)r << 32);
    if (lane == 0) S.wm[warp] = rv;
    __syncthreads();
    low = S.wm[0];
#pragma unroll
    for (int w = 1; w < kLpWarps; ++w) low = fminf(low, S.wm[w]);
    ties = low > -CUDART_INF_F;
  }
  const bool has = mx > low || (ties && mx == low);
  if (has) lp_append<kBf16>(S, cur, low, ties, i0);
  __syncthreads();
  if (S.count[cur] <= kLpCap) return lp_rank(S, cur, top);
  // more candidates than fit (many equal or ascending values): the largest key
  // below the last one, `top` times
  uint64_t last = ~0ull;
  for (int t = 0; t < top; ++t) {
    uint64_t best = 0;
    if (tid < top && S.list[cur][tid] < last) best = S.list[cur][tid];
    if (has) {
#pragma unroll 4
      for (int i = 0; i < C::kPer; ++i) {
        const float x = lp_own<kBf16>(S, i);
        const uint64_t k = lp_key(x, lp_index<kBf16>(i0, i));
        if (x > -CUDART_INF_F && k < last && k > best) best = k;
      }
    }
    best = warp_max_u64(best);
    if (lane == 0) S.red[warp] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kLpWarps; ++w) best = S.red[w] > best ? S.red[w] : best;
    last = best;
    if (tid == 0) S.list[1 - cur][t] = best;  // (0 once there are no more)
    __syncthreads();
  }
  if (tid < kLpTop) S.list[cur][tid] = 0;
  if (tid == 0) S.count[cur] = 0;
  return lp_last(S, 1 - cur, top);
}

template <bool kBf16>
__global__ void __launch_bounds__(kLpThreads, kLpCtas) token_logprobs_kernel(const LpArgs a) {
  using C = LpChunk<kBf16>;
  __shared__ LpShared S;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t m = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
  const int split = blockIdx.x;
  const char* row = reinterpret_cast<const char*>(a.logits) + m * a.ldl * (kBf16 ? 2 : 4);
  // The row is `head` values up to a 16-byte boundary, whole vectors, and a
  // tail. The vectors are cut into pieces; the values around them are a last
  // step of the first piece, one per thread.
  constexpr int kEs = kBf16 ? 2 : 4;
  const int64_t head = min((int64_t)((16 - reinterpret_cast<uintptr_t>(row) % 16) % 16) / kEs, a.V);
  const int64_t vecs = (a.V - head) / C::kVec, tail = head + vecs * C::kVec;
  const uint4* body = reinterpret_cast<const uint4*>(row + head * kEs);
  const int64_t per = ceil_div(vecs, (int64_t)a.splits);
  const int64_t v0 = split * per, v1 = v0 + per < vecs ? v0 + per : vecs;
  constexpr int kStep = kLpVecs * kLpThreads;  // vectors per chunk
  const int chunks = v1 > v0 ? (int)ceil_div(v1 - v0, (int64_t)kStep) : 0;
  const int around = split == 0 ? (int)(head + a.V - tail) : 0;
  const int steps = chunks + (around > 0);
  const int64_t mine = tid < head ? tid : tail + tid - head;  // this thread's value around the vectors
  if (tid < 2 * kLpTop) S.list[tid / kLpTop][tid % kLpTop] = 0;
  if (tid < 2) S.count[tid] = 0;
  if (chunks > kLpFold) {
    S.fold[0][tid] = -CUDART_INF_F;
#pragma unroll
    for (int i = 1; i < 5; ++i) S.fold[i][tid] = 0.0f;
  }
  int cur_list = 0;
  bool pending = false;  // this thread has candidates that are not ranked yet
  __syncthreads();

  float mx = -CUDART_INF_F, tau = -CUDART_INF_F;
  float sum = 0.0f, tsum = 0.0f;  // tsum in units of log2
  bool over = false;
  auto index0 = [&](int step) {  // row index of the thread's value 0
    return step < chunks ? (uint32_t)(head + (v0 + (int64_t)step * kStep + tid) * C::kVec) : (uint32_t)mine;
  };
  C cur;
  auto load = [&](C& c, int step) {
    if (step < chunks) c.load(body + v0 + (int64_t)step * kStep, (int)(v1 - v0 - (int64_t)step * kStep));
    else c.load_one(row, mine, tid < around);
  };
  if (steps > 0) load(cur, 0);
  const uint4* next = body + v0;  // chunk on its way, and the vectors from there on
  int left = (int)(v1 - v0);
  // a given id and its logit take two trips to memory: the first now, the
  // second after the first chunk
  const int64_t id = split == 0 && tid < a.G ? a.ids[m * a.G + tid] : -1;
  float x_id = 0.0f;
  int rank_at = 0;  // the next step whose candidates are ranked
  for (int step = 0; step < steps; ++step) {
    C nxt;
    next += kStep;
    left -= kStep;
    if (left > 0) nxt.load(next, left);
    else if (step + 1 < steps) nxt.load_one(row, mine, tid < around);
    const float cm = cur.max();
    if (step == 0 && id >= 0 && id < a.V) x_id = lp_load<kBf16>(row, id);
    if (cm > mx) {
      const float c = __expf(mx - cm);  // 0 while mx = -inf, where the sums are 0 (or NaN)
      const float d = fmaxf(mx - cm, -200.0f) * 1.44269504f;
      tsum = c * fmaf(sum, d, tsum);
      sum = c * sum;
      mx = cm;
    }
    // Differences in units of log2, two values per packed operation (the loop
    // was bound by instructions: 14 a value without). One of -inf is lifted to
    // -288, whose term is 0 in fp32 as well (0 * inf would not be); a NaN stays
    // one, and +inf becomes one (inf - inf).
    const float ref = mx == -CUDART_INF_F ? 0.0f : mx;
    const float2 nref = make_float2(-ref, -ref), log2e = make_float2(1.44269504f, 1.44269504f);
    float2 sum2, tsum2;  // of this chunk (its first terms start them: no more additions than in one chain)
#pragma unroll
    for (int i = 0; i < C::kPer; i += 2) {
      float2 d = __fmul2_rn(__fadd2_rn(make_float2(cur.at(i), cur.at(i + 1)), nref), log2e);
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(d.x) : "f"(d.x), "f"(-288.0f));
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(d.y) : "f"(d.y), "f"(-288.0f));
      float2 e;
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(d.x));
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(d.y));
      sum2 = i == 0 ? e : __fadd2_rn(sum2, e);
      tsum2 = i == 0 ? __fmul2_rn(e, d) : __ffma2_rn(e, d, tsum2);
    }
    sum += sum2.x + sum2.y;
    tsum += tsum2.x + tsum2.y;
    if (a.top > 0) {
      // Until the list is full every chunk is ranked. From then on values above
      // its last are collected, and ranked after 2, 4, 8, ... chunks (each time
      // the rate of such values halves) and at the end.
      if (step != rank_at && step + 1 != steps) {
        if (cm > tau) {
#pragma unroll
          for (int i = 0; i < kLpVecs; ++i) S.own[i][tid] = cur.v[i];
          lp_append<kBf16>(S, cur_list, tau, false, index0(step));
          pending = true;
        }
      } else {
        // the values around the vectors come last, the head's with lower indices
        // than the list's: equal to tau they may still be among the best
        const bool ties = step >= chunks;
        const bool has = cm > tau || (ties && cm == tau && cm > -CUDART_INF_F);
        if (has) {
#pragma unroll
          for (int i = 0; i < kLpVecs; ++i) S.own[i][tid] = cur.v[i];
        }
        if (tau == -CUDART_INF_F) {
          if (__syncthreads_or(has)) {
            tau = lp_take<kBf16>(S, cur_list, cm, tau, ties, index0(step), a.top);
            cur_list ^= 1;
          }
          rank_at = tau == -CUDART_INF_F ? step + 1 : step | (step + 1);
        } else {
          if (has) lp_append<kBf16>(S, cur_list, tau, ties, index0(step));
          pending |= has;
          if (__syncthreads_or(pending)) {
            over |= S.count[cur_list] > kLpCap;
            if (!over) {
              tau = lp_rank(S, cur_list, a.top);
              cur_list ^= 1;
              pending = false;
            }
          }
          rank_at = 2 * step + 1;
        }
      }
    }
    cur = nxt;
    if (step % kLpFold == kLpFold - 1 && step + 1 < chunks) {
      lp_fold(S.fold, mx, sum, tsum * 0.693147181f);
      sum = tsum = 0.0f;
    }
  }
  if (over) {
    // more candidates than the buffer holds (ascending values): once more, chunk
    // by chunk
    __syncthreads();
    if (tid < 2 * kLpTop) S.list[tid / kLpTop][tid % kLpTop] = 0;
    if (tid < 2) S.count[tid] = 0;
    __syncthreads();
    tau = -CUDART_INF_F;
    for (int step = 0; step < steps; ++step) {
      load(cur, step);
      const float cm = cur.max();
      const bool ties = step >= chunks, has = cm > tau || (ties && cm == tau && cm > -CUDART_INF_F);
      if (has) {
#pragma unroll
        for (int i = 0; i < kLpVecs; ++i) S.own[i][tid] = cur.v[i];
      }
      if (__syncthreads_or(has)) {
        tau = lp_take<kBf16>(S, cur_list, cm, tau, ties, index0(step), a.top);
        cur_list ^= 1;
      }
    }
  }
  tsum *= 0.693147181f;
  if (chunks > kLpFold)
    lp_join(mx, sum, tsum, S.fold[0][tid], S.fold[1][tid] + S.fold[2][tid], S.fold[3][tid] + S.fold[4][tid]);
  lp_join_warp(mx, sum, tsum);
  __syncthreads();
  if (lane == 0) {
    S.wm[warp] = mx;
    S.wS[warp] = sum;
    S.wT[warp] = tsum;
  }
  __syncthreads();
  mx = S.wm[0];
  sum = S.wS[0];
  tsum = S.wT[0];
#pragma unroll
  for (int w = 1; w < kLpWarps; ++w) lp_join(mx, sum, tsum, S.wm[w], S.wS[w], S.wT[w]);
  if (a.splits == 1) {
    lp_outputs<kBf16>(a, m, row, mx, sum, tsum, S.list[cur_list], id, x_id);
    return;
  }
  // The pieces of a row are a cluster: the first CTA joins them. Their lists are
  // sorted: the k-th largest of their r-th keys has k * r >= top keys at or above
  // it, and with r about sqrt(top) not many more. Those are ranked.
  if (tid < a.top) S.final_list[tid] = S.list[cur_list][tid];
  if (tid == 0) {
    S.stats[0] = mx;
    S.stats[1] = sum;
    S.stats[2] = tsum;
  }
  cluster_sync();
  constexpr int kKeys = kLpMaxSplits * kLpTop / kLpThreads;
  const int shift = 31 - __clz(a.splits), n = a.splits * a.top;
  uint64_t k[kKeys];
  const bool has = lane < a.splits;
  if (split == 0) {
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
      const int i = tid + u * kLpThreads;  // key i >> shift of a piece
      k[u] = i < n ? ld_cluster_u64(map_to_cta(&S.final_list[i >> shift], i & (a.splits - 1))) : 0;
    }
    const uint32_t st = map_to_cta(S.stats, has ? lane : 0);
    mx = has ? ld_cluster_f32(st) : -CUDART_INF_F;
    sum = has ? ld_cluster_f32(st + 4) : 0.0f;
    tsum = has ? ld_cluster_f32(st + 8) : 0.0f;
  }
  cluster_arrive();  // a piece's shared memory outlives its reading, no more
  if (split == 0) {
    lp_join_warp(mx, sum, tsum);
    if (a.top > 0) {
      if (tid < kLpTop) S.list[1][tid] = 0;
      if (tid == 0) S.count[0] = 0;
      int r = 1;
      while (r * r < a.top || r * a.splits < a.top) ++r;
      const int kth = (a.top + r - 1) / r;
#pragma unroll
      for (int u = 0; u < kKeys; ++u) {
        const int i = tid + u * kLpThreads;
        if (i < n && i >> shift == r - 1) S.list[0][i & (a.splits - 1)] = k[u];
      }
      __syncthreads();
      const uint64_t own = has ? S.list[0][lane] : 0;
      int above = 0;
      for (int j = 0; j < a.splits; ++j) above += S.list[0][j] > own;
      const uint32_t at = __ballot_sync(0xffffffffu, own != 0 && above == kth - 1);
      const uint64_t low = at ? S.list[0][__ffs(at) - 1] : 0;
#pragma unroll
      for (int u = 0; u < kKeys; ++u)
        if (k[u] != 0 && k[u] >= low) S.cand[atomicAdd(&S.count[0], 1)] = k[u];
      __syncthreads();
      const int c = S.count[0];
      for (int i = tid; i < c; i += kLpThreads) {
        const uint64_t key = S.cand[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < c; ++j) rank += S.cand[j] > key;
        if (rank < a.top) S.list[1][rank] = key;
      }
      __syncthreads();
    }
    lp_outputs<kBf16>(a, m, row, mx, sum, tsum, S.list[1], id, x_id);
  }
  cluster_wait();
}

// Pieces per row, a power of two, none much shorter than a chunk of 4096 bf16 values
// (two of fp32). Doubled while there are fewer than 3.25 CTAs an SM (131072 bf16, top
// 5: 200 rows 24.2 us in 4 pieces, 27.1 in 2; 246 rows 27.0 in 4, 29.1 in 2; 247 to
// 493 rows 29.2 to 39.5 in 2, 36.4 to 42.8 whole), but to 16, where a row's join is the
// longest, only below 2 (31 rows 11.4 us, 12.6 in 8; 40 rows 12.5 and 13.1; 42 rows
// 13.8 and 13.3; 61 rows 16.4 and 14.4).
int lp_splits(int64_t M, int64_t V, int sms) {
  int s = 1;
  while (s < kLpMaxSplits && M * s * 4 < (s < 8 ? 13 : 8) * (int64_t)sms && V > 4096 * (int64_t)s) s *= 2;
  return s;
}

template <bool kBf16>
static cudaError_t launch_lp(const LpArgs& a, int64_t M, cudaStream_t st) {
  auto kern = token_logprobs_kernel<kBf16>;
  if (a.splits > 8) {  // clusters of more than eight CTAs have to be asked for
    static std::atomic<uint64_t> attr_set{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
    if (!bit || !(attr_set.load(std::memory_order_acquire) & bit)) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      attr_set.fetch_or(bit, std::memory_order_release);
    }
  }
  // rows over grid.y and z (y is limited to 65535)
  const int64_t rows_y = M < 32768 ? M : 32768;
  for (int64_t m0 = 0; m0 < M;) {
    const int64_t z = M - m0 >= rows_y ? (M - m0) / rows_y : 1, y = M - m0 >= rows_y ? rows_y : M - m0;
    LpArgs b = a;
    b.logits = reinterpret_cast<const char*>(a.logits) + m0 * a.ldl * (kBf16 ? 2 : 4);
    if (a.ids) b.ids = a.ids + m0 * a.G;
    if (a.logprobs) b.logprobs = a.logprobs + m0 * a.G;
    if (a.entropy) b.entropy = a.entropy + m0;
    if (a.top_ids) b.top_ids = a.top_ids + m0 * a.top;
    if (a.top_logprobs) b.top_logprobs = a.top_logprobs + m0 * a.top;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.splits, (unsigned)y, (unsigned)z);
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.splits > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, b);
    if (e != cudaSuccess) return e;
    m0 += y * z;
  }
  return cudaSuccess;
}

cudaError_t launch_token_logprobs(const void* logits, bool bf16, int64_t M, int64_t V, int64_t ldl,
                                  const int64_t* ids, int64_t G, float* logprobs, float* entropy,
                                  int top, int64_t* top_ids, float* top_logprobs, cudaStream_t st) {
  const LpArgs a{logits, V, ldl, ids, logprobs, entropy, top_ids, top_logprobs, (int)G, top, lp_splits(M, V, num_sms())};
  return bf16 ? launch_lp<true>(a, M, st) : launch_lp<false>(a, M, st);
}

}  // namespace qg
