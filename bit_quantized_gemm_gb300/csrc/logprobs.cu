// logprobs.cu -- log probabilities of given tokens, entropy and the largest
// alternatives of each row of logits.
//
// With m = max x, S = sum e^(x-m), T = sum e^(x-m) (x-m) over a row of V:
//   log p[i] = x[i] - m - log S,   H = -sum p log p = log S - T / S
// (both terms of H are >= 0: nothing cancels). The alternatives are the first
// `top` values in the order (value descending, index ascending).
// Statistics are held in fp32.
//
// Rows without a distribution: -inf everywhere (a mask that leaves nothing)
// gives log p = -inf, H = 0 and no alternatives (index -1, -inf); a row with a
// NaN or +inf gives NaN and no alternatives (index -1, NaN). An alternative of
// -inf is none: its index is -1. An id below 0 asks for nothing and gives 0; an
// id >= V gives NaN.
//
// The plain form: one CTA per row, one pass for m, S, T and one pass for each
// alternative.
#include <math_constants.h>

#include "qg_common.cuh"

namespace qg {

template <bool kBf16>
__device__ __forceinline__ float load_logit(const void* row, int64_t i) {
  if (kBf16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
  return reinterpret_cast<const float*>(row)[i];
}

template <bool kBf16>
__global__ void __launch_bounds__(256) logprobs_plain_kernel(
    const void* __restrict__ logits, int64_t V, int64_t ldl, const int64_t* __restrict__ ids, int G,
    float* __restrict__ logprobs, float* __restrict__ entropy, int top,
    int64_t* __restrict__ top_ids, float* __restrict__ top_logprobs) {
  const int64_t m = blockIdx.x;
  const int tid = threadIdx.x;
  const char* row = reinterpret_cast<const char*>(logits) + m * ldl * (kBf16 ? 2 : 4);
  __shared__ float fs[256];
  __shared__ float ft[256];
  __shared__ int64_t is[256];
  float mx = -CUDART_INF_F;
  bool bad = false;
  for (int64_t i = tid; i < V; i += 256) {
    const float x = load_logit<kBf16>(row, i);
    bad |= !(x < CUDART_INF_F);
    mx = fmaxf(mx, x);
  }
  fs[tid] = mx;
  bad = __syncthreads_or(bad);
  for (int i = 0; i < 256; ++i) mx = fmaxf(mx, fs[i]);
  __syncthreads();
  const bool empty = mx == -CUDART_INF_F;
  float S = 0.0f, T = 0.0f;
  if (!bad && !empty)
    for (int64_t i = tid; i < V; i += 256) {
      const float d = load_logit<kBf16>(row, i) - mx;
      const float e = expf(d);
      S += e;
      if (e > 0.0f) T += e * d;
    }
  fs[tid] = S;
  ft[tid] = T;
  __syncthreads();
  S = T = 0.0f;
  for (int i = 0; i < 256; ++i) {
    S += fs[i];
    T += ft[i];
  }
  __syncthreads();
  const float shift = empty ? 0.0f : mx, lse = empty ? 0.0f : logf(S);
  auto logp = [&](float x) {
    if (bad) return CUDART_NAN_F;
    return x == -CUDART_INF_F ? x : (x - shift) - lse;
  };
  if (tid == 0 && entropy) entropy[m] = bad ? CUDART_NAN_F : empty ? 0.0f : lse - T / S;
  for (int g = tid; g < G; g += 256) {
    const int64_t id = ids[m * G + g];
    logprobs[m * G + g] = id < 0 ? 0.0f : id >= V ? CUDART_NAN_F : logp(load_logit<kBf16>(row, id));
  }
  float last = CUDART_INF_F;
  int64_t last_i = -1;
  for (int t = 0; t < top; ++t) {
    float best = -CUDART_INF_F;
    int64_t best_i = V;
    if (!bad)
      for (int64_t i = tid; i < V; i += 256) {
        const float x = load_logit<kBf16>(row, i);
        if ((x < last || (x == last && i > last_i)) && x > best) {
          best = x;
          best_i = i;
        }
      }
    fs[tid] = best;
    is[tid] = best_i;
    __syncthreads();
    for (int i = 0; i < 256; ++i)
      if (fs[i] > best || (fs[i] == best && is[i] < best_i)) {
        best = fs[i];
        best_i = is[i];
      }
    __syncthreads();
    last = best;
    last_i = best_i;
    if (tid == 0) {
      const bool none = bad || best == -CUDART_INF_F;
      top_ids[m * top + t] = none ? -1 : best_i;
      top_logprobs[m * top + t] = logp(best);
    }
  }
}

cudaError_t launch_token_logprobs(const void* logits, bool bf16, int64_t M, int64_t V, int64_t ldl,
                                  const int64_t* ids, int64_t G, float* logprobs, float* entropy,
                                  int top, int64_t* top_ids, float* top_logprobs, void* ws,
                                  cudaStream_t st) {
  (void)ws;
  if (bf16)
    logprobs_plain_kernel<true><<<(unsigned)M, 256, 0, st>>>(logits, V, ldl, ids, (int)G, logprobs,
                                                             entropy, top, top_ids, top_logprobs);
  else
    logprobs_plain_kernel<false><<<(unsigned)M, 256, 0, st>>>(logits, V, ldl, ids, (int)G, logprobs,
                                                              entropy, top, top_ids, top_logprobs);
  return cudaGetLastError();
}

int64_t token_logprobs_ws_bytes(int64_t M, int64_t V, int top) {
  (void)M; (void)V; (void)top;
  return 256;
}

}  // namespace qg
