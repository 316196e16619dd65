// Token log-probabilities of rows of logits: log-softmax values of given
// tokens, entropy, the best alternatives, and the gradient of the logits.
#include "frnnt_common.cuh"
#include "frnnt_internal.h"
#include "frnnt_ops.h"

namespace frnnt {
namespace {

constexpr int kThreads = 256;

// Order-preserving image of a float among unsigned integers; NaN below all.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0u;
  if (v == 0.f) v = 0.f;   // -0 and +0 are equal
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

template <typename F>
__device__ __forceinline__ float block_reduce(float v, float* sm, F f) {
  sm[threadIdx.x] = v;
  __syncthreads();
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    if (threadIdx.x < o) sm[threadIdx.x] = f(sm[threadIdx.x], sm[threadIdx.x + o]);
    __syncthreads();
  }
  const float r = sm[0];
  __syncthreads();
  return r;
}

// A block per row; one pass for the maximum, one for the sums, one for each
// alternative.
template <typename T>
__global__ void __launch_bounds__(kThreads) logprob_fwd_kernel(int V, int K, int top, long long ld, const T* logits,
                                                               const int32_t* tokens, float* logp, float* entropy,
                                                               float* lse, float* top_logp, int32_t* top_ids,
                                                               int32_t* status) {
  __shared__ float sm[kThreads];
  __shared__ unsigned long long best_sm[kThreads];
  const long long n = blockIdx.x;
  const T* z = logits + n * ld;
  float m = -INFINITY;
  for (int j = threadIdx.x; j < V; j += kThreads) m = fmaxf(m, to_f32<T>(z[j]));
  m = block_reduce(m, sm, [](float a, float b) { return fmaxf(a, b); });
  const float m0 = m == -INFINITY ? 0.f : m;
  float s = 0.f, w = 0.f;
  for (int j = threadIdx.x; j < V; j += kThreads) {
    const float d = to_f32<T>(z[j]) - m0, e = expf(d);
    s += e;
    if (e != 0.f) w += e * d;
  }
  s = block_reduce(s, sm, [](float a, float b) { return a + b; });
  w = block_reduce(w, sm, [](float a, float b) { return a + b; });
  const bool empty = s == 0.f;
  const float ls = logf(s), l = empty ? -INFINITY : m0 + ls;
  if (threadIdx.x == 0) {
    lse[n] = l;
    entropy[n] = empty ? 0.f : ls - w / s;
  }
  for (int k = threadIdx.x; k < K; k += kThreads) {
    const int t = tokens[n * K + k];
    if (t != FRNNT_NO_TOKEN && (t < 0 || t >= V) && status) atomicOr(status, FRNNT_STATUS_LABEL);
    logp[n * K + k] = t < 0 || t >= V ? 0.f : (empty ? -INFINITY : (to_f32<T>(z[t]) - m0) - ls);
  }
  unsigned long long last = ~0ull;
  for (int i = 0; i < top; ++i) {
    unsigned long long best = 0;
    for (int j = threadIdx.x; j < V; j += kThreads) {
      const unsigned long long c = ((unsigned long long)order_key(to_f32<T>(z[j])) << 32) | (uint32_t)~j;
      if (c < last && c > best) best = c;
    }
    best_sm[threadIdx.x] = best;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
      if (threadIdx.x < o && best_sm[threadIdx.x + o] > best_sm[threadIdx.x])
        best_sm[threadIdx.x] = best_sm[threadIdx.x + o];
      __syncthreads();
    }
    last = best_sm[0];
    __syncthreads();
    if (threadIdx.x == 0) {
      const int j = (int)~(uint32_t)last;
      top_ids[n * top + i] = j;
      top_logp[n * top + i] = empty ? -INFINITY : (to_f32<T>(z[j]) - m0) - ls;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) logprob_bwd_kernel(int V, int K, int top, long long ld, long long ldd,
                                                               const T* logits, const int32_t* tokens,
                                                               const float* lse, const float* entropy,
                                                               const int32_t* top_ids, const float* dlogp,
                                                               const float* dentropy, const float* dtop, T* dlogits,
                                                               int32_t* status) {
  __shared__ int ids[FRNNT_MAX_TOKENS + FRNNT_MAX_TOP];
  __shared__ float coef[FRNNT_MAX_TOKENS + FRNNT_MAX_TOP];
  const long long n = blockIdx.x;
  const int nk = dlogp ? K : 0, nt = dtop ? top : 0, cnt = nk + nt;
  for (int i = threadIdx.x; i < cnt; i += kThreads) {
    int t = i < nk ? tokens[n * K + i] : top_ids[n * top + i - nk];
    const bool none = i < nk && t == FRNNT_NO_TOKEN;
    if (!none && (t < 0 || t >= V) && status) atomicOr(status, FRNNT_STATUS_LABEL);
    if (t < 0 || t >= V) t = -1;
    ids[i] = t;
    coef[i] = t < 0 ? 0.f : (i < nk ? dlogp[n * K + i] : dtop[n * top + i - nk]);
  }
  __syncthreads();
  float c = 0.f;
  bool none = !dentropy;   // a row without any term gets zeros, whatever it holds
  for (int i = 0; i < cnt; ++i) {
    c += coef[i];
    none = none && ids[i] < 0;
  }
  const float l = lse[n], dh = dentropy ? dentropy[n] : 0.f, h = dentropy ? entropy[n] : 0.f;
  for (int j = threadIdx.x; j < V; j += kThreads) {
    const float lp = to_f32<T>(logits[n * ld + j]) - l, p = expf(lp);
    float g = p == 0.f ? 0.f : -p * (c + dh * (lp + h));
    for (int i = 0; i < cnt; ++i)
      if (ids[i] == j) g += coef[i];
    dlogits[n * ldd + j] = from_f32<T>(none || l == -INFINITY ? 0.f : g);
  }
}

int check(const frnnt_logprob_dims* d) {
  if (d->dtype != FRNNT_F32 && d->dtype != FRNNT_BF16) return FRNNT_ERR_UNSUPPORTED;
  if (d->N < 1 || d->V < 1 || d->K < 0 || d->K > FRNNT_MAX_TOKENS || d->top < 0 || d->top > FRNNT_MAX_TOP ||
      d->top > d->V || d->ld < d->V || d->ld > (1LL << 40))
    return FRNNT_ERR_DIMS;
  return FRNNT_OK;
}

}  // namespace
}  // namespace frnnt

using namespace frnnt;

extern "C" FRNNT_API int frnnt_token_logprobs(const frnnt_logprob_dims* d, const void* logits, const int32_t* tokens,
                                              float* logp, float* entropy, float* lse, float* top_logp,
                                              int32_t* top_ids, int32_t* status, void* stream) {
  if (!d) return FRNNT_ERR_NULL;
  if (const int rc = check(d)) return rc;
  if (!logits || !entropy || !lse || (d->K && (!tokens || !logp)) || (d->top && (!top_logp || !top_ids)))
    return FRNNT_ERR_NULL;
  if ((uintptr_t)logits % (d->dtype == FRNNT_BF16 ? 2 : 4)) return FRNNT_ERR_ALIGN;
  for (const void* p : {(const void*)tokens, (const void*)logp, (const void*)entropy, (const void*)lse,
                        (const void*)top_logp, (const void*)top_ids, (const void*)status})
    if ((uintptr_t)p % 4) return FRNNT_ERR_ALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  cudaGetLastError();   // clear a stale error so it is not reported as ours
  {
    StageScope sc("token_logprobs", st);
    if (d->dtype == FRNNT_BF16)
      logprob_fwd_kernel<__nv_bfloat16><<<d->N, kThreads, 0, st>>>(d->V, d->K, d->top, d->ld,
                                                                   (const __nv_bfloat16*)logits, tokens, logp,
                                                                   entropy, lse, top_logp, top_ids, status);
    else
      logprob_fwd_kernel<float><<<d->N, kThreads, 0, st>>>(d->V, d->K, d->top, d->ld, (const float*)logits, tokens,
                                                           logp, entropy, lse, top_logp, top_ids, status);
    note_launch();
  }
  return cudaGetLastError() == cudaSuccess ? FRNNT_OK : FRNNT_ERR_CUDA;
}

extern "C" FRNNT_API int frnnt_token_logprobs_bwd(const frnnt_logprob_dims* d, const void* logits,
                                                  const int32_t* tokens, const float* lse, const float* entropy,
                                                  const int32_t* top_ids, const float* dlogp, const float* dentropy,
                                                  const float* dtop, void* dlogits, int32_t* status, void* stream) {
  if (!d) return FRNNT_ERR_NULL;
  if (const int rc = check(d)) return rc;
  if (d->ldd < d->V || d->ldd > (1LL << 40)) return FRNNT_ERR_DIMS;
  if (dlogits == logits && d->ldd != d->ld) return FRNNT_ERR_DIMS;
  if (!logits || !lse || !dlogits || (dentropy && !entropy) || (d->K && dlogp && !tokens) ||
      (d->top && dtop && !top_ids))
    return FRNNT_ERR_NULL;
  const size_t es = d->dtype == FRNNT_BF16 ? 2 : 4;
  if ((uintptr_t)logits % es || (uintptr_t)dlogits % es) return FRNNT_ERR_ALIGN;
  for (const void* p : {(const void*)tokens, (const void*)lse, (const void*)entropy, (const void*)top_ids,
                        (const void*)dlogp, (const void*)dentropy, (const void*)dtop, (const void*)status})
    if ((uintptr_t)p % 4) return FRNNT_ERR_ALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  cudaGetLastError();   // clear a stale error so it is not reported as ours
  {
    StageScope sc("token_logprobs_bwd", st);
    if (d->dtype == FRNNT_BF16)
      logprob_bwd_kernel<__nv_bfloat16><<<d->N, kThreads, 0, st>>>(
          d->V, d->K, d->top, d->ld, d->ldd, (const __nv_bfloat16*)logits, tokens, lse, entropy, top_ids, dlogp,
          dentropy, dtop, (__nv_bfloat16*)dlogits, status);
    else
      logprob_bwd_kernel<float><<<d->N, kThreads, 0, st>>>(d->V, d->K, d->top, d->ld, d->ldd, (const float*)logits,
                                                           tokens, lse, entropy, top_ids, dlogp, dentropy, dtop,
                                                           (float*)dlogits, status);
    note_launch();
  }
  return cudaGetLastError() == cudaSuccess ? FRNNT_OK : FRNNT_ERR_CUDA;
}
