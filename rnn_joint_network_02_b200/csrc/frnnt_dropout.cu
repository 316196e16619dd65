// Dropout from a counter-based generator: y = x * keep / (1 - p), the mask
// recomputed from (seed, counter) wherever it is needed and never stored.
#include "frnnt_common.cuh"
#include "frnnt_internal.h"
#include "frnnt_ops.h"

namespace frnnt {
namespace {

// One Philox4x32-10 block (Salmon, Moraes, Dror, Shaw, "Parallel Random
// Numbers: As Easy as 1, 2, 3"): ten rounds of two 32 x 32 -> 64-bit products
// over a 128-bit counter, the key bumped by the two Weyl constants.
__device__ __forceinline__ uint4 philox(uint64_t counter, uint64_t seed) {
  uint32_t c0 = (uint32_t)counter, c1 = (uint32_t)(counter >> 32), c2 = 0, c3 = 0;
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
    const uint32_t n0 = (uint32_t)(q >> 32) ^ c1 ^ k0, n2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)q;
    c3 = (uint32_t)p;
    c0 = n0;
    c2 = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

struct DropParams {
  long long C, n, x_ld, y_ld;
  uint32_t limit;      // bits below it drop
  float scale;
  uint64_t seed, offset;
  const uint64_t* rng;
};

// A thread per counter: 8 consecutive elements.
template <typename T>
__global__ void dropout_kernel(DropParams p, const T* x, T* y) {
  const long long g = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (g * 8 >= p.n) return;
  const uint64_t seed = p.rng ? p.rng[0] : p.seed;
  const uint64_t off = p.offset + (p.rng ? p.rng[1] : 0);
  const uint4 w = philox(off + (uint64_t)g, seed);
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
  for (int j = 0; j < 8; ++j) {
    const long long e = g * 8 + j;
    if (e >= p.n) break;
    const long long r = e / p.C, c = e - r * p.C;
    const uint32_t bits = (words[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
    const float v = to_f32<T>(x[r * p.x_ld + c]);
    y[r * p.y_ld + c] = from_f32<T>(bits >= p.limit ? v * p.scale : 0.f);
  }
}

template <typename T>
void launch(const DropParams& p, const void* x, void* y, cudaStream_t st) {
  const long long groups = (p.n + 7) / 8;
  dropout_kernel<T><<<(unsigned)((groups + 255) / 256), 256, 0, st>>>(p, (const T*)x, (T*)y);
  note_launch();
}

}  // namespace
}  // namespace frnnt

using namespace frnnt;

extern "C" FRNNT_API int frnnt_dropout(const frnnt_dropout_dims* d, const void* x, void* y, const uint64_t* rng,
                                       void* stream) {
  if (!d || !x || !y) return FRNNT_ERR_NULL;
  if (d->dtype != FRNNT_F32 && d->dtype != FRNNT_BF16) return FRNNT_ERR_UNSUPPORTED;
  // (the comparison's negation also refuses a NaN p)
  if (d->R < 1 || d->C < 1 || d->R > (1LL << 40) / d->C || d->x_ld < d->C || d->y_ld < d->C ||
      !(d->p >= 0.f && d->p <= 1.f))
    return FRNNT_ERR_DIMS;
  const size_t es = d->dtype == FRNNT_BF16 ? 2 : 4;
  if ((uintptr_t)x % es || (uintptr_t)y % es || (uintptr_t)rng % 8) return FRNNT_ERR_ALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  cudaGetLastError();   // clear a stale error so it is not reported as ours
  DropParams p;
  p.C = d->C;
  p.n = d->R * d->C;
  p.x_ld = d->x_ld;
  p.y_ld = d->y_ld;
  p.limit = (uint32_t)((double)d->p * 65536.0 + 0.5);
  p.scale = p.limit < 65536u ? 65536.f / (float)(65536u - p.limit) : 0.f;
  p.seed = d->seed;
  p.offset = d->offset;
  p.rng = rng;
  {
    StageScope sc("dropout", st);
    if (d->dtype == FRNNT_BF16) launch<__nv_bfloat16>(p, x, y, st);
    else launch<float>(p, x, y, st);
  }
  return cudaGetLastError() == cudaSuccess ? FRNNT_OK : FRNNT_ERR_CUDA;
}
