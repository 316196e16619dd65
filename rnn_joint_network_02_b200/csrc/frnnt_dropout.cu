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

// Bit j: element j of the counter's eight stays.
__device__ __forceinline__ uint32_t keep_bits(uint64_t counter, uint64_t seed, uint32_t limit) {
  const uint4 w = philox(counter, seed);
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
  uint32_t k = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) k |= (uint32_t)(((words[j >> 1] >> (16 * (j & 1))) & 0xFFFFu) >= limit) << j;
  return k;
}

constexpr int kThreads = 256;
constexpr int kGroups = 2;   // counters a thread has in flight

// The 8 elements of a counter, in one access: 16 bytes of a 16-bit type, 32 of
// a 32-bit one.
template <typename T>
struct alignas(8 * sizeof(T)) Group {
  uint32_t v[2 * sizeof(T)];
};
__device__ __forceinline__ void load(Group<__nv_bfloat16>& g, const __nv_bfloat16* p) {
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(g.v[0]), "=r"(g.v[1]), "=r"(g.v[2]), "=r"(g.v[3])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void load(Group<float>& g, const float* p) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(g.v[0]), "=r"(g.v[1]), "=r"(g.v[2]), "=r"(g.v[3]), "=r"(g.v[4]), "=r"(g.v[5]), "=r"(g.v[6]),
                 "=r"(g.v[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store(const Group<__nv_bfloat16>& g, __nv_bfloat16* p) {
  asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(g.v[0]), "r"(g.v[1]), "r"(g.v[2]), "r"(g.v[3])
               : "memory");
}
__device__ __forceinline__ void store(const Group<float>& g, float* p) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(g.v[0]), "r"(g.v[1]),
               "r"(g.v[2]), "r"(g.v[3]), "r"(g.v[4]), "r"(g.v[5]), "r"(g.v[6]), "r"(g.v[7])
               : "memory");
}

// An element is read and written once, and the generator costs 20 wide products
// a counter, 2.5 an element.  32-bit: bound by memory, 32000 x 1024 40 us (6.5
// TB/s, the copy rate; a thread per counter with single elements: 136 us).  16-bit:
// half the bytes and the same instructions, bound by those: 29 us (4.5 TB/s), and 33
// in rows at a distance, whose place costs a division.
// Rows whose groups of 8 elements are whole and aligned: a thread takes whole
// counters.  With one row (contiguous memory) the last group may be short; the
// first thread takes its elements one by one.
template <typename T>
__global__ void __launch_bounds__(kThreads) dropout_vec_kernel(DropParams p, const T* x, T* y) {
  const uint64_t seed = p.rng ? p.rng[0] : p.seed;
  const uint64_t first = p.offset + (p.rng ? p.rng[1] : 0);
  const long long groups = p.n >> 3, per_row = p.C >> 3;
  const long long g0 = (long long)blockIdx.x * (kThreads * kGroups) + threadIdx.x;
  Group<T> in[kGroups];
  long long at[kGroups];
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const long long g = g0 + k * kThreads;
    if (g < groups) {
      long long r = 0, c = g;
      if (per_row < groups) {
        r = g / per_row;
        c = g - r * per_row;
      }
      at[k] = r * p.y_ld + c * 8;
      load(in[k], x + r * p.x_ld + c * 8);
    }
  }
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const long long g = g0 + k * kThreads;
    if (g < groups) {
      const uint4 bits = philox(first + (uint64_t)g, seed);
      const uint32_t words[4] = {bits.x, bits.y, bits.z, bits.w};
      uint32_t* v = in[k].v;
#pragma unroll
      for (int j = 0; j < 4; ++j) {   // elements 2j and 2j + 1
        const bool k0 = (words[j] & 0xFFFFu) >= p.limit, k1 = (words[j] >> 16) >= p.limit;
        if constexpr (sizeof(T) == 4) {
          v[2 * j] = k0 ? __float_as_uint(__uint_as_float(v[2 * j]) * p.scale) : 0u;
          v[2 * j + 1] = k1 ? __float_as_uint(__uint_as_float(v[2 * j + 1]) * p.scale) : 0u;
        } else {
          const float a = __uint_as_float(v[j] << 16) * p.scale, b = __uint_as_float(v[j] & 0xFFFF0000u) * p.scale;
          const __nv_bfloat162 o = __floats2bfloat162_rn(k0 ? a : 0.f, k1 ? b : 0.f);
          v[j] = *reinterpret_cast<const uint32_t*>(&o);
        }
      }
      store(in[k], y + at[k]);
    }
  }
  // the short last group
  if (g0 == 0)
    for (long long e = groups * 8; e < p.n; ++e) {
      const bool stay = keep_bits(first + (uint64_t)groups, seed, p.limit) >> (e & 7) & 1;
      y[e] = from_f32<T>(stay ? to_f32<T>(x[e]) * p.scale : 0.f);
    }
}

// Any layout: a warp takes 32 counters, and its lanes walk their 256 elements
// side by side, each asking the lane that has the element's counter.  Bound by
// its instructions, one element each: 32000 x 1023 in rows of 1025, fp32 92 us (2.9
// TB/s), bf16 79.
template <typename T>
__global__ void __launch_bounds__(kThreads) dropout_any_kernel(DropParams p, const T* x, T* y) {
  const int lane = threadIdx.x & 31;
  const long long warp = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const long long e0 = warp * 256;
  if (e0 >= p.n) return;
  const uint64_t seed = p.rng ? p.rng[0] : p.seed;
  const uint64_t first = p.offset + (p.rng ? p.rng[1] : 0);
  const uint32_t mine = keep_bits(first + (uint64_t)(warp * 32 + lane), seed, p.limit);
  long long r = (e0 + lane) / p.C, c = e0 + lane - r * p.C;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t k = __shfl_sync(0xFFFFFFFFu, mine, j * 4 + (lane >> 3));
    if (e0 + j * 32 + lane < p.n) {
      const float v = to_f32<T>(x[r * p.x_ld + c]);
      y[r * p.y_ld + c] = from_f32<T>((k >> (lane & 7)) & 1 ? v * p.scale : 0.f);
    }
    c += 32;
    if (c >= p.C) {
      const long long over = c / p.C;
      r += over;
      c -= over * p.C;
    }
  }
}

template <typename T>
void launch(const DropParams& p, bool rows, const void* x, void* y, cudaStream_t st) {
  const bool aligned = (uintptr_t)x % sizeof(Group<T>) == 0 && (uintptr_t)y % sizeof(Group<T>) == 0;
  const bool whole = !rows || (p.C % 8 == 0 && p.x_ld % 8 == 0 && p.y_ld % 8 == 0);
  if (aligned && whole) {
    const long long per = 8LL * kThreads * kGroups;
    launch_k(dropout_vec_kernel<T>, dim3((unsigned)((p.n + per - 1) / per)), dim3(kThreads), 0, st, 1, p,
             (const T*)x, (T*)y);
  } else {
    const long long per = 8LL * kThreads;
    launch_k(dropout_any_kernel<T>, dim3((unsigned)((p.n + per - 1) / per)), dim3(kThreads), 0, st, 1, p,
             (const T*)x, (T*)y);
  }
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
      !(d->p >= 0.0 && d->p <= 1.0))
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
  p.limit = (uint32_t)(d->p * 65536.0 + 0.5);
  p.scale = p.limit < 65536u ? 65536.f / (float)(65536u - p.limit) : 0.f;
  p.seed = d->seed;
  p.offset = d->offset;
  p.rng = rng;
  {
    StageScope sc("dropout", st);
    const bool rows = d->R > 1 && (d->x_ld != d->C || d->y_ld != d->C);   // not one run of memory
    if (!rows) p.C = p.n;
    if (d->dtype == FRNNT_BF16) launch<__nv_bfloat16>(p, rows, x, y, st);
    else launch<float>(p, rows, x, y, st);
  }
  return cudaGetLastError() == cudaSuccess ? FRNNT_OK : FRNNT_ERR_CUDA;
}
