// Shared device helpers of the frnnt library (not part of the C ABI).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "frnnt.h"

namespace frnnt {

__host__ __device__ inline int clampi(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

// Lengths as every kernel sees them: clamped into range so that invalid
// inputs (already flagged in the status word by the validation kernel) can
// never turn into out-of-bounds accesses.
struct Lengths {
  int Tb, Ub;
};
__device__ inline Lengths lengths_of(const int32_t* T_len, const int32_t* U_len, int b, int T, int U) {
  Lengths l;
  l.Tb = clampi(T_len[b], 1, T);
  l.Ub = clampi(U_len[b], 0, U);
  return l;
}
// Status bits found by one thread of a block that checks the lengths and
// labels (strided by nthreads): FRNNT_STATUS_LENGTH for T_len outside [1,T] or
// U_len outside [0,U], FRNNT_STATUS_LABEL for a label (u < U_len) outside
// [0,V) or equal to blank.
__device__ inline int validate_bits(int B, int T, int U, int V, int blank, const int32_t* labels,
                                    const int32_t* T_len, const int32_t* U_len, int tid, int nthreads) {
  int bits = 0;
  for (int b = tid; b < B; b += nthreads) {
    const int tl = T_len[b], ul = U_len[b];
    if (tl < 1 || tl > T || ul < 0 || ul > U) bits |= FRNNT_STATUS_LENGTH;
  }
  const long long n = (long long)B * U;
  for (long long i = tid; i < n; i += nthreads) {
    const int b = (int)(i / U), u = (int)(i % U);
    const int tl = T_len[b], ul = U_len[b];
    if (tl < 1 || tl > T || ul < 0 || ul > U) continue;   // length already flagged
    if (u >= ul) continue;                                // padding label
    const int y = labels[i];
    if (y < 0 || y >= V || y == blank) bits |= FRNNT_STATUS_LABEL;
  }
  return bits;
}
__device__ inline int label_of(const int32_t* labels, int b, int u, int U, int V) {
  return clampi(labels[(size_t)b * U + u], 0, V - 1);
}

// log(exp(a) + exp(b)) in fp32, exact for -inf operands: max + ln(1 + e^-|a-b|),
// with the 1 + e^-d in [1, 2] taken by the hardware exp2 / log2 (absolute error
// of the correction term ~1e-7, far below fp32 rounding of the running sums).
// Both -inf: the correction is NaN and the select returns -inf.  A select, not
// a branch, so that independent calls interleave (a branch per call serialises them).
__device__ __forceinline__ float log_add_exp(float a, float b) {
  const float m = fmaxf(a, b);
  const float r = m + __logf(1.f + __expf(-fabsf(a - b)));
  return m == -INFINITY ? m : r;
}

// ---- pairs of fp32 values in one 64-bit register: two operations an instruction
__device__ __forceinline__ uint64_t f2_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 f2_open(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Cluster barrier (release / acquire at cluster scope), in two halves: every
// thread of every block of the cluster makes both.  A block's shared memory may
// be written by the others only after a barrier that it took part in, and each
// such write must be followed by one before the block may exit.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// The address of p's place in the shared memory of block `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cluster(const void* p, int rank) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}

template <typename T> __device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

}  // namespace frnnt
