// Gated linear recurrence h_t = a_t h_{t-1} + (1 - a_t) x_t, a = sigmoid(gate):
// forward over padded sequences, backward, and one step of many hypotheses.
#include <initializer_list>

#include "frnnt_common.cuh"
#include "frnnt_internal.h"
#include "frnnt_ops.h"

namespace frnnt {
namespace {

// A block walks along one sequence, 64 channels wide, kChunk steps at a time.
// Lane l of every warp holds channels 2l and 2l+1 (one 4- or 8-byte access a
// step, 32 lanes side by side); warp w takes the kSteps steps from w * kSteps on.
constexpr int kChunk = FRNNT_SCAN_CHUNK;
constexpr int kSteps = 8;
constexpr int kWarps = kChunk / kSteps;
constexpr int kTile = 64;

// a = sigmoid(gate) and s = 1 - a = sigmoid(-gate), each to relative precision:
// with e = exp(-gate), a = 1 / (1 + e), and s = e a where that is below 1/2 (1 -
// a would lose its digits where the memory is long and a is near 1), 1 - a
// above (where e may be infinite).  The hardware exp2 and reciprocal are good
// to 2^-22, and the rounded exponent adds |gate| 2^-24.
struct Gate {
  float a, s;
};
__device__ __forceinline__ Gate gate_of(float g) {
  float e, a;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(1.f + e));
  return Gate{a, e > 1.f ? 1.f - a : e * a};
}

__device__ __forceinline__ int length_of(const int32_t* lengths, int b, int T, int32_t* status) {
  if (!lengths) return T;
  const int l = lengths[b];
  if ((l < 0 || l > T) && status && threadIdx.x == 0) atomicOr(status, FRNNT_STATUS_LENGTH);
  return clampi(l, 0, T);
}

// Two neighbouring channels as they lie in memory.
template <typename T>
struct Pair;
template <>
struct Pair<float> {
  using Raw = float2;
  static __device__ __forceinline__ float2 open(float2 r) { return r; }
  static __device__ __forceinline__ float2 pack(float a, float b) { return make_float2(a, b); }
  static __device__ __forceinline__ float2 join(float a, float b) { return make_float2(a, b); }
};
template <>
struct Pair<__nv_bfloat16> {
  using Raw = uint32_t;
  static __device__ __forceinline__ float2 open(uint32_t r) {
    return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ uint32_t join(__nv_bfloat16 a, __nv_bfloat16 b) {
    return (uint32_t)__bfloat16_as_ushort(a) | ((uint32_t)__bfloat16_as_ushort(b) << 16);
  }
};

// VEC: every pair is aligned to its size and D is even; otherwise channel by
// channel, `two` telling whether the second exists.
template <typename T, bool VEC>
__device__ __forceinline__ typename Pair<T>::Raw load_pair(const T* p, bool two) {
  using Raw = typename Pair<T>::Raw;
  if (VEC) return __ldg(reinterpret_cast<const Raw*>(p));
  return Pair<T>::join(__ldg(p), two ? __ldg(p + 1) : from_f32<T>(0.f));
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_pair(T* p, float a, float b, bool two) {
  using Raw = typename Pair<T>::Raw;
  if (VEC) {
    *reinterpret_cast<Raw*>(p) = Pair<T>::pack(a, b);
  } else {
    p[0] = from_f32<T>(a);
    if (two) p[1] = from_f32<T>(b);
  }
}

// Writes v to the same shared-memory place of block `rank` of the cluster.
__device__ __forceinline__ void store_cluster(float4* p, float4 v, int rank) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(in_cluster(p, rank)), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}

// Forward.  h_t = a_t h_{t-1} + b_t composes: over a run of steps h_out = A h_in
// + H with A the product of the a and H the run's result from zero.  Each
// warp forms its run's (A, H), the block joins them in shared memory, and
// each warp walks its run again from its true entering state, out of
// registers: x and gate are read once, h written once.  The block carries the
// state from chunk to chunk.  Where there are too few (sequence, channel
// tile) pairs to fill the GPU, CL blocks of a cluster take the chunks in turn
// and tell each other their chunk's (A, H) through distributed shared memory,
// one cluster barrier a round.
template <typename T, bool VEC, int CL>
__global__ void __launch_bounds__(kWarps * 32)
    scan_fwd_kernel(frnnt_recurrence_dims d, const T* __restrict__ x, const T* __restrict__ gate,
                    const int32_t* __restrict__ lengths, const float* __restrict__ h0, T* __restrict__ h,
                    float* __restrict__ h_last, float* __restrict__ saved, int32_t* status) {
  using Raw = typename Pair<T>::Raw;
  __shared__ float4 run[2][kWarps][32];
  __shared__ float4 part[2][CL][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int b = blockIdx.y, rank = CL > 1 ? blockIdx.x % CL : 0;
  const int c = (blockIdx.x / CL) * kTile + 2 * lane;
  const bool live = c < d.D, two = c + 1 < d.D;
  const int len = length_of(lengths, b, d.T, status), nc = (d.T + kChunk - 1) / kChunk;
  const int rounds = ((len + kChunk - 1) / kChunk + CL - 1) / CL;
  const T* xp = x + b * d.x_sb + c;
  const T* gp = gate + b * d.gate_sb + c;
  T* hp = h + b * d.h_sb + c;
  if (CL > 1) cluster_arrive();

  Raw rx[kSteps], rg[kSteps];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      if (live && t0 + i < len) {
        rx[i] = load_pair<T, VEC>(xp + (t0 + i) * d.x_st, two);
        rg[i] = load_pair<T, VEC>(gp + (t0 + i) * d.gate_st, two);
      }
  };
  float2 carry = make_float2(0.f, 0.f);
  if (h0 && live) carry = make_float2(h0[(long long)b * d.D + c], two ? h0[(long long)b * d.D + c + 1] : 0.f);
  int t0 = rank * kChunk + w * kSteps;
  if (rounds > 0) fetch(t0);
  if (CL > 1) cluster_wait();     // the other blocks run: their shared memory may be written from here on
  for (int r = 0; r < rounds; ++r, t0 += CL * kChunk) {
    float2 a[kSteps], v[kSteps];
    float4 m = make_float4(1.f, 0.f, 1.f, 0.f);   // A, H of the two channels
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      a[i] = make_float2(1.f, 1.f);
      v[i] = make_float2(0.f, 0.f);
      if (live && t0 + i < len) {
        const float2 xv = Pair<T>::open(rx[i]), gv = Pair<T>::open(rg[i]);
        const Gate g0 = gate_of(gv.x), g1 = gate_of(gv.y);
        a[i] = make_float2(g0.a, g1.a);
        v[i] = make_float2(g0.s * xv.x, g1.s * xv.y);
      }
      m.x *= a[i].x;
      m.y = fmaf(a[i].x, m.y, v[i].x);
      m.z *= a[i].y;
      m.w = fmaf(a[i].y, m.w, v[i].y);
    }
    if (r + 1 < rounds) fetch(t0 + CL * kChunk);
    run[r & 1][w][lane] = m;
    __syncthreads();
    float4 before = make_float4(1.f, 0.f, 1.f, 0.f), all = before;   // runs before this warp's; the whole chunk
    for (int k = 0; k < nw; ++k) {
      if (k == w) before = all;
      const float4 o = run[r & 1][k][lane];
      all = make_float4(all.x * o.x, fmaf(o.x, all.y, o.y), all.z * o.z, fmaf(o.z, all.w, o.w));
    }
    float2 in = carry;              // the state that enters this block's chunk
    if (CL > 1) {
      if (w < CL) store_cluster(&part[r & 1][rank][lane], all, w);
      cluster_arrive();
      cluster_wait();
#pragma unroll
      for (int k = 0; k < CL; ++k) {
        if (k == rank) in = carry;
        const float4 o = part[r & 1][k][lane];
        carry = make_float2(fmaf(o.x, carry.x, o.y), fmaf(o.z, carry.y, o.w));
      }
    } else {
      carry = make_float2(fmaf(all.x, carry.x, all.y), fmaf(all.z, carry.y, all.w));
    }
    if (saved && w == 0 && live && t0 < len) {
      float* sp = saved + ((long long)b * nc + t0 / kChunk) * d.D + c;
      sp[0] = in.x;
      if (two) sp[1] = in.y;
    }
    float2 s = make_float2(fmaf(before.x, in.x, before.y), fmaf(before.z, in.y, before.w));
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      s = make_float2(fmaf(a[i].x, s.x, v[i].x), fmaf(a[i].y, s.y, v[i].y));
      if (live && t0 + i < d.T) {
        const bool on = t0 + i < len;
        store_pair<T, VEC>(hp + (t0 + i) * d.h_st, on ? s.x : 0.f, on ? s.y : 0.f, two);
      }
    }
  }
  // rows of whole rounds past the sequence
  for (int t = rounds * CL * kChunk + rank * nw + w; t < d.T; t += CL * nw)
    if (live) store_pair<T, VEC>(hp + t * d.h_st, 0.f, 0.f, two);
  if (rank == 0 && w == 0 && live) {
    h_last[(long long)b * d.D + c] = carry.x;
    if (two) h_last[(long long)b * d.D + c + 1] = carry.y;
  }
}

// Backward.  With q_t = a_t g_t, what step t hands to step t-1, q_t = a_t
// (q_{t+1} + dh_t) is the same recurrence run from the end: over a run of
// steps q_out = A q_in + Q with the same A.  The chunk's states are formed
// again from its saved state by the forward composition, in the same exchange,
// so x, gate and dh are read once, dx and dgate written once, and h is not read.
template <typename T, bool VEC, int CL>
__global__ void __launch_bounds__(kWarps * 32)
    scan_bwd_kernel(frnnt_recurrence_dims d, const T* __restrict__ x, const T* __restrict__ gate,
                    const int32_t* __restrict__ lengths, const float* __restrict__ saved, const T* __restrict__ dh,
                    const float* __restrict__ dh_last, T* __restrict__ dx, T* __restrict__ dgate,
                    float* __restrict__ dh0, int32_t* status) {
  using Raw = typename Pair<T>::Raw;
  __shared__ float4 run[2][kWarps][32];    // A, H of the two channels
  __shared__ float2 back[2][kWarps][32];   // Q
  __shared__ float4 part[2][CL][32];       // A, Q of a block's chunk
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int b = blockIdx.y, rank = CL > 1 ? blockIdx.x % CL : 0;
  const int c = (blockIdx.x / CL) * kTile + 2 * lane;
  const bool live = c < d.D, two = c + 1 < d.D;
  const int len = length_of(lengths, b, d.T, status), nc = (d.T + kChunk - 1) / kChunk;
  const int rounds = ((len + kChunk - 1) / kChunk + CL - 1) / CL;
  const T* xp = x + b * d.x_sb + c;
  const T* gp = gate + b * d.gate_sb + c;
  const T* hp = dh + b * d.dh_sb + c;
  T* dxp = dx + b * d.dx_sb + c;
  T* dgp = dgate + b * d.dgate_sb + c;
  if (CL > 1) cluster_arrive();

  Raw rx[kSteps], rg[kSteps], rh[kSteps];
  float2 start = make_float2(0.f, 0.f);
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      if (live && t0 + i < len && t0 >= 0) {
        rx[i] = load_pair<T, VEC>(xp + (t0 + i) * d.x_st, two);
        rg[i] = load_pair<T, VEC>(gp + (t0 + i) * d.gate_st, two);
        rh[i] = load_pair<T, VEC>(hp + (t0 + i) * d.dh_st, two);
      }
    if (live && t0 >= 0 && t0 < len) {
      const float* sp = saved + ((long long)b * nc + t0 / kChunk) * d.D + c;
      start = make_float2(sp[0], two ? sp[1] : 0.f);
    }
  };
  float2 carry = make_float2(0.f, 0.f);
  if (dh_last && live)
    carry = make_float2(dh_last[(long long)b * d.D + c], two ? dh_last[(long long)b * d.D + c + 1] : 0.f);
  // rounds from the end; within a round rank 0 has the latest chunk
  int t0 = (rounds * CL - 1 - rank) * kChunk + w * kSteps;
  if (rounds > 0) fetch(t0);
  if (CL > 1) cluster_wait();
  for (int r = 0; r < rounds; ++r, t0 -= CL * kChunk) {
    float2 a[kSteps], s[kSteps], xv[kSteps], e[kSteps], past[kSteps];
    float4 m = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      a[i] = make_float2(1.f, 1.f);
      s[i] = xv[i] = e[i] = make_float2(0.f, 0.f);
      if (live && t0 + i < len) {
        const float2 gv = Pair<T>::open(rg[i]);
        const Gate g0 = gate_of(gv.x), g1 = gate_of(gv.y);
        a[i] = make_float2(g0.a, g1.a);
        s[i] = make_float2(g0.s, g1.s);
        xv[i] = Pair<T>::open(rx[i]);
        e[i] = Pair<T>::open(rh[i]);
      }
      m.x *= a[i].x;
      m.y = fmaf(a[i].x, m.y, s[i].x * xv[i].x);
      m.z *= a[i].y;
      m.w = fmaf(a[i].y, m.w, s[i].y * xv[i].y);
    }
    float2 q = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = kSteps - 1; i >= 0; --i) q = make_float2(a[i].x * (q.x + e[i].x), a[i].y * (q.y + e[i].y));
    float2 v = start;
    if (r + 1 < rounds) fetch(t0 - CL * kChunk);
    run[r & 1][w][lane] = m;
    back[r & 1][w][lane] = q;
    __syncthreads();
    for (int k = 0; k < w; ++k) {
      const float4 o = run[r & 1][k][lane];
      v = make_float2(fmaf(o.x, v.x, o.y), fmaf(o.z, v.y, o.w));
    }
    float4 before = make_float4(1.f, 0.f, 1.f, 0.f), all = before;   // runs after this warp's; the whole chunk
    for (int k = nw - 1; k >= 0; --k) {
      if (k == w) before = all;
      const float4 o = run[r & 1][k][lane];
      const float2 p = back[r & 1][k][lane];
      all = make_float4(all.x * o.x, fmaf(o.x, all.y, p.x), all.z * o.z, fmaf(o.z, all.w, p.y));
    }
    float2 in = carry;
    if (CL > 1) {
      if (w < CL) store_cluster(&part[r & 1][rank][lane], all, w);
      cluster_arrive();
      cluster_wait();
#pragma unroll
      for (int k = 0; k < CL; ++k) {
        if (k == rank) in = carry;
        const float4 o = part[r & 1][k][lane];
        carry = make_float2(fmaf(o.x, carry.x, o.y), fmaf(o.z, carry.y, o.w));
      }
    } else {
      carry = make_float2(fmaf(all.x, carry.x, all.y), fmaf(all.z, carry.y, all.w));
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      past[i] = make_float2(v.x - xv[i].x, v.y - xv[i].y);
      v = make_float2(fmaf(a[i].x, v.x, s[i].x * xv[i].x), fmaf(a[i].y, v.y, s[i].y * xv[i].y));
    }
    q = make_float2(fmaf(before.x, in.x, before.y), fmaf(before.z, in.y, before.w));
#pragma unroll
    for (int i = kSteps - 1; i >= 0; --i) {
      const float2 g = make_float2(q.x + e[i].x, q.y + e[i].y);
      q = make_float2(a[i].x * g.x, a[i].y * g.y);
      if (live && t0 + i < d.T && t0 >= 0) {
        const bool on = t0 + i < len;
        store_pair<T, VEC>(dxp + (t0 + i) * d.dx_st, on ? s[i].x * g.x : 0.f, on ? s[i].y * g.y : 0.f, two);
        store_pair<T, VEC>(dgp + (t0 + i) * d.dgate_st, on ? q.x * s[i].x * past[i].x : 0.f,
                           on ? q.y * s[i].y * past[i].y : 0.f, two);
      }
    }
  }
  for (int t = rounds * CL * kChunk + rank * nw + w; t < d.T; t += CL * nw)
    if (live) {
      store_pair<T, VEC>(dxp + t * d.dx_st, 0.f, 0.f, two);
      store_pair<T, VEC>(dgp + t * d.dgate_st, 0.f, 0.f, two);
    }
  if (dh0 && rank == 0 && w == 0 && live) {
    dh0[(long long)b * d.D + c] = carry.x;
    if (two) dh0[(long long)b * d.D + c + 1] = carry.y;
  }
}

template <typename T>
__global__ void step_kernel(frnnt_step_dims d, const T* x, const T* gate, const float* state, const int32_t* parent,
                            const uint8_t* advance, T* h, float* new_state, int32_t* status) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  const long long n = blockIdx.y;
  if (c >= d.D) return;
  int from = (int)n;
  if (parent) {
    from = parent[n];
    if ((from < 0 || from >= d.S) && status) atomicOr(status, FRNNT_STATUS_INDEX);
    from = clampi(from, 0, d.S - 1);
  }
  float v = state[(long long)from * d.D + c];
  if (!advance || advance[n]) {
    const Gate g = gate_of(to_f32<T>(gate[n * d.gate_sn + c]));
    v = fmaf(g.a, v, g.s * to_f32<T>(x[n * d.x_sn + c]));
  }
  new_state[n * d.D + c] = v;
  h[n * d.D + c] = from_f32<T>(v);
}

bool dtype_ok(frnnt_dtype t) { return t == FRNNT_F32 || t == FRNNT_BF16; }

constexpr long long kMaxStride = 1LL << 40;

bool in_strides_ok(long long sb, long long st) { return sb >= 0 && st >= 0 && sb <= kMaxStride && st <= kMaxStride; }

// No two of the B x T rows of D elements share an address: sequence-major or
// step-major, with any gaps.
bool out_strides_ok(long long sb, long long st, int B, int T, int D) {
  if (!in_strides_ok(sb, st)) return false;
  const bool seq_major = (T == 1 || st >= D) && (B == 1 || sb >= (long long)(T - 1) * st + D);
  const bool step_major = (B == 1 || sb >= D) && (T == 1 || st >= (long long)(B - 1) * sb + D);
  return seq_major || step_major;
}

int check(const frnnt_recurrence_dims* d, bool bwd) {
  if (!dtype_ok(d->dtype)) return FRNNT_ERR_UNSUPPORTED;
  if (d->B < 1 || d->T < 1 || d->D < 1 || d->B > 65535 || d->T > (1 << 30) || d->D > (1 << 30)) return FRNNT_ERR_DIMS;
  if (!in_strides_ok(d->x_sb, d->x_st) || !in_strides_ok(d->gate_sb, d->gate_st)) return FRNNT_ERR_DIMS;
  if (!bwd && !out_strides_ok(d->h_sb, d->h_st, d->B, d->T, d->D)) return FRNNT_ERR_DIMS;
  if (bwd && (!in_strides_ok(d->dh_sb, d->dh_st) || !out_strides_ok(d->dx_sb, d->dx_st, d->B, d->T, d->D) ||
              !out_strides_ok(d->dgate_sb, d->dgate_st, d->B, d->T, d->D)))
    return FRNNT_ERR_DIMS;
  return FRNNT_OK;
}

bool aligned(const void* p, size_t n) { return (uintptr_t)p % n == 0; }
size_t size_of(frnnt_dtype t) { return t == FRNNT_BF16 ? 2 : 4; }

// Blocks that share a sequence's chunks.
int cluster_of(const frnnt_recurrence_dims& d) {
  const long long tiles = (long long)((d.D + kTile - 1) / kTile) * d.B;
  const int nc = (d.T + kChunk - 1) / kChunk;
  int cl = 1;
  while (cl < 8 && cl < nc && tiles * cl < 148) cl *= 2;
  return cl;
}

template <typename... P, typename... A>
void launch_scan(void (*kernel)(P...), const frnnt_recurrence_dims& d, int cl, cudaStream_t st, A... args) {
  const int warps = d.T < kChunk ? (d.T + kSteps - 1) / kSteps : kWarps;
  const dim3 grid((d.D + kTile - 1) / kTile * cl, d.B);
  launch_k(kernel, grid, dim3(warps * 32), 0, st, cl, args...);
  note_launch();
}

// Pairs of channels can be moved whole.
bool pairs_ok(const frnnt_recurrence_dims& d, std::initializer_list<const void*> ptrs,
              std::initializer_list<long long> strides) {
  if (d.D % 2) return false;
  for (const void* p : ptrs)
    if (!aligned(p, 2 * size_of(d.dtype))) return false;
  for (long long v : strides)
    if (v % 2) return false;
  return true;
}

template <typename T, bool VEC>
void scan_fwd(const frnnt_recurrence_dims& d, const void* x, const void* gate, const int32_t* lengths,
              const float* h0, void* h, float* h_last, float* saved, int32_t* status, cudaStream_t st) {
  auto go = [&](auto kernel, int cl) {
    launch_scan(kernel, d, cl, st, d, (const T*)x, (const T*)gate, lengths, h0, (T*)h, h_last, saved, status);
  };
  switch (cluster_of(d)) {
    case 1: return go(scan_fwd_kernel<T, VEC, 1>, 1);
    case 2: return go(scan_fwd_kernel<T, VEC, 2>, 2);
    case 4: return go(scan_fwd_kernel<T, VEC, 4>, 4);
    default: return go(scan_fwd_kernel<T, VEC, 8>, 8);
  }
}

template <typename T, bool VEC>
void scan_bwd(const frnnt_recurrence_dims& d, const void* x, const void* gate, const int32_t* lengths,
              const float* saved, const void* dh, const float* dh_last, void* dx, void* dgate, float* dh0,
              int32_t* status, cudaStream_t st) {
  auto go = [&](auto kernel, int cl) {
    launch_scan(kernel, d, cl, st, d, (const T*)x, (const T*)gate, lengths, saved, (const T*)dh, dh_last, (T*)dx,
                (T*)dgate, dh0, status);
  };
  switch (cluster_of(d)) {
    case 1: return go(scan_bwd_kernel<T, VEC, 1>, 1);
    case 2: return go(scan_bwd_kernel<T, VEC, 2>, 2);
    case 4: return go(scan_bwd_kernel<T, VEC, 4>, 4);
    default: return go(scan_bwd_kernel<T, VEC, 8>, 8);
  }
}

}  // namespace
}  // namespace frnnt

using namespace frnnt;

extern "C" FRNNT_API int frnnt_recurrence_fwd(const frnnt_recurrence_dims* d, const void* x, const void* gate,
                                              const int32_t* lengths, const float* h0, void* h, float* h_last,
                                              float* saved, int32_t* status, void* stream) {
  if (!d) return FRNNT_ERR_NULL;
  if (const int rc = check(d, false)) return rc;
  if (!x || !gate || !h || !h_last) return FRNNT_ERR_NULL;
  const size_t es = size_of(d->dtype);
  if (!aligned(x, es) || !aligned(gate, es) || !aligned(h, es) || !aligned(lengths, 4) || !aligned(h0, 4) ||
      !aligned(h_last, 4) || !aligned(saved, 4) || !aligned(status, 4))
    return FRNNT_ERR_ALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  cudaGetLastError();   // clear a stale error so it is not reported as ours
  {
    StageScope sc("recurrence_fwd", st);
    const bool vec = pairs_ok(*d, {x, gate, h}, {d->x_sb, d->x_st, d->gate_sb, d->gate_st, d->h_sb, d->h_st});
    const bool bf = d->dtype == FRNNT_BF16;
    (bf ? vec ? scan_fwd<__nv_bfloat16, true> : scan_fwd<__nv_bfloat16, false>
        : vec ? scan_fwd<float, true> : scan_fwd<float, false>)(*d, x, gate, lengths, h0, h, h_last, saved, status, st);
  }
  return cudaGetLastError() == cudaSuccess ? FRNNT_OK : FRNNT_ERR_CUDA;
}

extern "C" FRNNT_API int frnnt_recurrence_bwd(const frnnt_recurrence_dims* d, const void* x, const void* gate,
                                              const int32_t* lengths, const float* saved, const void* dh,
                                              const float* dh_last, void* dx, void* dgate, float* dh0,
                                              int32_t* status, void* stream) {
  if (!d) return FRNNT_ERR_NULL;
  if (const int rc = check(d, true)) return rc;
  if (!x || !gate || !saved || !dh || !dx || !dgate) return FRNNT_ERR_NULL;
  const size_t es = size_of(d->dtype);
  if (!aligned(x, es) || !aligned(gate, es) || !aligned(dh, es) || !aligned(dx, es) || !aligned(dgate, es) ||
      !aligned(lengths, 4) || !aligned(saved, 4) || !aligned(dh_last, 4) || !aligned(dh0, 4) || !aligned(status, 4))
    return FRNNT_ERR_ALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  cudaGetLastError();   // clear a stale error so it is not reported as ours
  {
    StageScope sc("recurrence_bwd", st);
    const bool vec = pairs_ok(*d, {x, gate, dh, dx, dgate},
                              {d->x_sb, d->x_st, d->gate_sb, d->gate_st, d->dh_sb, d->dh_st, d->dx_sb, d->dx_st,
                               d->dgate_sb, d->dgate_st});
    const bool bf = d->dtype == FRNNT_BF16;
    (bf ? vec ? scan_bwd<__nv_bfloat16, true> : scan_bwd<__nv_bfloat16, false>
        : vec ? scan_bwd<float, true> : scan_bwd<float, false>)(*d, x, gate, lengths, saved, dh, dh_last, dx, dgate,
                                                                dh0, status, st);
  }
  return cudaGetLastError() == cudaSuccess ? FRNNT_OK : FRNNT_ERR_CUDA;
}

extern "C" FRNNT_API int frnnt_recurrence_step(const frnnt_step_dims* d, const void* x, const void* gate,
                                               const float* state, const int32_t* parent, const uint8_t* advance,
                                               void* h, float* new_state, int32_t* status, void* stream) {
  if (!d) return FRNNT_ERR_NULL;
  if (!dtype_ok(d->dtype)) return FRNNT_ERR_UNSUPPORTED;
  if (d->N < 1 || d->N > 65535 || d->S < 1 || d->D < 1 || !in_strides_ok(d->x_sn, d->gate_sn) ||
      (!parent && d->N > d->S) || (parent && new_state == state))
    return FRNNT_ERR_DIMS;
  if (!x || !gate || !state || !h || !new_state) return FRNNT_ERR_NULL;
  const size_t es = size_of(d->dtype);
  if (!aligned(x, es) || !aligned(gate, es) || !aligned(h, es) || !aligned(state, 4) || !aligned(parent, 4) ||
      !aligned(new_state, 4) || !aligned(status, 4))
    return FRNNT_ERR_ALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  cudaGetLastError();   // clear a stale error so it is not reported as ours
  {
    StageScope sc("recurrence_step", st);
    const dim3 grid((d->D + 127) / 128, d->N);
    if (d->dtype == FRNNT_BF16)
      step_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(*d, (const __nv_bfloat16*)x, (const __nv_bfloat16*)gate, state,
                                                       parent, advance, (__nv_bfloat16*)h, new_state, status);
    else
      step_kernel<float><<<grid, 128, 0, st>>>(*d, (const float*)x, (const float*)gate, state, parent, advance,
                                               (float*)h, new_state, status);
    note_launch();
  }
  return cudaGetLastError() == cudaSuccess ? FRNNT_OK : FRNNT_ERR_CUDA;
}
