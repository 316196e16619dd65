// Gated linear recurrence h_t = a_t h_{t-1} + (1 - a_t) x_t, a = sigmoid(gate):
// forward over padded sequences, backward, and one step of many hypotheses.
#include "frnnt_common.cuh"
#include "frnnt_internal.h"
#include "frnnt_ops.h"

namespace frnnt {
namespace {

constexpr int kChunk = FRNNT_SCAN_CHUNK;

// a = sigmoid(gate) and s = 1 - a = sigmoid(-gate), each to full relative
// precision (1 - a formed by subtraction would lose the digits of s where the
// memory is long and a is near 1).
struct Gate {
  float a, s;
};
__device__ __forceinline__ Gate gate_of(float g) {
  const float u = expf(-fabsf(g));
  const float big = 1.f / (1.f + u), small = u * big;
  return g >= 0.f ? Gate{big, small} : Gate{small, big};
}

__device__ __forceinline__ int length_of(const int32_t* lengths, int b, int T, int32_t* status) {
  if (!lengths) return T;
  const int l = lengths[b];
  if ((l < 0 || l > T) && status) atomicOr(status, FRNNT_STATUS_LENGTH);
  return clampi(l, 0, T);
}

// A thread per channel, one step after another.
template <typename T>
__global__ void scan_fwd_kernel(frnnt_recurrence_dims d, const T* x, const T* gate, const int32_t* lengths,
                                const float* h0, T* h, float* h_last, float* saved, int32_t* status) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
  if (c >= d.D) return;
  const int len = length_of(lengths, b, d.T, status), nc = (d.T + kChunk - 1) / kChunk;
  float v = h0 ? h0[(long long)b * d.D + c] : 0.f;
  for (int t = 0; t < d.T; ++t) {
    if (saved && t % kChunk == 0) saved[((long long)b * nc + t / kChunk) * d.D + c] = v;
    float o = 0.f;
    if (t < len) {
      const Gate g = gate_of(to_f32<T>(gate[b * d.gate_sb + t * d.gate_st + c]));
      v = fmaf(g.a, v, g.s * to_f32<T>(x[b * d.x_sb + t * d.x_st + c]));
      o = v;
    }
    h[b * d.h_sb + t * d.h_st + c] = from_f32<T>(o);
  }
  h_last[(long long)b * d.D + c] = v;
}

template <typename T>
__global__ void scan_bwd_kernel(frnnt_recurrence_dims d, const T* x, const T* gate, const int32_t* lengths,
                                const float* saved, const T* dh, const float* dh_last, T* dx, T* dgate, float* dh0,
                                int32_t* status) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
  if (c >= d.D) return;
  const int len = length_of(lengths, b, d.T, status), nc = (d.T + kChunk - 1) / kChunk;
  float q = dh_last ? dh_last[(long long)b * d.D + c] : 0.f;
  for (int k = nc - 1; k >= 0; --k) {
    float past[kChunk];
    float v = saved[((long long)b * nc + k) * d.D + c];
    const int t0 = k * kChunk, t1 = min(d.T, t0 + kChunk);
    for (int t = t0; t < t1 && t < len; ++t) {
      past[t - t0] = v;
      const Gate g = gate_of(to_f32<T>(gate[b * d.gate_sb + t * d.gate_st + c]));
      v = fmaf(g.a, v, g.s * to_f32<T>(x[b * d.x_sb + t * d.x_st + c]));
    }
    for (int t = t1 - 1; t >= t0; --t) {
      float ox = 0.f, og = 0.f;
      if (t < len) {
        const Gate g = gate_of(to_f32<T>(gate[b * d.gate_sb + t * d.gate_st + c]));
        const float e = to_f32<T>(dh[b * d.dh_sb + t * d.dh_st + c]) + q;
        ox = e * g.s;
        og = e * (past[t - t0] - to_f32<T>(x[b * d.x_sb + t * d.x_st + c])) * g.a * g.s;
        q = g.a * e;
      }
      dx[b * d.dx_sb + t * d.dx_st + c] = from_f32<T>(ox);
      dgate[b * d.dgate_sb + t * d.dgate_st + c] = from_f32<T>(og);
    }
  }
  if (dh0) dh0[(long long)b * d.D + c] = q;
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
  if (d->B < 1 || d->T < 1 || d->D < 1 || d->B > 65535) return FRNNT_ERR_DIMS;
  if (!in_strides_ok(d->x_sb, d->x_st) || !in_strides_ok(d->gate_sb, d->gate_st)) return FRNNT_ERR_DIMS;
  if (!bwd && !out_strides_ok(d->h_sb, d->h_st, d->B, d->T, d->D)) return FRNNT_ERR_DIMS;
  if (bwd && (!in_strides_ok(d->dh_sb, d->dh_st) || !out_strides_ok(d->dx_sb, d->dx_st, d->B, d->T, d->D) ||
              !out_strides_ok(d->dgate_sb, d->dgate_st, d->B, d->T, d->D)))
    return FRNNT_ERR_DIMS;
  return FRNNT_OK;
}

bool aligned(const void* p, size_t n) { return (uintptr_t)p % n == 0; }
size_t size_of(frnnt_dtype t) { return t == FRNNT_BF16 ? 2 : 4; }

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
    const dim3 grid((d->D + 63) / 64, d->B);
    if (d->dtype == FRNNT_BF16)
      scan_fwd_kernel<__nv_bfloat16><<<grid, 64, 0, st>>>(*d, (const __nv_bfloat16*)x, (const __nv_bfloat16*)gate,
                                                          lengths, h0, (__nv_bfloat16*)h, h_last, saved, status);
    else
      scan_fwd_kernel<float><<<grid, 64, 0, st>>>(*d, (const float*)x, (const float*)gate, lengths, h0, (float*)h,
                                                  h_last, saved, status);
    note_launch();
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
    const dim3 grid((d->D + 63) / 64, d->B);
    if (d->dtype == FRNNT_BF16)
      scan_bwd_kernel<__nv_bfloat16><<<grid, 64, 0, st>>>(
          *d, (const __nv_bfloat16*)x, (const __nv_bfloat16*)gate, lengths, saved, (const __nv_bfloat16*)dh, dh_last,
          (__nv_bfloat16*)dx, (__nv_bfloat16*)dgate, dh0, status);
    else
      scan_bwd_kernel<float><<<grid, 64, 0, st>>>(*d, (const float*)x, (const float*)gate, lengths, saved,
                                                  (const float*)dh, dh_last, (float*)dx, (float*)dgate, dh0, status);
    note_launch();
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
