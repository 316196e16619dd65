// Token log-probabilities of rows of logits: log-softmax values of given
// tokens, entropy, the best alternatives, and the gradient of the logits.
#include <algorithm>
#include <type_traits>

#include "frnnt_common.cuh"
#include "frnnt_internal.h"
#include "frnnt_ops.h"

namespace frnnt {
namespace {

constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;
constexpr int kWarps = 8;    // warps of a block
constexpr int kVecs = 4;     // 16-byte vectors a lane holds at a time: a warp takes 2 KB of a row at once
constexpr unsigned kAll = 0xFFFFFFFFu;
// Exponents are held above this: 2^-160 is 0 in fp32, and 0 times it is 0, where 0 times -inf (a forbidden entry's)
// would be NaN.
constexpr float kFloor = -160.f;

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float at_least(float x, float lo) {   // a NaN stays
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(lo));
  return r;
}

// ------------------------------------------------------------------ rows
// A row as 16-byte vectors between an unaligned head and a tail, each shorter
// than a vector: those of the row itself, or of the row that it is written to.
template <typename T>
struct Row {
  static constexpr int E = 16 / sizeof(T);
  const T* p;
  int head, nvec, tail;
  __device__ __forceinline__ Row(const T* row, int V) : Row(row, V, row) {}
  __device__ __forceinline__ Row(const T* row, int V, const T* to) : p(row) {
    const int off = (int)((uintptr_t)to / sizeof(T) % E);
    head = min(off ? E - off : 0, V);
    nvec = (V - head) / E;
    tail = V - head - nvec * E;
  }
  __device__ __forceinline__ const uint4* vec(int v) const { return reinterpret_cast<const uint4*>(p + head) + v; }
  // Bytes from a 16-byte boundary to the first vector.
  __device__ __forceinline__ int skew() const { return (int)((uintptr_t)(p + head) & 15); }
  // The column of the lane's element of head and tail together, or -1: lanes
  // 0 .. and lanes 8 ..
  __device__ __forceinline__ int edge(int lane) const {
    return lane < 8 ? (lane < head ? lane : -1) : (lane - 8 < tail ? head + nvec * E + lane - 8 : -1);
  }
};

template <typename T>
__device__ __forceinline__ void unpack(uint4 r, float (&f)[16 / sizeof(T)]) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      f[i] = __uint_as_float(u[i]);
    } else {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
}

// ------------------------------------------------------------------ softmax statistics
// s = sum of 2^d and w = sum of 2^d d over the values seen, with d = (z - m)
// log2 e and m the largest of them: lse = m + ln s, and the entropy ln s - ln2 w / s.
struct Stats {
  float m, s, w;
};

__device__ __forceinline__ void rescale(Stats& a, float m) {   // to a reference m >= a.m, not -inf
  const float d = fmaxf((a.m - m) * kLog2e, -1000.f), f = exp2_approx(d);
  a.w = f * fmaf(d, a.s, a.w);
  a.s *= f;
  a.m = m;
}
__device__ __forceinline__ void join(Stats& a, Stats b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) {   // neither has a value (or they hold NaN only)
    a.s += b.s;
    return;
  }
  rescale(a, m);
  rescale(b, m);
  a.s += b.s;
  a.w += b.w;
}
__device__ __forceinline__ void join_warp(Stats& a) {
  float m = a.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
  if (m > -INFINITY) rescale(a, m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a.s += __shfl_xor_sync(kAll, a.s, o);
    a.w += __shfl_xor_sync(kAll, a.w, o);
  }
}

// ------------------------------------------------------------------ best alternatives
// Candidates are ordered by one number: the value's order-preserving image above
// the inverted column, so that equal values rank by column, the lowest first.
// 0 is no candidate.  Wide: any value (NaN ranks below everything), any column.
struct Wide {
  using Key = uint64_t;
  static __device__ __forceinline__ uint32_t image(float v) {
    if (v != v) return 0u;
    const uint32_t b = __float_as_uint(v + 0.f);   // -0 becomes +0: they are equal
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  }
  static __device__ __forceinline__ float value_of(uint32_t k) {
    return k == 0u ? NAN : __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
  }
  static __device__ __forceinline__ Key key(float v, int col) { return ((Key)image(v) << 32) | (uint32_t)~col; }
  static __device__ __forceinline__ float value(Key k) { return value_of((uint32_t)(k >> 32)); }
  static __device__ __forceinline__ int column(Key k) { return (int)~(uint32_t)k; }
};
// Narrow: 16-bit values, columns below 65535, at half the instructions and
// shared memory.
struct Narrow {
  using Key = uint32_t;
  static __device__ __forceinline__ Key key(float v, int col) {
    return (Wide::image(v) & 0xFFFF0000u) | (0xFFFFu - (uint32_t)col);
  }
  static __device__ __forceinline__ float value(Key k) {
    return __uint_as_float(((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k) & 0xFFFF0000u);   // (0: a NaN)
  }
  static __device__ __forceinline__ int column(Key k) { return (int)(0xFFFFu - (k & 0xFFFFu)); }
};

// Descending order across the lanes (bitonic): merges of 2, 4, ... 32 sorted runs.
template <typename Key>
__device__ __forceinline__ Key exchange(Key x, int apart, bool keep_larger) {
  const Key y = __shfl_xor_sync(kAll, x, apart);
  return (x > y) == keep_larger ? x : y;
}
template <typename Key>
__device__ __forceinline__ Key sort_desc(Key x, int lane) {
#pragma unroll
  for (int run = 2; run <= 32; run *= 2)
#pragma unroll
    for (int apart = run / 2; apart > 0; apart /= 2)
      x = exchange(x, apart, ((lane & apart) == 0) == ((lane & run) == 0 || run == 32));
  return x;
}
// The 32 largest of two descending lists, descending.
template <typename Key>
__device__ __forceinline__ Key merge_desc(Key x, Key y, int lane) {
  const Key r = __shfl_xor_sync(kAll, y, 31);   // reversed: the maxima form a bitonic sequence
  x = x > r ? x : r;
#pragma unroll
  for (int apart = 16; apart > 0; apart /= 2) x = exchange(x, apart, (lane & apart) == 0);
  return x;
}

// Candidates wait in shared memory, in any order, until they are placed.
constexpr int kWaitingBytes = 2048;
template <typename Order>
constexpr int kWaiting = kWaitingBytes / (int)sizeof(typename Order::Key);

// A value that at least `top` of the row's elements reach, from 32 lanes' maxima
// of disjoint parts of it: the top-th largest of them, -inf where fewer are
// above it.  Each lane counts the larger ones (in shared memory: `all`, 32
// places of the warp's own).
__device__ __forceinline__ float bound_of(float m, int lane, int top, float* all) {
  all[lane] = m;
  __syncwarp();
  int larger = 0;
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    const float4 o = *reinterpret_cast<const float4*>(all + k);
    larger += (o.x > m) + (o.y > m) + (o.z > m) + (o.w > m);
  }
  const uint32_t kth = __reduce_min_sync(kAll, larger < top ? Wide::image(m) : 0xFFFFFFFFu);
  return Wide::value_of(kth);
}

// ------------------------------------------------------------------ forward
struct FwdParams {
  int N, V, K, top;
  long long ld;
  const int32_t* tokens;
  float *logp, *entropy, *lse, *top_logp;
  int32_t *top_ids, *status;
  float* lse_rest;   // lse where it is not wanted
};

// What a lane holds of a row: kVecs vectors, from vector `base` on, 32 apart.
struct Chunk {
  uint4 v[kVecs];
};
template <typename T>
__device__ __forceinline__ void load_chunk(Chunk& c, const Row<T>& row, int base, int lane) {
  const uint4* q = row.vec(base + lane);
  if (base + 32 * kVecs <= row.nvec) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) c.v[u] = __ldg(q + 32 * u);
  } else {
    const uint32_t none = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;   // -inf
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
      c.v[u] = base + u * 32 + lane < row.nvec ? __ldg(q + 32 * u) : make_uint4(none, none, none, none);
  }
}

// The largest of a vector's elements (a NaN counts as none).
template <typename T>
__device__ __forceinline__ float vector_max(uint4 r) {
  if constexpr (sizeof(T) == 4) {
    return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)), fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
  } else {
    uint32_t a, b;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(r.x), "r"(r.y));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(r.z), "r"(r.w));
    asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    const float lo = __uint_as_float(a << 16), hi = __uint_as_float(a & 0xFFFF0000u);
    return fmaxf(lo, fmaxf(hi, -INFINITY));
  }
}

// The statistics of the first n of a chunk's vectors.  The maximum is taken on
// the packed elements, which are unpacked once, vector by vector.
template <typename T, bool WHOLE>
__device__ __forceinline__ void scan_chunk(const Chunk& c, int n, Stats& st, float (&vmax)[kVecs]) {
  constexpr int E = Row<T>::E;
  float m = -INFINITY;
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    vmax[u] = WHOLE || u < n ? vector_max<T>(c.v[u]) : -INFINITY;
    m = fmaxf(m, vmax[u]);
  }
  const float ref = fmaxf(m, st.m);
  if (ref > st.m) rescale(st, ref);
  // a lane that has seen only -inf (or NaN) sums about 0
  const float at = ref == -INFINITY ? 0.f : -ref;
  const uint64_t at2 = f2_of(at, at), l2e = f2_of(kLog2e, kLog2e);
  uint64_t s2 = f2_of(0.f, 0.f), w2 = s2;
#pragma unroll
  for (int u = 0; u < kVecs; ++u)
    if (WHOLE || u < n) {
      float z[E];
      unpack<T>(c.v[u], z);
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const float2 d = f2_open(f2_mul(f2_add(f2_of(z[i], z[i + 1]), at2), l2e));
        const float d0 = at_least(d.x, kFloor), d1 = at_least(d.y, kFloor);
        const uint64_t e2 = f2_of(exp2_approx(d0), exp2_approx(d1));
        s2 = f2_add(s2, e2);
        w2 = f2_fma(e2, f2_of(d0, d1), w2);
      }
    }
  const float2 s = f2_open(s2), w = f2_open(w2);
  st.s += s.x + s.y;
  st.w += w.x + w.y;

}

// (vmax: the vectors' maxima)
template <typename T>
__device__ __forceinline__ void scan(const Chunk& c, const Row<T>& row, int base, Stats& st, float (&vmax)[kVecs]) {
  if (base + 32 * kVecs <= row.nvec) scan_chunk<T, true>(c, kVecs, st, vmax);
  else scan_chunk<T, false>(c, (row.nvec - base + 31) / 32, st, vmax);
}

// Head and tail: one element a lane (-inf where there is none).
template <typename T>
__device__ __forceinline__ float load_edge(const Row<T>& row, int lane) {
  const int col = row.edge(lane);
  return col >= 0 ? to_f32<T>(__ldg(row.p + col)) : -INFINITY;
}
__device__ __forceinline__ void scan_edge(float z, Stats& st) {
  const float ref = fmaxf(z, st.m);
  if (ref > st.m) rescale(st, ref);
  const float d = at_least((z + (ref == -INFINITY ? 0.f : -ref)) * kLog2e, kFloor), e = exp2_approx(d);
  st.s += e;
  st.w = fmaf(e, d, st.w);
}

// ---- best alternatives of a row
// The scan leaves every lane with the largest of its own elements, so a bound
// on the top-th value costs a few reductions, and only what the lanes hold
// whose largest reaches it is read again (from cache): 32 vectors at a time,
// one a lane, whichever lane had them.  With random rows 32 ln(32 / (32 - top))
// elements reach the bound: 9 for the best 8, 31 for 20.  `put` takes a value
// and its column; `who`: 32 places of the warp's own.
template <typename T, typename Put>
__device__ __forceinline__ void collect_vector(const Row<T>& row, int v, float bound, Put put) {
  constexpr int E = Row<T>::E;
  const uint4 r = __ldg(row.vec(v));
  if (!(vector_max<T>(r) >= bound)) return;
  float z[E];
  unpack<T>(r, z);
  unsigned elems = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) elems |= (unsigned)(z[i] >= bound) << i;
  while (elems) {
    const int i = __ffs(elems) - 1;
    elems &= elems - 1;
    const int word = sizeof(T) == 4 ? i : i >> 1;
    uint32_t y = word == 0 ? r.x : word == 1 ? r.y : word == 2 ? r.z : r.w;
    if (sizeof(T) == 2) y = (i & 1) ? y & 0xFFFF0000u : y << 16;
    put(__uint_as_float(y), row.head + v * E + i);
  }
}
template <typename T, typename Put>
__device__ __forceinline__ void collect(const Row<T>& row, int g, int G, int lane, float most, float bound, float edge,
                                        uint8_t* who, Put put) {
  const unsigned from = __ballot_sync(kAll, most >= bound);
  if (!from) return;
  if (most >= bound) who[__popc(from & ((1u << lane) - 1))] = (uint8_t)lane;
  __syncwarp();
  const int span = 32 * kVecs, first = g * span;
  const int chunks = max(0, (row.nvec - first + G * span - 1) / (G * span));   // of the warp
  const int items = __popc(from) * chunks * kVecs;
  for (int t = lane; t < items; t += 32) {
    const int q = t / kVecs, owner = chunks == 1 ? q : q / chunks;
    const int v = first + (q - owner * chunks) * (G * span) + (t % kVecs) * 32 + who[owner];
    if (v < row.nvec) collect_vector(row, v, bound, put);
  }
  if (g == 0 && edge >= bound && row.edge(lane) >= 0) put(edge, row.edge(lane));
}
// A row of one chunk: its vectors' maxima are still at hand, so only the vectors
// that reach the bound are read again.  `who`: 128 places.
template <typename T, typename Put>
__device__ __forceinline__ void collect_short(const Row<T>& row, int lane, const float (&vmax)[kVecs], float bound,
                                              float edge, uint8_t* who, Put put) {
  static_assert(32 * kVecs <= 128, "a place for each vector, numbered in a byte");
  int items = 0;
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const bool may = vmax[u] >= bound;
    const unsigned from = __ballot_sync(kAll, may);
    if (may) who[items + __popc(from & ((1u << lane) - 1))] = (uint8_t)(u * 32 + lane);
    items += __popc(from);
  }
  __syncwarp();
  for (int t = lane; t < items; t += 32) collect_vector(row, who[t], bound, put);
  if (edge >= bound && row.edge(lane) >= 0) put(edge, row.edge(lane));
}

// Rows that the bound does not thin out (many equal values, or fewer than `top`
// elements above -inf): one warp goes through the row in order, with the list
// of the best so far, which stops later columns of equal value.  Descending,
// one a lane; `buffer`: 64 places.  Latency of a load and a ballot every 32
// columns, 0.27 us: 7 x 131071 bf16 with 5 columns left, or all equal, 1.1 ms (7 us
// where a bound thins the rows out); 64 x 4096 fp32 22 to 25 us (4).
template <typename T>
__device__ __noinline__ uint64_t best_in_order(const T* p, int V, int top, uint64_t* buffer) {
  const int lane = threadIdx.x & 31;
  uint64_t best = 0, last = 0;
  int waiting = 0;
  for (int j = 0; j < V || waiting; j += 32) {
    const uint64_t x = j + lane < V ? Wide::key(to_f32<T>(__ldg(p + j + lane)), j + lane) : 0;
    const unsigned from = __ballot_sync(kAll, x > last);
    if (x > last) buffer[waiting + __popc(from & ((1u << lane) - 1))] = x;
    waiting += __popc(from);
    if (waiting > 32 || (waiting && j + 32 >= V)) {
      __syncwarp();
      best = merge_desc(best, sort_desc(lane < waiting ? buffer[lane] : 0, lane), lane);
      const uint64_t rest = lane + 32 < waiting ? buffer[lane + 32] : 0;
      __syncwarp();
      if (lane + 32 < waiting) buffer[lane] = rest;
      waiting = max(0, waiting - 32);
      last = __shfl_sync(kAll, best, top - 1);
    }
  }
  return best;
}

// A row's values from its joined statistics; ls = ln st.s.  st.s is 0 where
// nothing but -inf was seen.  The sum of m and ls goes out with what rounding
// took from it (the two-sum of Knuth), which is all of ls where m is huge.
__device__ __forceinline__ void write_stats(const FwdParams& p, long long n, const Stats& st, float ls) {
  const bool empty = st.s == 0.f;
  const float lse = st.m + ls, part = lse - st.m;
  const float rest = (st.m - (lse - part)) + (ls - part);
  p.lse_rest[n] = empty ? 0.f : rest;   // (first: its place may be lse's)
  p.lse[n] = empty ? -INFINITY : lse;
  p.entropy[n] = empty ? 0.f : fmaf(st.w / st.s, -kLn2, ls);
}
__device__ __forceinline__ void write_token(const FwdParams& p, long long n, int k, const Stats& st, float ls,
                                            int token, float z) {
  const bool given = token >= 0 && token < p.V;
  if (!given && token != FRNNT_NO_TOKEN && p.status) atomicOr(p.status, FRNNT_STATUS_LABEL);
  p.logp[n * p.K + k] = !given ? 0.f : st.s == 0.f ? -INFINITY : (z - st.m) - ls;
}
template <typename Order>
__device__ __forceinline__ void write_top(const FwdParams& p, long long n, int place, const Stats& st, float ls,
                                          typename Order::Key x) {
  if (place < p.top) {
    p.top_ids[n * p.top + place] = Order::column(x);
    p.top_logp[n * p.top + place] = st.s == 0.f ? -INFINITY : (Order::value(x) - st.m) - ls;
  }
}
// How many of the n candidates (and zeros up to a multiple of 16 bytes) are
// larger than x.
template <typename Key>
__device__ __forceinline__ int larger_than(Key x, const Key* all, int n) {
  constexpr int kAtOnce = 16 / sizeof(Key);
  int larger = 0;
  for (int k = 0; k < n; k += kAtOnce) {
    Key o[kAtOnce];
    *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(all + k);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) larger += o[i] > x;
  }
  return larger;
}
// The row's alternatives from its candidates.  Few: each finds its place by
// counting the larger ones (no step waits for another); more: sorted; too
// many, or no bound: the row in order.
template <typename T, typename Order>
__device__ __forceinline__ void finish_top(const FwdParams& p, long long n, int lane, const Stats& st, float ls,
                                           const T* row, float bound, int found, unsigned char* waiting) {
  using Key = typename Order::Key;
  constexpr int kAtOnce = 16 / sizeof(Key);
  Key* buffer = reinterpret_cast<Key*>(waiting);
  if (bound > -INFINITY && found <= 64) {
    if (lane < kAtOnce - 1) buffer[found + lane] = 0;
    __syncwarp();
    for (int j = lane; j < found; j += 32) {
      const Key x = buffer[j];
      write_top<Order>(p, n, larger_than(x, buffer, found), st, ls, x);
    }
  } else if (bound > -INFINITY && found <= kWaiting<Order>) {
    Key best = 0;
    for (int k = 0; k < found; k += 32) {
      const Key x = sort_desc<Key>(k + lane < found ? buffer[k + lane] : 0, lane);
      best = k ? merge_desc<Key>(best, x, lane) : x;
    }
    write_top<Order>(p, n, lane, st, ls, best);
  } else {
    write_top<Wide>(p, n, lane, st, ls, best_in_order(row, p.V, p.top, reinterpret_cast<uint64_t*>(waiting)));
  }
}

// A warp's share of N rows: warp i of the grid takes rows i N / warps on, so that
// no two differ by more than one row.  `step`: N / warps in 2^-32, rounded up.
struct Share {
  int first, count;
  __device__ __forceinline__ Share(int N, uint64_t step, int w) {
    const uint64_t at = (uint64_t)(blockIdx.x * kWarps + w) * step;
    first = min(N, (int)(at >> 32));
    count = min(N, (int)((at + step) >> 32)) - first;
  }
};

// Rows of a few KB.  One pass over the row with a running maximum and sums in
// fp32.  Bound by latency: 370 instructions a row of 1024 (200 are the elements')
// fill 62 % of the issue slots, the exponentials 46 % of their unit and the loads 40 %
// of DRAM, with 24 warps an SM (80 registers) and 15 dependent shuffles at the end
// of a row.  32400 x 1024 bf16: 18.7 us (3.5 TB/s; with 10
// rows for most warps instead of 9 or 10 for each: 20.3; a warp a row without a
// next one on its way: 31), with the best 8: 37 us, 20: 45 us.
// A warp takes its share of rows, one after another, with the next one's vectors
// on their way.  Lane i keeps row i's joined statistics, so that the logarithms,
// divisions and stores of up to 32 rows are made at once, a lane a row; the
// values of their first tokens are fetched before the rows are scanned.
constexpr int kEarly = 2;
template <typename T, bool TOP>
__global__ void __launch_bounds__(kWarps * 32, 3)
    logprob_warp_kernel(FwdParams p, uint64_t step, const T* __restrict__ logits) {
  using Order = std::conditional_t<sizeof(T) == 2, Narrow, Wide>;   // (its rows are shorter than 65535)
  __shared__ __align__(16) unsigned char waiting[TOP ? kWarps : 1][kWaitingBytes];
  __shared__ int counts[kWarps];
  __shared__ uint8_t who[kWarps][32 * kVecs];
  __shared__ __align__(16) float maxima[kWarps][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const Share rows(p.N, step, w);
  if (!rows.count) return;
  const long long n0 = rows.first;
  const int count = rows.count;
  Chunk next;
  Row<T> row(logits + n0 * p.ld, p.V);
  load_chunk(next, row, 0, lane);
  float edge = row.head + row.tail ? load_edge(row, lane) : -INFINITY;

  const long long mine = n0 + lane;   // the row that this lane finishes
  const bool have = lane < count;
  int token[kEarly];
  float zt[kEarly];
#pragma unroll
  for (int k = 0; k < kEarly; ++k) token[k] = have && k < p.K ? p.tokens[mine * p.K + k] : FRNNT_NO_TOKEN;
#pragma unroll
  for (int k = 0; k < kEarly; ++k)
    zt[k] = token[k] >= 0 && token[k] < p.V ? to_f32<T>(__ldg(logits + mine * p.ld + token[k])) : 0.f;

  Stats kept{0.f, 0.f, 0.f};
  for (int i = 0; i < count; ++i) {
    Stats st{-INFINITY, 0.f, 0.f};
    float vmax[kVecs] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    const Row<T> here = row;
    const float z = edge;
    if (i + 1 < count) row = Row<T>(logits + (n0 + i + 1) * p.ld, p.V);
    for (int base = 0;; base += 32 * kVecs) {
      const Chunk c = next;
      const bool last = base + 32 * kVecs >= here.nvec;
      if (!last) {
        load_chunk(next, here, base + 32 * kVecs, lane);
      } else if (i + 1 < count) {
        load_chunk(next, row, 0, lane);
        edge = row.head + row.tail ? load_edge(row, lane) : -INFINITY;
      }
      if (here.nvec) scan<T>(c, here, base, st, vmax);
      if (last) break;
    }
    if (here.head + here.tail) scan_edge(z, st);
    const float most = st.m;   // of this lane's elements
    join_warp(st);
    if (lane == i) kept = st;
    if constexpr (TOP) {
      const float bound = bound_of(most, lane, p.top, maxima[w]);
      if (lane == 0) counts[w] = 0;
      __syncwarp();
      auto put = [&](float v, int col) {
        const int at = atomicAdd(&counts[w], 1);
        if (at < kWaiting<Order>) reinterpret_cast<typename Order::Key*>(waiting[w])[at] = Order::key(v, col);
      };
      if (bound > -INFINITY) {
        if (here.nvec <= 32 * kVecs) collect_short(here, lane, vmax, bound, z, who[w], put);
        else collect(here, 0, 1, lane, most, bound, z, who[w], put);
      }
      __syncwarp();
      finish_top<T, Order>(p, n0 + i, lane, st, logf(st.s), here.p, bound, counts[w], waiting[w]);
      __syncwarp();
    }
  }
  if (!have) return;
  const float ls = logf(kept.s);
  write_stats(p, mine, kept, ls);
#pragma unroll
  for (int k = 0; k < kEarly; ++k)
    if (k < p.K) write_token(p, mine, k, kept, ls, token[k], zt[k]);
  for (int k = kEarly; k < p.K; ++k) {
    const int t = p.tokens[mine * p.K + k];
    write_token(p, mine, k, kept, ls, t, t >= 0 && t < p.V ? to_f32<T>(__ldg(logits + mine * p.ld + t)) : 0.f);
  }
}

// Short rows, where a warp a row would leave most lanes idle: G lanes a row, each
// with C of its columns, G apart, element by element (any alignment; a warp's
// rows lie next to each other, so its accesses cover whole sectors all the same).
// Everything is in registers: bound by the instructions of each element.  60000
// x 128 bf16: 10.7 us (1.4 TB/s), x 24: 3.5 us.  A candidate for the alternatives
// finds its place by counting the larger ones: of the whole row, or, with a warp
// a row, of what reaches the bound.
template <typename T, int G, int C, bool TOP>
__global__ void __launch_bounds__(kWarps * 32) logprob_few_kernel(FwdParams p, const T* __restrict__ logits) {
  using Order = std::conditional_t<sizeof(T) == 2, Narrow, Wide>;
  using Key = typename Order::Key;
  constexpr int kRows = 32 / G, kAtOnce = 16 / sizeof(Key);
  __shared__ __align__(16) Key all[TOP ? kWarps * kRows : 1][G * C + kAtOnce];   // (rows apart in the banks)
  __shared__ __align__(16) float maxima[TOP && G == 32 ? kWarps : 1][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane % G;
  const long long first = ((long long)blockIdx.x * kWarps + w) * kRows;
  if (first >= p.N) return;
  const bool have = first + lane / G < p.N;
  const long long n = have ? first + lane / G : p.N - 1;
  const T* const row = logits + n * p.ld;
  const int token = g < p.K ? p.tokens[n * p.K + g] : FRNNT_NO_TOKEN;
  float z[C];
#pragma unroll
  for (int e = 0; e < C; ++e) z[e] = g + G * e < p.V ? to_f32<T>(__ldg(row + g + G * e)) : -INFINITY;
  const float zt = token >= 0 && token < p.V ? to_f32<T>(__ldg(row + token)) : 0.f;

  Stats st{-INFINITY, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < C; ++e) st.m = fmaxf(st.m, z[e]);
  const float most = st.m;   // of this lane's elements
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) st.m = fmaxf(st.m, __shfl_xor_sync(kAll, st.m, o));
  const float ref = st.m == -INFINITY ? 0.f : st.m;
#pragma unroll
  for (int e = 0; e < C; ++e) {
    const float d = at_least((z[e] - ref) * kLog2e, kFloor), x = exp2_approx(d);
    st.s += x;
    st.w = fmaf(x, d, st.w);
  }
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) {
    st.s += __shfl_xor_sync(kAll, st.s, o);
    st.w += __shfl_xor_sync(kAll, st.w, o);
  }
  const float ls = logf(st.s);
  if (have) {
    if (g == 0) write_stats(p, n, st, ls);
    if (g < p.K) write_token(p, n, g, st, ls, token, zt);
    for (int k = g + G; k < p.K; k += G) {
      const int t = p.tokens[n * p.K + k];
      write_token(p, n, k, st, ls, t, t >= 0 && t < p.V ? to_f32<T>(__ldg(row + t)) : 0.f);
    }
  }
  if constexpr (TOP) {
    Key* const mine = all[w * kRows + lane / G];
    const float bound = G == 32 ? bound_of(most, lane, p.top, maxima[w]) : -INFINITY;
    if (bound > -INFINITY) {
      int found = 0;
#pragma unroll
      for (int e = 0; e < C; ++e) {
        const bool may = z[e] >= bound;   // (no column behind the last: those are -inf)
        const unsigned from = __ballot_sync(kAll, may);
        if (may) mine[found + __popc(from & ((1u << lane) - 1))] = Order::key(z[e], g + G * e);
        found += __popc(from);
      }
      if (lane < kAtOnce - 1) mine[found + lane] = 0;
      __syncwarp();
      for (int j = lane; j < found; j += 32) {
        const Key x = mine[j];
        write_top<Order>(p, n, larger_than(x, mine, found), st, ls, x);
      }
    } else {
      Key key[C];
      int place[C] = {};
#pragma unroll
      for (int e = 0; e < C; ++e) mine[g + G * e] = key[e] = g + G * e < p.V ? Order::key(z[e], g + G * e) : 0;
      __syncwarp();
      for (int k = 0; k < p.V; k += kAtOnce) {
        Key o[kAtOnce];
        *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(mine + k);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
          for (int e = 0; e < C; ++e) place[e] += o[i] > key[e];
      }
#pragma unroll
      for (int e = 0; e < C; ++e)
        if (have && g + G * e < p.V) write_top<Order>(p, n, place[e], st, ls, key[e]);
    }
  }
}

// Long rows, and few.  8190 x 32768 bf16: 91 us (5.9 TB/s; the exponentials'
// unit is busy 70 % of the time); 7 x 131071 bf16 with the best 20: 7.2 us in
// clusters of 8 blocks, most of it launch, cluster barriers and the final sort.
// A cluster of CL blocks of W warps a row.  One block: it takes rows in turn, with the
// next row's vectors on their way.  The warps' statistics (and the maxima of the
// lanes, over the warps) meet in shared memory, in every block of a cluster;
// one warp, another each row, finishes the row.  What meets has two places, so
// that the next row's can be put down while this one's are read.
template <int SHARE>
struct Meeting {
  Stats stats[SHARE];
  float most[SHARE][32];
  __align__(16) unsigned char waiting[kWaitingBytes];
  int count;
};
template <typename T, bool TOP, int CL, int W>
__global__ void __launch_bounds__(W * 32, 24 / W) logprob_block_kernel(FwdParams p, const T* __restrict__ logits) {
  constexpr int kShare = W * CL, kStride = kShare * 32 * kVecs;
  __shared__ Meeting<kShare> meetings[CL > 1 ? 1 : 2];
  __shared__ uint8_t who[W][32];
  __shared__ __align__(16) float maxima[W][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int rank = CL > 1 ? blockIdx.x % CL : 0, g = rank * W + w;
  if (CL > 1) cluster_arrive();
  const long long step = CL > 1 ? p.N : gridDim.x;   // a cluster takes one row
  long long n = blockIdx.x / CL;
  Chunk next;
  Row<T> row(logits + n * p.ld, p.V);
  if (g * 32 * kVecs < row.nvec) load_chunk(next, row, g * 32 * kVecs, lane);
  float edge = g == 0 && row.head + row.tail ? load_edge(row, lane) : -INFINITY;
  if (threadIdx.x == 0)
    for (Meeting<kShare>& m : meetings) m.count = 0;
  __syncthreads();
  for (int i = 0; n < p.N; ++i, n += step) {
    Meeting<kShare>& meet = meetings[CL > 1 ? 0 : i & 1];
    const int writer = CL > 1 ? 0 : i % W;
    int token = FRNNT_NO_TOKEN;
    float zt = 0.f;
    if (g == writer) {
      if (lane < p.K) token = p.tokens[n * p.K + lane];
      if (token >= 0 && token < p.V) zt = to_f32<T>(__ldg(row.p + token));
    }
    Stats st{-INFINITY, 0.f, 0.f};
    const Row<T> here = row;
    const float z = edge;
    const bool more = n + step < p.N;
    if (more) row = Row<T>(logits + (n + step) * p.ld, p.V);
    for (int base = g * 32 * kVecs;; base += kStride) {
      const Chunk c = next;
      if (base + kStride < here.nvec) {
        load_chunk(next, here, base + kStride, lane);
      } else if (more) {
        if (g * 32 * kVecs < row.nvec) load_chunk(next, row, g * 32 * kVecs, lane);
        edge = g == 0 && row.head + row.tail ? load_edge(row, lane) : -INFINITY;
      }
      float vmax[kVecs];
      if (base < here.nvec) scan<T>(c, here, base, st, vmax);
      if (base + kStride >= here.nvec) break;
    }
    if (g == 0 && here.head + here.tail) scan_edge(z, st);
    const float most = st.m;   // of this lane's elements
    join_warp(st);
    if (CL > 1) {
      cluster_wait();   // all blocks run: their shared memory may be written
      if (lane < (TOP ? CL : 1)) {
        const uint32_t at = in_cluster(&meet.stats[g], lane);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(st.m) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 4), "f"(st.s) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 8), "f"(st.w) : "memory");
      }
      if constexpr (TOP)
        for (int k = 0; k < CL; ++k)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(in_cluster(&meet.most[g][lane], k)), "f"(most) : "memory");
      cluster_arrive();
      cluster_wait();
      if (!TOP && rank != 0) return;
    } else {
      if (lane == 0) meet.stats[g] = st;
      if constexpr (TOP) meet.most[g][lane] = most;
      __syncthreads();
    }
    float bound = -INFINITY;
    if constexpr (TOP) {
      float m = -INFINITY;
#pragma unroll 8
      for (int k = 0; k < kShare; ++k) m = fmaxf(m, meet.most[k][lane]);
      bound = bound_of(m, lane, p.top, maxima[w]);
      if (bound > -INFINITY)
        collect(here, g, kShare, lane, most, bound, z, who[w], [&](float v, int col) {
          const uint64_t x = Wide::key(v, col);
          if constexpr (CL > 1) {
            uint32_t at;
            asm volatile("atom.shared::cluster.add.u32 %0, [%1], 1;"
                         : "=r"(at)
                         : "r"(in_cluster(&meet.count, 0))
                         : "memory");
            if (at < kWaiting<Wide>)
              asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(in_cluster(meet.waiting, 0) + 8 * at), "l"(x)
                           : "memory");
          } else {
            const int at = atomicAdd(&meet.count, 1);
            if (at < kWaiting<Wide>) reinterpret_cast<uint64_t*>(meet.waiting)[at] = x;
          }
        });
      if (CL > 1) {
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
      } else {
        __syncthreads();
      }
    }
    if (w == writer) {
      st = lane < kShare ? meet.stats[lane] : Stats{-INFINITY, 0.f, 0.f};
#pragma unroll
      for (int k = 32; k < kShare; k += 32) join(st, meet.stats[k + lane]);
      join_warp(st);
      const float ls = logf(st.s);
      if (lane == 0) write_stats(p, n, st, ls);
      if (lane < p.K) write_token(p, n, lane, st, ls, token, zt);
      if constexpr (TOP) {
        finish_top<T, Wide>(p, n, lane, st, ls, here.p, bound, meet.count, meet.waiting);
        __syncwarp();
        if (lane == 0) meet.count = 0;
      }
    }
  }
}

// ------------------------------------------------------------------ backward
struct BwdParams {
  int N, V, K, top;
  int segments, share;     // warps that share a row, vectors that one of them takes
  long long ld, ldd;
  const int32_t *tokens, *top_ids;
  const float *lse, *entropy, *dlogp, *dentropy, *dtop;
  int32_t* status;
  const float* lse_rest;   // lse, with a factor of 0, where there is none
  float rest_factor;       // else -log2 e
};

template <typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[16 / sizeof(T)]) {
  uint4 r;
  if constexpr (sizeof(T) == 4) {
    r = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  } else {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    r = make_uint4(u[0], u[1], u[2], u[3]);
  }
  *reinterpret_cast<uint4*>(p) = r;
}

// The gradient of a row: dz_j = p_j (A + B log2 p_j) with -A = sum of the
// coefficients + dentropy entropy and -B = dentropy ln2, plus the coefficients
// of column j.  With d_j = (z_j - l) log2 e, l the log-sum-exp rounded to fp32, and c
// what rounding took from it, log2 p_j = d_j + c: without c an offset of all
// logits, |l| 2^-24, would be an error of every p (and p = 1 in a row of the type's
// lowest value).  dz_j = 2^d_j 2^c (A + B c + B d_j) costs nothing an element.
struct Slope {
  float l, A, B;
  static __device__ __forceinline__ Slope of(float l, float c, float A, float B) {
    const float f = exp2_approx(c);
    return Slope{l, f * fmaf(B, c, A), f * B};
  }
  __device__ __forceinline__ float at(float z) const {
    const float d = at_least((z - l) * kLog2e, kFloor);
    return exp2_approx(d) * fmaf(B, d, A);
  }
  template <typename T>
  __device__ __forceinline__ void vector(uint4 raw, T* to) const {
    constexpr int E = 16 / sizeof(T);
    const uint64_t l2 = f2_of(-l, -l), l2e = f2_of(kLog2e, kLog2e), A2 = f2_of(A, A), B2 = f2_of(B, B);
    float f[E];
    unpack<T>(raw, f);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float2 d = f2_open(f2_mul(f2_add(f2_of(f[i], f[i + 1]), l2), l2e));
      const float d0 = at_least(d.x, kFloor), d1 = at_least(d.y, kFloor);
      const float2 g = f2_open(f2_mul(f2_of(exp2_approx(d0), exp2_approx(d1)), f2_fma(B2, f2_of(d0, d1), A2)));
      f[i] = g.x;
      f[i + 1] = g.y;
    }
    store_vec<T>(to, f);
  }
  // kVecs vectors of a lane, 32 apart, those below n
  template <typename T>
  __device__ __forceinline__ void chunk(const uint4 (&raw)[kVecs], T* to, int n) const {
    if (n >= 32 * (kVecs - 1) + 1) {
#pragma unroll
      for (int u = 0; u < kVecs; ++u) vector<T>(raw[u], to + 32 * u * (16 / (int)sizeof(T)));
    } else {
#pragma unroll
      for (int u = 0; u < kVecs; ++u)
        if (32 * u < n) vector<T>(raw[u], to + 32 * u * (16 / (int)sizeof(T)));
    }
  }
};
__device__ __forceinline__ float rest_of(const BwdParams& p, long long n) { return p.rest_factor * p.lse_rest[n]; }
// A lane's vectors, 32 apart, of a warp's share [base, end) of a row.  SKEW: rows
// may start elsewhere in their 16 bytes than the gradient's.  Then vector v of 16-
// bit elements lies in two aligned ones, v and v + 1 (both hold some of the row);
// a lane loads the first of each and shifts it together with the next lane's
// (8190 x 32768: 202 us; stored element by element instead: 669, aligned: 169).
// Of 32-bit elements, it loads the four (333 us; shifted: 358, aligned: 326).
// (plain loads: dlogits may be the logits' memory, and non-coherent ones are for memory that the kernel does not write)
template <bool SKEW>
struct Vecs {
  uint4 raw[kVecs];
  template <typename T>
  static __device__ __forceinline__ const uint4* aligned(const Row<T>& row, int skew) {
    return reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(row.p + row.head) - skew);
  }
  template <typename T>
  __device__ __forceinline__ void load(const Row<T>& row, int base, int end, int lane) {
    constexpr bool kShift = SKEW && sizeof(T) == 2;
    if (base >= end) return;
    if (SKEW && !kShift && row.skew()) {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(row.p + row.head) + 4 * (base + lane);
#pragma unroll
      for (int u = 0; u < kVecs; ++u, src += 128)
        if (32 * u < end - base - lane) raw[u] = make_uint4(src[0], src[1], src[2], src[3]);
      return;
    }
    const int skew = kShift ? row.skew() : 0, n = end - base - lane + (skew != 0);
    const uint4* src = aligned(row, skew) + base + lane;
    if (n >= 32 * (kVecs - 1) + 1) {
#pragma unroll
      for (int u = 0; u < kVecs; ++u) raw[u] = src[32 * u];
    } else {
#pragma unroll
      for (int u = 0; u < kVecs; ++u)
        if (32 * u < n) raw[u] = src[32 * u];
    }
  }
  // The vectors from the aligned ones: each with the next lane's, shifted (the
  // last lane's next one is lane 0's next, or loaded).
  template <typename T>
  __device__ __forceinline__ void shift(const Row<T>& row, int base, int end, int lane) {
    constexpr bool kShift = SKEW && sizeof(T) == 2;
    const int skew = kShift ? row.skew() : 0;
    if (skew == 0) return;
    uint4 behind = make_uint4(0u, 0u, 0u, 0u);
    if (lane == 0 && base + 32 * kVecs <= end) behind = aligned(row, skew)[base + 32 * kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const uint4 after = u + 1 < kVecs ? raw[u + 1] : behind;
      uint32_t w[8] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      w[4] = __shfl_sync(kAll, lane == 0 ? after.x : w[0], (lane + 1) & 31);
      w[5] = __shfl_sync(kAll, lane == 0 ? after.y : w[1], (lane + 1) & 31);
      w[6] = __shfl_sync(kAll, lane == 0 ? after.z : w[2], (lane + 1) & 31);
      w[7] = __shfl_sync(kAll, lane == 0 ? after.w : w[3], (lane + 1) & 31);
#pragma unroll
      for (int i = 0; i < 6; ++i) w[i] = (skew & 8) ? w[i + 2] : w[i];
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = (skew & 4) ? w[i + 1] : w[i];
      const int half = (skew & 2) * 8;
      raw[u] = make_uint4(__funnelshift_r(w[0], w[1], half), __funnelshift_r(w[1], w[2], half),
                          __funnelshift_r(w[2], w[3], half), __funnelshift_r(w[3], w[4], half));
    }
  }
};

// Bound by memory: a row is read and its gradient written.  32400 x 1024 bf16:
// 23.7 us (5.6 TB/s; a warp a row with its scalars loaded row by row: 34 us).
// Rows of a few KB with few coefficients: a warp takes its share of rows, one
// after another, with the next one's vectors on their way.  Lane i prepares row i's slope
// (the loads of up to 32 rows' scalars at once) and, when all rows are
// written, writes the columns of its tokens again.  Every element is read
// before it is written, by the same warp, so dlogits may be the logits' memory.
constexpr int kSlots = 4;
template <typename T, bool SKEW>
__global__ void __launch_bounds__(kWarps * 32, SKEW && sizeof(T) == 2 ? 2 : 3)
    logprob_bwd_rows_kernel(BwdParams p, uint64_t step, const T* logits, T* dlogits) {
  constexpr int E = Row<T>::E;
  const int lane = threadIdx.x & 31;
  const Share rows(p.N, step, threadIdx.x >> 5);
  if (!rows.count) return;
  const long long n0 = rows.first;
  const int count = rows.count;
  Row<T> row(logits + n0 * p.ld, p.V, dlogits + n0 * p.ldd);
  Vecs<SKEW> next;
  next.load(row, 0, row.nvec, lane);
  float edge = row.edge(lane) >= 0 ? to_f32<T>(row.p[row.edge(lane)]) : 0.f;

  const long long mine = n0 + lane;
  const int nk = p.dlogp ? p.K : 0, slots = nk + (p.dtop ? p.top : 0);   // at most kSlots
  int id[kSlots];
  float coef[kSlots], zt[kSlots], sum = 0.f;
  Slope own{-INFINITY, 0.f, 0.f};
  if (lane < count) {
    const float de = p.dentropy ? p.dentropy[mine] : 0.f, h = p.dentropy ? p.entropy[mine] : 0.f;
    bool any = p.dentropy != nullptr;
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      id[k] = -1;
      coef[k] = zt[k] = 0.f;
      if (k < slots) {
        const int t = k < nk ? p.tokens[mine * p.K + k] : p.top_ids[mine * p.top + k - nk];
        if (t >= 0 && t < p.V) {
          id[k] = t;
          coef[k] = k < nk ? p.dlogp[mine * p.K + k] : p.dtop[mine * p.top + k - nk];
          zt[k] = to_f32<T>(logits[mine * p.ld + t]);
          any = true;
        } else if (!(k < nk && t == FRNNT_NO_TOKEN) && p.status) {
          atomicOr(p.status, FRNNT_STATUS_LABEL);
        }
      }
      sum += coef[k];
    }
    if (any) own = Slope::of(p.lse[mine], rest_of(p, mine), -fmaf(de, h, sum), -de * kLn2);
  }
  for (int i = 0; i < count; ++i) {
    const Slope g{__shfl_sync(kAll, own.l, i), __shfl_sync(kAll, own.A, i), __shfl_sync(kAll, own.B, i)};
    const Row<T> here = row;
    T* const out = dlogits + (n0 + i) * p.ldd;
    T* const body = out + here.head;
    const float z = edge;
    const int col = here.edge(lane);
    if (i + 1 < count) row = Row<T>(logits + (n0 + i + 1) * p.ld, p.V, dlogits + (n0 + i + 1) * p.ldd);
    for (int base = lane;; base += 32 * kVecs) {
      Vecs<SKEW> now = next;
      const bool last = base - lane + 32 * kVecs >= here.nvec;
      if (!last) {
        next.load(here, base - lane + 32 * kVecs, here.nvec, lane);
      } else if (i + 1 < count) {
        next.load(row, 0, row.nvec, lane);
        if (row.edge(lane) >= 0) edge = to_f32<T>(row.p[row.edge(lane)]);
      }
      T* to = body + (long long)base * E;
      if (g.l != -INFINITY) {
        now.shift(here, base - lane, here.nvec, lane);
        g.chunk<T>(now.raw, to, here.nvec - base);
      } else {   // a row without any term, or with nothing left by its mask, gets zeros
        const float zero[E] = {};
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
          if (base + 32 * u < here.nvec) store_vec<T>(to + 32 * u * E, zero);
      }
      if (last) break;
    }
    if (col >= 0) out[col] = from_f32<T>(g.l == -INFINITY ? 0.f : g.at(z));
  }
  __syncwarp();   // the dense part of all rows is written
  if (lane < count && own.l != -INFINITY) {
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      float total = 0.f;   // of all slots with the same column
#pragma unroll
      for (int j = 0; j < kSlots; ++j) total += id[j] == id[k] ? coef[j] : 0.f;
      if (id[k] >= 0) dlogits[mine * p.ldd + id[k]] = from_f32<T>(own.at(zt[k]) + total);
    }
  }
}

// Short rows: G lanes a row, as in the forward pass.  Every lane goes through the
// row's coefficients and adds up those of its own columns, so no column is
// written twice and every element is read and written by one lane (dlogits may be
// the logits' memory).  Bound by latency and instructions (70 % of the issue slots,
// loads awaited): five blocks an SM, 60000 x 128 bf16, two tokens and the entropy:
// 16.1 us (of the form before: four 18.3, five 16.0, six 16.7), x 24: 4.8.
template <typename T, int G, int C>
__global__ void __launch_bounds__(kWarps * 32, 5) logprob_bwd_few_kernel(BwdParams p, const T* logits, T* dlogits) {
  const int lane = threadIdx.x & 31, g = lane % G;
  const long long n = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * (32 / G) + lane / G;
  if (n >= p.N) return;   // (no lane waits for another)
  const T* const row = logits + n * p.ld;
  T* const out = dlogits + n * p.ldd;
  float z[C], total[C] = {}, sum = 0.f;
#pragma unroll
  for (int e = 0; e < C; ++e) z[e] = g + G * e < p.V ? to_f32<T>(row[g + G * e]) : 0.f;
  const float l = p.lse[n], de = p.dentropy ? p.dentropy[n] : 0.f, h = p.dentropy ? p.entropy[n] : 0.f;
  const float c = rest_of(p, n);
  bool any = p.dentropy != nullptr;
  const int nk = p.dlogp ? p.K : 0, slots = nk + (p.dtop ? p.top : 0);
#pragma unroll 2
  for (int k = 0; k < slots; ++k) {
    const int t = k < nk ? p.tokens[n * p.K + k] : p.top_ids[n * p.top + k - nk];
    const float x = k < nk ? p.dlogp[n * p.K + k] : p.dtop[n * p.top + k - nk];
    if (t >= 0 && t < p.V) {
      sum += x;
      any = true;
#pragma unroll
      for (int e = 0; e < C; ++e) total[e] += t == g + G * e ? x : 0.f;
    } else if (g == 0 && !(k < nk && t == FRNNT_NO_TOKEN) && p.status) {
      atomicOr(p.status, FRNNT_STATUS_LABEL);
    }
  }
  const float A = -fmaf(de, h, sum), B = -de * kLn2;   // (few columns a lane: see Slope)
#pragma unroll
  for (int e = 0; e < C; ++e) {   // a row without any term, or with nothing left by its mask, gets zeros
    const float d = at_least(fmaf(z[e] - l, kLog2e, c), kFloor);
    if (g + G * e < p.V)
      out[g + G * e] = from_f32<T>(!any || l == -INFINITY ? 0.f : fmaf(exp2_approx(d), fmaf(B, d, A), total[e]));
  }
}

// Any row: `segments` warps share it (no reduction: each needs the row's scalars
// only), of 16 KB each, or less where there are few (54 x 6769 bf16: 3.3 us; with
// 16 KB: 7.2).  8190 x 32768 bf16: 169 us (6.4 TB/s, the copy rate).  The columns
// with coefficients are written again by the warp that wrote them, a lane two
// slots.
template <typename T, bool SKEW>
__global__ void __launch_bounds__(kWarps * 32) logprob_bwd_kernel(BwdParams p, const T* logits, T* dlogits) {
  constexpr int E = Row<T>::E;
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long n = unit / p.segments;
  const int seg = (int)(unit - n * p.segments);
  if (n >= p.N) return;
  T* out = dlogits + n * p.ldd;
  const Row<T> row(logits + n * p.ld, p.V, out);
  const int v0 = seg * p.share, v1 = min(row.nvec, v0 + p.share);

  // coefficients: slots lane and lane + 32 of the given tokens and the alternatives
  const int nk = p.dlogp ? p.K : 0, count = nk + (p.dtop ? p.top : 0);
  int id[2];
  float coef[2], zt[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = lane + 32 * i;
    id[i] = -1;
    coef[i] = zt[i] = 0.f;
    if (k < count) {
      const int t = k < nk ? p.tokens[n * p.K + k] : p.top_ids[n * p.top + k - nk];
      if (t >= 0 && t < p.V) {
        id[i] = t;
        coef[i] = k < nk ? p.dlogp[n * p.K + k] : p.dtop[n * p.top + k - nk];
        zt[i] = to_f32<T>(row.p[t]);
      } else if (!(k < nk && t == FRNNT_NO_TOKEN) && p.status) {
        atomicOr(p.status, FRNNT_STATUS_LABEL);
      }
    }
  }
  const float l = p.lse[n], de = p.dentropy ? p.dentropy[n] : 0.f, h = p.dentropy ? p.entropy[n] : 0.f;
  const float c = rest_of(p, n);
  float sum = coef[0] + coef[1];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  float total[2] = {0.f, 0.f};   // of all slots with the same column
  for (int k = 0; k < count; ++k) {
    const int t = __shfl_sync(kAll, k < 32 ? id[0] : id[1], k & 31);
    const float x = __shfl_sync(kAll, k < 32 ? coef[0] : coef[1], k & 31);
    if (t == id[0]) total[0] += x;
    if (t == id[1]) total[1] += x;
  }
  // a row without any term, or with nothing left by its mask, gets zeros
  const bool none = l == -INFINITY || (!p.dentropy && !__any_sync(kAll, id[0] >= 0 || id[1] >= 0));
  const Slope g = Slope::of(l, c, -fmaf(de, h, sum), -de * kLn2);
  auto patch = [&](int lo, int hi) {   // columns lo .. hi - 1 have been written by this warp
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (id[i] >= lo && id[i] < hi) out[id[i]] = from_f32<T>(g.at(zt[i]) + total[i]);
  };

  T* const body = out + row.head;
  if (none) {
    float zero[E] = {};
    for (int v = v0 + lane; v < v1; v += 32) store_vec<T>(body + (long long)v * E, zero);
    if (seg == 0 && row.edge(lane) >= 0) out[row.edge(lane)] = from_f32<T>(0.f);
    return;
  }
  for (int base = v0; base < v1; base += 32 * kVecs) {
    Vecs<SKEW> now;
    now.load(row, base, v1, lane);
    now.shift(row, base, v1, lane);
    g.chunk<T>(now.raw, body + (long long)(base + lane) * E, v1 - base - lane);
    patch(row.head + base * E, row.head + min(v1, base + 32 * kVecs) * E);
  }
  if (seg == 0 && row.head + row.tail > 0) {
    const int col = row.edge(lane);
    if (col >= 0) out[col] = from_f32<T>(g.at(to_f32<T>(row.p[col])));
    patch(0, row.head);
    patch(row.head + row.nvec * E, p.V);
  }
}

// ------------------------------------------------------------------ launches
constexpr int kBlocks = 148 * 3;   // resident at a time

// Short rows: `go` with the lanes of a row and the columns of a lane.  As many
// columns as keep the row's reductions few, up to 16; with alternatives a warp a
// row as soon as counting the whole row costs more than a bound (64 bf16 logits,
// best 8: 38 us for 60000 rows counted, 28 with a bound).
using std::integral_constant;
template <int G, int C, typename Go>
bool take(Go go) {
  go(integral_constant<int, G>(), integral_constant<int, C>());
  note_launch();
  return true;
}
// 60000 rows of 24 / 64 / 128 / 256 / 512 bf16 logits: 3.5 / 5.5 / 10.6 / 15.3 / 25.7 us here, 22 / 23 / 24 / 25 / 28
// in logprob_warp_kernel (fp32 3.7 / 6.3 / 10.7 / 14.0 / 24.4 and 20 / 21 / 22 / 23 / 24)
template <typename Go>
bool with_few_fwd(int V, Go go) {
  if (V <= 16) return take<2, 8>(go);
  if (V <= 32) return take<4, 8>(go);
  if (V <= 64) return take<8, 8>(go);
  if (V <= 128) return take<16, 8>(go);
  if (V <= 256) return take<16, 16>(go);
  return V <= 512 && take<32, 16>(go);
}
// with the best 8 alternatives, 24 / 64 / 128 / 256 bf16 logits: 12 / 29 / 33 / 40 us here, 58 / 70 / 60 / 59 there
template <typename Go>
bool with_few_top(int V, Go go) {
  if (V <= 16) return take<4, 4>(go);
  if (V <= 32) return take<8, 4>(go);
  if (V <= 64) return take<32, 2>(go);
  if (V <= 128) return take<32, 4>(go);
  return V <= 256 && take<32, 8>(go);
}
// The gradient, whose every lane goes through all coefficients.  2 of them, 24 / 64 / 128 / 256 logits: 4.8 / 8.3 /
// 16 / 33 us here (256 with 16 columns a lane), 21 / 21 / 23 / 24 in logprob_bwd_rows_kernel; 8 of them, 64 / 128: 14 /
// 25 here, 38 / 41 in logprob_bwd_kernel; 24 of them: 29 / 55 and 48 / 47
template <typename Go>
bool with_few_bwd(int V, int slots, Go go) {
  if (V <= 16) return take<2, 8>(go);
  if (V <= 32) return take<4, 8>(go);
  if (V <= 64) return take<8, 8>(go);
  return V <= 128 && slots <= 16 && take<16, 8>(go);
}
// All resident warps, and no more than 32 rows for one.
struct Rows32 {
  int blocks;
  uint64_t step;
  explicit Rows32(int N) {
    const int most = (N + kWarps - 1) / kWarps;
    blocks = most < kBlocks ? most : std::max(kBlocks, (most + 31) / 32);
    const uint64_t warps = (uint64_t)blocks * kWarps;
    step = (((uint64_t)N << 32) + warps - 1) / warps;
  }
};
inline dim3 few_grid(int N, int G) {
  const int rows = kWarps * 32 / G;   // of a block
  return dim3((N + rows - 1) / rows);
}

template <typename T, bool TOP>
void launch_fwd(const FwdParams& p, const T* logits, cudaStream_t st) {
  auto few = [&](auto G, auto C) {
    launch_k(logprob_few_kernel<T, G(), C(), TOP>, few_grid(p.N, G()), dim3(kWarps * 32), 0, st, 1, p, logits);
  };
  if constexpr (TOP) {
    if (with_few_top(p.V, few)) return;
  } else {
    if (with_few_fwd(p.V, few)) return;
  }
  const long long chunk = 32 * kVecs * 16 / sizeof(T);   // a warp's share at a time, in elements
  const long long chunks = (p.V + chunk - 1) / chunk;
  if (chunks <= 2 || (chunks < kWarps && p.N >= 148 * kWarps)) {
    const Rows32 rows(p.N);
    launch_k(logprob_warp_kernel<T, TOP>, dim3(rows.blocks), dim3(kWarps * 32), 0, st, 1, p, rows.step, logits);
  } else {
    int cl = 1;
    while (cl < 8 && (long long)p.N * cl < 148 && chunks > (long long)kWarps * cl) cl *= 2;
    auto go = [&](auto kernel, int grid, int warps) {
      launch_k(kernel, dim3(grid), dim3(warps * 32), 0, st, cl, p, logits);
    };
    // with rows enough for it, two warps a block, so that fewer wait for each other at the end of a row (8190 x 32768
    // bf16: 100 us with 8 warps, 97 with 4, 91 with 2; 16001 x 4097 fp32: 60, 49, 45); 8 get a single row done sooner
    if (p.N >= 4 * kBlocks) go(logprob_block_kernel<T, TOP, 1, 2>, 4 * kBlocks, 2);
    else if (cl == 1) go(logprob_block_kernel<T, TOP, 1, kWarps>, p.N < kBlocks ? p.N : kBlocks, kWarps);
    else if (cl == 2) go(logprob_block_kernel<T, TOP, 2, kWarps>, p.N * 2, kWarps);
    else if (cl == 4) go(logprob_block_kernel<T, TOP, 4, kWarps>, p.N * 4, kWarps);
    else go(logprob_block_kernel<T, TOP, 8, kWarps>, p.N * 8, kWarps);
  }
  note_launch();
}

template <typename T>
void launch_bwd(BwdParams p, const T* logits, T* dlogits, cudaStream_t st) {
  const long long vecs = p.V / (long long)(16 / sizeof(T));
  const int slots = (p.dlogp ? p.K : 0) + (p.dtop ? p.top : 0);
  auto few = [&](auto G, auto C) {
    launch_k(logprob_bwd_few_kernel<T, G(), C()>, few_grid(p.N, G()), dim3(kWarps * 32), 0, st, 1, p, logits, dlogits);
  };
  if (with_few_bwd(p.V, slots, few)) return;
  // rows of logits and gradient that start at different places of their 16 bytes
  const bool skewed = (((uintptr_t)logits - (uintptr_t)dlogits) | (uintptr_t)((p.ld - p.ldd) * sizeof(T))) % 16 != 0;
  if (slots <= kSlots && vecs <= 2 * 32 * kVecs) {
    const Rows32 rows(p.N);
    launch_k(skewed ? logprob_bwd_rows_kernel<T, true> : logprob_bwd_rows_kernel<T, false>, dim3(rows.blocks),
             dim3(kWarps * 32), 0, st, 1, p, rows.step, logits, dlogits);
  } else {
    // one to eight chunks a warp, fewer where that gives every SM 16 warps sooner
    const long long chunks = (vecs + 32 * kVecs - 1) / (32 * kVecs), all = chunks * p.N, enough = all / (148 * 16);
    const long long most = std::min(8LL, std::max(1LL, enough));
    p.segments = (int)std::max(1LL, (chunks + most - 1) / most);
    p.share = 32 * kVecs * (int)((chunks + p.segments - 1) / p.segments);
    const long long warps = (long long)p.N * p.segments;
    launch_k(skewed ? logprob_bwd_kernel<T, true> : logprob_bwd_kernel<T, false>,
             dim3((unsigned)((warps + kWarps - 1) / kWarps)), dim3(kWarps * 32), 0, st, 1, p, logits, dlogits);
  }
  note_launch();
}

int check(const frnnt_logprob_dims* d) {
  if (d->dtype != FRNNT_F32 && d->dtype != FRNNT_BF16) return FRNNT_ERR_UNSUPPORTED;
  if (d->N < 1 || d->N > (1 << 27) || d->V < 1 || d->V > (1 << 30) || d->K < 0 || d->K > FRNNT_MAX_TOKENS ||
      d->top < 0 || d->top > FRNNT_MAX_TOP || d->top > d->V || d->ld < d->V || d->ld > (1LL << 40))
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
                        (const void*)top_logp, (const void*)top_ids, (const void*)status,
                        (const void*)d->lse_rest})
    if ((uintptr_t)p % 4) return FRNNT_ERR_ALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  cudaGetLastError();   // clear a stale error so it is not reported as ours
  {
    StageScope sc("token_logprobs", st);
    const FwdParams p{d->N, d->V, d->K, d->top, d->ld, tokens, logp, entropy, lse, top_logp, top_ids, status,
                      d->lse_rest ? d->lse_rest : lse};
    if (d->dtype == FRNNT_BF16) {
      auto* z = (const __nv_bfloat16*)logits;
      d->top ? launch_fwd<__nv_bfloat16, true>(p, z, st) : launch_fwd<__nv_bfloat16, false>(p, z, st);
    } else {
      auto* z = (const float*)logits;
      d->top ? launch_fwd<float, true>(p, z, st) : launch_fwd<float, false>(p, z, st);
    }
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
                        (const void*)dlogp, (const void*)dentropy, (const void*)dtop, (const void*)status,
                        (const void*)d->lse_rest})
    if ((uintptr_t)p % 4) return FRNNT_ERR_ALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  cudaGetLastError();   // clear a stale error so it is not reported as ours
  {
    StageScope sc("token_logprobs_bwd", st);
    const BwdParams p{d->N, d->V, d->K,    d->top, 1,     0,        d->ld, d->ldd,
                      tokens, top_ids, lse, entropy, dlogp, dentropy, dtop,  status,
                      d->lse_rest ? d->lse_rest : lse, d->lse_rest ? -kLog2e : 0.f};
    if (d->dtype == FRNNT_BF16) launch_bwd(p, (const __nv_bfloat16*)logits, (__nv_bfloat16*)dlogits, st);
    else launch_bwd(p, (const float*)logits, (float*)dlogits, st);
  }
  return cudaGetLastError() == cudaSuccess ? FRNNT_OK : FRNNT_ERR_CUDA;
}
