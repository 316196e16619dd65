// Gated linear recurrence h_t = a_t h_{t-1} + (1 - a_t) x_t, a = sigmoid(gate):
// forward over padded sequences, backward, and one step of many hypotheses.
#include <atomic>
#include <climits>
#include <initializer_list>
#include <type_traits>

#include "frnnt_common.cuh"
#include "frnnt_internal.h"
#include "frnnt_ops.h"
#include "sm100.cuh"

namespace frnnt {
namespace {

// A block walks along one sequence, 64 channels wide, kChunk steps at a
// time.  Lane l of every warp holds channels 2l and 2l + 1 (of unaligned rows l
// and l + half the tile: see kApart); warp w takes the kSteps steps from w *
// kSteps on.
constexpr int kChunk = FRNNT_SCAN_CHUNK;
constexpr int kSteps = 16;
constexpr int kWarps = kChunk / kSteps;

// a = sigmoid(gate) and s = 1 - a = sigmoid(-gate), each to relative precision:
// with e = exp(-gate), a = 1 / (1 + e), and s = e a where that is below 1/2 (1 -
// a would lose its digits where the memory is long and a is near 1), 1 - a
// above (where e may be infinite).  The hardware exp2 and reciprocal are good
// to 2^-22, and the rounded exponent adds |gate| 2^-24.
struct Gates {   // of two channels
  uint64_t a, s;
};
__device__ __forceinline__ Gates gates_of(uint64_t g) {
  const float2 x = f2_open(f2_mul(g, f2_of(-1.44269504f, -1.44269504f)));
  float e0, e1, a0, a1;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(x.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(x.y));
  const uint64_t e = f2_of(e0, e1), one = f2_of(1.f, 1.f);
  const float2 d = f2_open(f2_add(e, one));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a0) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a1) : "f"(d.y));
  const uint64_t a = f2_of(a0, a1);
  const float2 small = f2_open(f2_mul(e, a)), big = f2_open(f2_fma(a, f2_of(-1.f, -1.f), one));
  return Gates{a, f2_of(e0 > 1.f ? big.x : small.x, e1 > 1.f ? big.y : small.y)};
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
  static __device__ __forceinline__ uint64_t open(float2 r) { return f2_of(r.x, r.y); }
  static __device__ __forceinline__ float2 pack(float2 v) { return v; }
};
template <>
struct Pair<__nv_bfloat16> {
  using Raw = uint32_t;
  static __device__ __forceinline__ uint64_t open(uint32_t r) {
    return f2_of(__uint_as_float(r << 16), __uint_as_float(r & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float2 f) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

// One array of a chunk in shared memory: kChunk rows of kPitch elements.
// VEC: every row of the array starts on a 16-byte boundary.  Otherwise a row is
// copied from the boundary at or before it (which lies in the same
// allocation: those start on 256-byte boundaries) and read at that offset, and
// a block takes 16 bytes' worth of channels less, so that the row still fits.
constexpr int kPitch = 64;
template <typename T, bool VEC>
constexpr int kTile = VEC ? kPitch : kPitch - 16 / (int)sizeof(T);
// From a lane's first channel to its second.  Unaligned rows are read and written
// one element at a time, so those of neighbouring lanes are neighbours.
template <typename T, bool VEC>
constexpr int kApart = VEC ? 1 : kTile<T, VEC> / 2;

template <typename T>
struct Stage {
  T v[kChunk][kPitch];
};

// Rows t0 .. of one array, from channel c0 on.
template <typename T, bool VEC>
struct Rows {
  const char* first;   // of step 0
  long long step;      // bytes
  int width;           // bytes of a row that exist
  __device__ __forceinline__ Rows(const T* p, long long step_elems, int c0, int D)
      : first(reinterpret_cast<const char*>(p + c0)), step(step_elems * (long long)sizeof(T)),
        width(min(kTile<T, VEC>, D - c0) * (int)sizeof(T)) {}

  // Starts the copy of the block's rows t0 .. (16 a warp) into `to`; rows from
  // len on get `rest` (two 16-bit values or one 32-bit one).
  __device__ __forceinline__ void fetch(Stage<T>& to, int t0, int len, uint32_t rest) const {
    constexpr int kPerRow = kPitch * sizeof(T) / 16, kTimes = kSteps * kPerRow / 32;
    const int j = threadIdx.x % kPerRow, r0 = threadIdx.x / kPerRow, rows = blockDim.x / kPerRow;
    const char* src = first + (t0 + r0) * step;
    uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to.v[r0])) + 16 * j;
    const long long skip = rows * step;
    const int left = len - t0 - r0;
    if (len - t0 >= kTimes * rows) {
      if (VEC) {
        const int bytes = max(0, min(16, width - 16 * j));
        src = bytes > 0 ? src + 16 * j : first;
#pragma unroll
        for (int k = 0; k < kTimes; ++k, src += skip, dst += rows * (uint32_t)sizeof(to.v[0]))
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(bytes > 0 ? src : first),
                       "r"(bytes)
                       : "memory");
      } else {
#pragma unroll
        for (int k = 0; k < kTimes; ++k) copy(dst + k * rows * (uint32_t)sizeof(to.v[0]), src + k * skip, j);
      }
    } else {
      for (int k = 0; k < kTimes; ++k, src += skip, dst += rows * (uint32_t)sizeof(to.v[0])) {
        if (k * rows < left) copy(dst, src, j);
        else asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(rest) : "memory");
      }
    }
  }
  __device__ __forceinline__ void copy(uint32_t dst, const char* row, int j) const {
    const int skew = VEC ? 0 : (int)((uintptr_t)row & 15);
    const int bytes = max(0, min(16, width + skew - 16 * j));   // 0: zeros, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(row - skew + (bytes > 0 ? 16 * j : 0)),
                 "r"(bytes)
                 : "memory");
  }
  // Where row t0 + i of the stage starts, for read().
  __device__ __forceinline__ uint32_t skew(int t0) const { return VEC ? 0u : (uint32_t)(uintptr_t)(first + t0 * step); }
  // The lane's two channels of row w0 + i; skew0: skew() of row w0.
  __device__ __forceinline__ uint64_t read(const Stage<T>& from, int w0, int i, int lane, uint32_t skew0) const {
    if (VEC) return Pair<T>::open(reinterpret_cast<const typename Pair<T>::Raw*>(from.v[w0 + i])[lane]);
    // (the last lanes' channels are past the tile: whatever lies there does)
    const uint32_t off = ((skew0 + (uint32_t)i * (uint32_t)step) & 15u) + (uint32_t)sizeof(T) * lane;
    const T* q = reinterpret_cast<const T*>(reinterpret_cast<const char*>(from.v[w0 + i]) + off);
    return f2_of(to_f32<T>(q[0]), to_f32<T>(q[kApart<T, VEC>]));
  }
};
// Neutral rows: with gate = +inf, a = 1 and 1 - a = 0, and the state stays as it is.
template <typename T>
constexpr uint32_t kOpen = sizeof(T) == 4 ? 0x7F800000u : 0x7F807F80u;

// A pair at a 32-bit byte offset from a block-wide base.
template <typename T>
__device__ __forceinline__ void store_at(char* base, uint32_t off, uint64_t v) {
  *reinterpret_cast<typename Pair<T>::Raw*>(base + off) = Pair<T>::pack(f2_open(v));
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_pair(T* p, float2 v, bool two) {
  using Raw = typename Pair<T>::Raw;
  if (VEC) {
    *reinterpret_cast<Raw*>(p) = Pair<T>::pack(v);
  } else {
    p[0] = from_f32<T>(v.x);
    if (two) p[kApart<T, VEC>] = from_f32<T>(v.y);
  }
}

// The lane's channels of a [rows, D] fp32 array.
template <int APART>
__device__ __forceinline__ uint64_t load_state(const float* p, long long row, int D, int c, bool live, bool two) {
  if (!p || !live) return f2_of(0.f, 0.f);
  const float* q = p + row * D + c;
  return f2_of(q[0], two ? q[APART] : 0.f);
}
template <int APART>
__device__ __forceinline__ void store_state(float* p, long long row, int D, int c, bool live, bool two, uint64_t v) {
  if (!p || !live) return;
  const float2 f = f2_open(v);
  float* q = p + row * D + c;
  q[0] = f.x;
  if (two) q[APART] = f.y;
}

// A run of steps as a map of its entering value: out = A in + R.
struct Map {
  uint64_t A, R;
};
__device__ __forceinline__ Map map_one() { return Map{f2_of(1.f, 1.f), f2_of(0.f, 0.f)}; }
__device__ __forceinline__ Map then(Map f, Map g) { return Map{f2_mul(g.A, f.A), f2_fma(g.A, f.R, g.R)}; }
__device__ __forceinline__ uint64_t apply(Map f, uint64_t v) { return f2_fma(f.A, v, f.R); }

// A launch in which the exchange below fails on purpose (frnnt_test_lose_scan_maps): block 0 of every cluster, in one
// round (counted from the last when negative), sends no map (kLose), or behaves as if its wait had run out (kQuit).
struct Trial {
  enum { kNone, kLose, kQuit };
  int kind = kNone, round = 0;
  uint32_t tries = sm100::kMaxTries;   // polls of a wait
  __device__ __forceinline__ int of(int rank, int rounds) const {   // the round in which this block is to fail
    return kind == kNone || rank != 0 ? -1 : round < 0 ? rounds + round : round;
  }
};

// The blocks of a cluster tell each other the map of their chunk: the first warp
// of every block sends it to every block's shared memory, where an mbarrier
// counts the bytes of all CL maps.  Two buffers: a warp that sends round r + 2
// has received round r + 1 from all, and each sent that after it had read round r.
// A wait that runs out ends the block after its round: it neither sends nor
// arrives again, so the others' waits run out a round later at the latest, and it
// leaves when no map can still come (see leave).  Beside waits that went on
// regardless this costs nothing to 2 % (2 x 32749 x 1024 bf16: 94 -> 91 us, backward
// 148; 3 x 10000 x 1024: 44.4 -> 45.7 and 68.0 -> 69.4; 2 x 16384 x 1023: 84 -> 85
// and 138 -> 139).  With a vote of the lanes and a branch in the first warp's way the
// backward passes took up to 163 and 147.
template <int CL>
struct Exchange {
  static constexpr uint32_t kBytes = 32 * sizeof(ulonglong2);   // of a map
  ulonglong2 maps[2][CL][32];
  uint64_t full[2];
  int gave_up;    // 1 + the round whose wait ran out, 0: none
  int sent[CL];   // rounds that a block sent which gave up before its last one (else: all)

  __device__ __forceinline__ void init() {
    if (threadIdx.x == 0) {
      sm100::mbar_init(&full[0], 1);
      sm100::mbar_init(&full[1], 1);
      sm100::fence_barrier_init();
      gave_up = 0;
#pragma unroll
      for (int k = 0; k < CL; ++k) sent[k] = INT_MAX;   // (a thread each: 146 for 139 us, see above)
    }
  }
  __device__ __forceinline__ void send(int r, int rank, int lane, Map m, int odd, const Trial& trial) {
    if (lane == 0) sm100::mbar_arrive_expect_tx(&full[r & 1], CL * kBytes);
    if (r == odd && trial.kind == Trial::kLose) return;
#pragma unroll
    for (int k = 0; k < CL; ++k)
      asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(
                       in_cluster(&maps[r & 1][rank][lane], k)),
                   "l"(m.A), "l"(m.R), "r"(in_cluster(&full[r & 1], k))
                   : "memory");
  }
  __device__ __forceinline__ bool wait(int r, uint32_t tries) {
    bool ok = sm100::mbar_try_wait_cluster(&full[r & 1], (r >> 1) & 1, 0);
    for (uint32_t i = 0; !ok && i < tries; ++i)
      ok = sm100::mbar_try_wait_cluster(&full[r & 1], (r >> 1) & 1, sm100::kSuspendNs);
    return ok;
  }
  // The carry after this round; `in`: what enters block `rank`'s chunk.  A lane
  // whose wait runs out says so in gave_up, which all warps see after the next
  // block barrier; its carry means nothing.
  __device__ __forceinline__ uint64_t receive(int r, int rank, int lane, uint64_t carry, uint64_t& in, int odd,
                                              const Trial& trial, int32_t* status) {
    const bool ok = wait(r, trial.tries) && !(r == odd && trial.kind == Trial::kQuit);
    if (!ok) {
      gave_up = r + 1;
      if (status) atomicOr(status, FRNNT_STATUS_TIMEOUT);
    }
    for (int k = 0; k < CL; ++k) {
      if (k == rank) in = carry;
      const ulonglong2 o = maps[r & 1][k][lane];
      carry = f2_fma(o.x, carry, o.y);
    }
    return carry;
  }
  // The end of a block that gave up in round r, which it sent.  Maps of rounds r
  // and r + 1 may still be on their way to it (r + 2 needs its r + 1).  Every
  // block of the cluster gives up too or has left after its last round, so all
  // of them meet here or are gone; what each sent is known then, and the bytes
  // of that are awaited.  While this block has a round to send, no block can
  // have received all rounds and left, so the count may be told to each.
  __device__ __noinline__ void leave(int rank, int rounds, uint32_t tries) {
    const int r = gave_up - 1;
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (threadIdx.x < CL && r + 1 < rounds)
      asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(in_cluster(&sent[rank], threadIdx.x)), "r"(r + 1)
                   : "memory");
    cluster_arrive();
    cluster_wait();   // (for the threads that have not exited)
    if (threadIdx.x != 0) return;
    uint32_t missing = 0, ahead = 0;
    for (int k = 0; k < CL; ++k) {
      missing += sent[k] <= r;
      ahead += r + 1 < rounds && sent[k] > r + 1;
    }
    if (missing)   // the arrival in send() expects the bytes of all
      asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" ::"r"(sm100::smem_u32(&full[r & 1])),
                   "r"(missing * kBytes)
                   : "memory");
    wait(r, tries);
    if (ahead) {
      sm100::mbar_arrive_expect_tx(&full[(r + 1) & 1], ahead * kBytes);
      wait(r + 1, tries);
    }
  }
};
template <>
struct Exchange<1> {
  __device__ __forceinline__ void init() {}
  static constexpr int gave_up = 0;
};

// Forward.  h_t = a_t h_{t-1} + b_t composes: over a run of steps h_out = A h_in
// + R with A the product of the a and R the run's result from zero.  Each
// warp forms its run's map, the block joins them in shared memory, and each
// warp walks its run again from its true entering state, out of registers: x
// and gate are read once, h written once.  The block carries the state from
// chunk to chunk and has the next chunks on their way meanwhile.  Where there
// are too few (sequence, channel tile) pairs to fill the GPU, CL blocks of a
// cluster take the chunks in turn.
// Bound by memory (three elements moved a step and channel) where there are
// tiles enough: 32 x 4096 x 1024 bf16 143 us (5.6 TB/s).  2 x 32749 x 1024 bf16,
// clusters of 8: 91 us (4.5 TB/s), its 256 blocks not spread evenly over the
// SMs, and latency: one exchange and three block barriers a round.  16 steps a thread, in registers, halve the
// work on maps against 8 (326 us, one element at a time); results put into
// shared memory and written 16 bytes a lane were no faster.
template <typename T, bool VEC, int CL, int STAGES>
__global__ void __launch_bounds__(kWarps * 32, 2)
    scan_fwd_kernel(frnnt_recurrence_dims d, const T* __restrict__ x, const T* __restrict__ gate,
                    const int32_t* __restrict__ lengths, const float* __restrict__ h0, T* __restrict__ h,
                    float* __restrict__ h_last, float* __restrict__ saved, int32_t* status, Trial trial) {
  extern __shared__ __align__(128) unsigned char smem[];
  Stage<T>* stage = reinterpret_cast<Stage<T>*>(smem);   // [STAGES][x, gate]
  __shared__ ulonglong2 run[kWarps][32];
  __shared__ Exchange<CL> ex;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int b = blockIdx.y, rank = CL > 1 ? blockIdx.x % CL : 0;
  const int c0 = (blockIdx.x / CL) * kTile<T, VEC>, c = c0 + (VEC ? 2 : 1) * lane;
  const bool live = lane < kTile<T, VEC> / 2 && c < d.D, two = c + kApart<T, VEC> < d.D, whole = c0 + kPitch <= d.D;
  const int len = length_of(lengths, b, d.T, status), nc = (d.T + kChunk - 1) / kChunk;
  const int rounds = ((len + kChunk - 1) / kChunk + CL - 1) / CL;
  const Rows<T, VEC> xs(x + b * d.x_sb, d.x_st, c0, d.D), gs(gate + b * d.gate_sb, d.gate_st, c0, d.D);
  T* hp = h + b * d.h_sb + c;
  ex.init();
  if (CL > 1) cluster_arrive();
  auto fetch = [&](int r) {
    if (r < rounds) {
      const int t = (r * CL + rank) * kChunk;
      xs.fetch(stage[2 * (r % STAGES)], t, len, 0u);
      gs.fetch(stage[2 * (r % STAGES) + 1], t, len, kOpen<T>);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int r = 0; r < STAGES - 1; ++r) fetch(r);
  uint64_t carry = load_state<kApart<T, VEC>>(h0, b, d.D, c, live, two);
  if (CL > 1) cluster_wait();     // the other blocks run, their mbarriers are ready
  [[maybe_unused]] const int odd = trial.of(rank, rounds);
  for (int r = 0; r < rounds; ++r) {
    const int t0 = (r * CL + rank) * kChunk + w * kSteps;
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
    __syncthreads();              // this round's rows are here; the stage before is free
    fetch(r + STAGES - 1);
    const Stage<T>&sx = stage[2 * (r % STAGES)], &sg = stage[2 * (r % STAGES) + 1];
    const uint32_t xk = xs.skew(t0), gk = gs.skew(t0);
    uint64_t a[kSteps], v[kSteps];
    Map m = map_one();
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const Gates g = gates_of(gs.read(sg, w * kSteps, i, lane, gk));
      a[i] = g.a;
      v[i] = f2_mul(g.s, xs.read(sx, w * kSteps, i, lane, xk));
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) m = then(m, Map{a[i], v[i]});
    run[w][lane] = make_ulonglong2(m.A, m.R);
    __syncthreads();
    if (w == 0) {   // what enters each run, in the place of its R
      uint64_t in = carry;
      if constexpr (CL > 1) {
        Map all = map_one();
        for (int k = 0; k < nw; ++k) all = then(all, Map{run[k][lane].x, run[k][lane].y});
        ex.send(r, rank, lane, all, odd, trial);
        carry = ex.receive(r, rank, lane, carry, in, odd, trial, status);
      }
      if (t0 < len) store_state<kApart<T, VEC>>(saved, (long long)b * nc + t0 / kChunk, d.D, c, live, two, in);
      for (int k = 0; k < nw; ++k) {
        const ulonglong2 o = run[k][lane];
        run[k][lane].y = in;
        in = apply(Map{o.x, o.y}, in);
      }
      if constexpr (CL == 1) carry = in;
    }
    __syncthreads();
    const bool stop = CL > 1 && ex.gave_up != 0;   // read early, used after the run
    uint64_t s = run[w][lane].y;
    if (VEC && whole && t0 + kSteps <= len) {
      char* base = reinterpret_cast<char*>(h + b * d.h_sb + c0 + (long long)(r * CL + rank) * kChunk * d.h_st);
      const uint32_t step = (uint32_t)d.h_st * (uint32_t)sizeof(T);
      uint32_t off = w * kSteps * step + lane * 2 * (uint32_t)sizeof(T);
#pragma unroll
      for (int i = 0; i < kSteps; ++i, off += step) {
        s = f2_fma(a[i], s, v[i]);
        store_at<T>(base, off, s);
      }
    } else if (!VEC && t0 + kSteps <= len) {
      T* out = hp + (long long)t0 * d.h_st;
#pragma unroll
      for (int i = 0; i < kSteps; ++i, out += d.h_st) {
        s = f2_fma(a[i], s, v[i]);
        if (live) store_pair<T, VEC>(out, f2_open(s), two);
      }
    } else {
      T* out = hp + (long long)t0 * d.h_st;
#pragma unroll
      for (int i = 0; i < kSteps; ++i, out += d.h_st) {
        s = f2_fma(a[i], s, v[i]);
        if (live && t0 + i < d.T)
          store_pair<T, VEC>(out, t0 + i < len ? f2_open(s) : make_float2(0.f, 0.f), two);
      }
    }
    if (stop) break;
  }
  // rows of whole rounds past the sequence
  for (int t = rounds * CL * kChunk + rank * nw + w; t < d.T; t += CL * nw)
    if (live) store_pair<T, VEC>(hp + t * d.h_st, make_float2(0.f, 0.f), two);
  if (rank == 0 && w == 0) store_state<kApart<T, VEC>>(h_last, b, d.D, c, live, two, carry);
  if constexpr (CL > 1)
    if (rounds && ex.gave_up) ex.leave(rank, rounds, trial.tries);
}

// Backward.  With q_t = a_t g_t, what step t hands to step t - 1, q_t = a_t
// (q_{t+1} + dh_t) is the same recurrence run from the end: over a run of
// steps q_out = A q_in + Q with the same A.  The chunk's states are formed
// again from its saved state by the forward maps, in the same exchange, so x,
// gate and dh are read once, dx and dgate written once, and h is not read.
// 32 x 4096 x 1024 bf16: 247 us (5.4 TB/s); 2 x 32749 x 1024 bf16: 148 us (4.5
// TB/s).  Results written through shared memory: 271 us and 158 us.
template <typename T, bool VEC, int CL, int STAGES>
__global__ void __launch_bounds__(kWarps * 32, 2)
    scan_bwd_kernel(frnnt_recurrence_dims d, const T* __restrict__ x, const T* __restrict__ gate,
                    const int32_t* __restrict__ lengths, const float* __restrict__ saved, const T* __restrict__ dh,
                    const float* __restrict__ dh_last, T* __restrict__ dx, T* __restrict__ dgate,
                    float* __restrict__ dh0, int32_t* status, Trial trial) {
  extern __shared__ __align__(128) unsigned char smem[];
  Stage<T>* stage = reinterpret_cast<Stage<T>*>(smem);   // [STAGES][x, gate, dh]
  __shared__ ulonglong2 run[kWarps][32];   // forward maps
  __shared__ uint64_t back[kWarps][32];    // Q of the backward maps
  __shared__ Exchange<CL> ex;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int b = blockIdx.y, rank = CL > 1 ? blockIdx.x % CL : 0;
  const int c0 = (blockIdx.x / CL) * kTile<T, VEC>, c = c0 + (VEC ? 2 : 1) * lane;
  const bool live = lane < kTile<T, VEC> / 2 && c < d.D, two = c + kApart<T, VEC> < d.D, whole = c0 + kPitch <= d.D;
  const int len = length_of(lengths, b, d.T, status), nc = (d.T + kChunk - 1) / kChunk;
  const int rounds = ((len + kChunk - 1) / kChunk + CL - 1) / CL;
  const Rows<T, VEC> xs(x + b * d.x_sb, d.x_st, c0, d.D), gs(gate + b * d.gate_sb, d.gate_st, c0, d.D),
      hs(dh + b * d.dh_sb, d.dh_st, c0, d.D);
  T* dxp = dx + b * d.dx_sb + c;
  T* dgp = dgate + b * d.dgate_sb + c;
  ex.init();
  if (CL > 1) cluster_arrive();
  // rounds from the end; within a round rank 0 has the latest chunk
  auto chunk_at = [&](int r) { return ((rounds - r) * CL - 1 - rank) * kChunk; };
  auto fetch = [&](int r) {
    if (r < rounds) {
      const int t = chunk_at(r);
      Stage<T>* to = stage + 3 * (r % STAGES);
      xs.fetch(to[0], t, len, 0u);
      gs.fetch(to[1], t, len, kOpen<T>);
      hs.fetch(to[2], t, len, 0u);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int r = 0; r < STAGES - 1; ++r) fetch(r);
  uint64_t carry = load_state<kApart<T, VEC>>(dh_last, b, d.D, c, live, two);
  if (CL > 1) cluster_wait();
  [[maybe_unused]] const int odd = trial.of(rank, rounds);
  for (int r = 0; r < rounds; ++r) {
    const int t0 = chunk_at(r) + w * kSteps;
    uint64_t v = f2_of(0.f, 0.f);   // (the first warp's)
    if (w == 0 && t0 < len) v = load_state<kApart<T, VEC>>(saved, (long long)b * nc + t0 / kChunk, d.D, c, live, two);
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
    __syncthreads();              // this round's rows are here; the stage before is free
    fetch(r + STAGES - 1);
    const Stage<T>* at = stage + 3 * (r % STAGES);
    const uint32_t xk = xs.skew(t0), gk = gs.skew(t0), hk = hs.skew(t0);
    uint64_t a[kSteps], s[kSteps], past[kSteps];
    Map m = map_one();
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const Gates g = gates_of(gs.read(at[1], w * kSteps, i, lane, gk));
      a[i] = g.a;
      s[i] = g.s;
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) m = then(m, Map{a[i], f2_mul(s[i], xs.read(at[0], w * kSteps, i, lane, xk))});
    uint64_t q = f2_of(0.f, 0.f);
#pragma unroll
    for (int i = kSteps - 1; i >= 0; --i) q = f2_mul(a[i], f2_add(q, hs.read(at[2], w * kSteps, i, lane, hk)));
    run[w][lane] = make_ulonglong2(m.A, m.R);
    back[w][lane] = q;
    __syncthreads();
    if (w == 0) {   // what enters each run, in the place of its R and Q
      uint64_t in = carry;
      if constexpr (CL > 1) {
        Map all = map_one();
        for (int k = nw - 1; k >= 0; --k) all = then(all, Map{run[k][lane].x, back[k][lane]});
        ex.send(r, rank, lane, all, odd, trial);
      }
      for (int k = 0; k < nw; ++k) {
        const ulonglong2 o = run[k][lane];
        run[k][lane].y = v;
        v = apply(Map{o.x, o.y}, v);
      }
      if constexpr (CL > 1) carry = ex.receive(r, rank, lane, carry, in, odd, trial, status);
      for (int k = nw - 1; k >= 0; --k) {
        const uint64_t o = back[k][lane];
        back[k][lane] = in;
        in = apply(Map{run[k][lane].x, o}, in);
      }
      if constexpr (CL == 1) carry = in;
    }
    __syncthreads();
    const bool stop = CL > 1 && ex.gave_up != 0;   // read early, used after the run
    v = run[w][lane].y;
    q = back[w][lane];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {   // the states again
      const uint64_t xv = xs.read(at[0], w * kSteps, i, lane, xk);
      past[i] = f2_fma(xv, f2_of(-1.f, -1.f), v);
      v = f2_fma(a[i], v, f2_mul(s[i], xv));
    }
    if (VEC && whole && t0 + kSteps <= len) {
      const long long first = chunk_at(r);
      char* bx = reinterpret_cast<char*>(dx + b * d.dx_sb + c0 + first * d.dx_st);
      char* bg = reinterpret_cast<char*>(dgate + b * d.dgate_sb + c0 + first * d.dgate_st);
      const uint32_t sx = (uint32_t)d.dx_st * (uint32_t)sizeof(T), sg = (uint32_t)d.dgate_st * (uint32_t)sizeof(T);
      uint32_t ox = (w * kSteps + kSteps - 1) * sx + lane * 2 * (uint32_t)sizeof(T);
      uint32_t og = (w * kSteps + kSteps - 1) * sg + lane * 2 * (uint32_t)sizeof(T);
#pragma unroll
      for (int i = kSteps - 1; i >= 0; --i, ox -= sx, og -= sg) {
        const uint64_t g = f2_add(q, hs.read(at[2], w * kSteps, i, lane, hk));
        q = f2_mul(a[i], g);
        store_at<T>(bx, ox, f2_mul(s[i], g));
        store_at<T>(bg, og, f2_mul(f2_mul(q, s[i]), past[i]));
      }
    } else if (!VEC && t0 + kSteps <= len) {
      T* px = dxp + (t0 + kSteps - 1) * d.dx_st;
      T* pg = dgp + (t0 + kSteps - 1) * d.dgate_st;
#pragma unroll
      for (int i = kSteps - 1; i >= 0; --i, px -= d.dx_st, pg -= d.dgate_st) {
        const uint64_t g = f2_add(q, hs.read(at[2], w * kSteps, i, lane, hk));
        q = f2_mul(a[i], g);
        if (live) {
          store_pair<T, VEC>(px, f2_open(f2_mul(s[i], g)), two);
          store_pair<T, VEC>(pg, f2_open(f2_mul(f2_mul(q, s[i]), past[i])), two);
        }
      }
    } else {
      T* px = dxp + (t0 + kSteps - 1) * d.dx_st;
      T* pg = dgp + (t0 + kSteps - 1) * d.dgate_st;
#pragma unroll
      for (int i = kSteps - 1; i >= 0; --i, px -= d.dx_st, pg -= d.dgate_st) {
        const uint64_t g = f2_add(q, hs.read(at[2], w * kSteps, i, lane, hk));
        q = f2_mul(a[i], g);
        if (live && t0 + i < d.T) {
          const bool on = t0 + i < len;
          const float2 zero = make_float2(0.f, 0.f);
          store_pair<T, VEC>(px, on ? f2_open(f2_mul(s[i], g)) : zero, two);
          store_pair<T, VEC>(pg, on ? f2_open(f2_mul(f2_mul(q, s[i]), past[i])) : zero, two);
        }
      }
    }
    if (stop) break;
  }
  for (int t = rounds * CL * kChunk + rank * nw + w; t < d.T; t += CL * nw)
    if (live) {
      store_pair<T, VEC>(dxp + t * d.dx_st, make_float2(0.f, 0.f), two);
      store_pair<T, VEC>(dgp + t * d.dgate_st, make_float2(0.f, 0.f), two);
    }
  if (rank == 0 && w == 0) store_state<kApart<T, VEC>>(dh0, b, d.D, c, live, two, carry);
  if constexpr (CL > 1)
    if (rounds && ex.gave_up) ex.leave(rank, rounds, trial.tries);
}

// One step: a thread takes C neighbouring channels of a row in one access an
// array (4 where all rows are aligned to that, else 1).  Bound by memory, and
// for a beam's few rows by the launch: 4096 x 4096 bf16 36 us (6.5 TB/s), 64 x
// 640 2.1 us.
template <typename T, int C>
struct alignas(C * sizeof(T)) Channels {
  T v[C];
};
constexpr int kStepThreads = 128;
template <typename T, int C>
__global__ void __launch_bounds__(kStepThreads)
    step_kernel(frnnt_step_dims d, const T* __restrict__ x, const T* __restrict__ gate, const float* state,
                const int32_t* __restrict__ parent, const uint8_t* __restrict__ advance, T* __restrict__ h,
                float* new_state, int32_t* status) {
  const int c = (blockIdx.x * kStepThreads + threadIdx.x) * C;
  const long long n = blockIdx.y;
  if (c >= d.D) return;
  const bool go = !advance || advance[n];
  Channels<T, C> xv, gv, out;
  if (go) {   // before the parent is known
    gv = *reinterpret_cast<const Channels<T, C>*>(gate + n * d.gate_sn + c);
    xv = *reinterpret_cast<const Channels<T, C>*>(x + n * d.x_sn + c);
  }
  int from = (int)n;
  if (parent) {
    from = parent[n];
    if ((from < 0 || from >= d.S) && status && c == 0) atomicOr(status, FRNNT_STATUS_INDEX);
    from = clampi(from, 0, d.S - 1);
  }
  Channels<float, C> v = *reinterpret_cast<const Channels<float, C>*>(state + (long long)from * d.D + c);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if (go) {
      const Gates g = gates_of(f2_of(to_f32<T>(gv.v[i]), 0.f));
      v.v[i] = fmaf(f2_open(g.a).x, v.v[i], f2_open(g.s).x * to_f32<T>(xv.v[i]));
    }
    out.v[i] = from_f32<T>(v.v[i]);
  }
  *reinterpret_cast<Channels<float, C>*>(new_state + n * d.D + c) = v;
  *reinterpret_cast<Channels<T, C>*>(h + n * d.D + c) = out;
}

bool dtype_ok(frnnt_dtype t) { return t == FRNNT_F32 || t == FRNNT_BF16; }

// (the kernels hold step strides in 32 bits)
bool in_strides_ok(long long sb, long long st) { return sb >= 0 && st >= 0 && sb <= (1LL << 40) && st <= (1LL << 30); }

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

// Chunks in shared memory at a time: three of two arrays, two of three (96 KB of
// a 16-bit type: two blocks an SM; a block of a 32-bit type has the SM alone).
constexpr int stages_of(int arrays) { return arrays == 2 ? 3 : 2; }
// What the last lanes may read past the last row (see Rows::read).
constexpr int kSlack = 16;

template <typename T, int ARRAYS>
constexpr int kMostBytes = (int)sizeof(Stage<T>) * ARRAYS * stages_of(ARRAYS) + kSlack;

// Test setting (frnnt_test_refuse_clusters): the runtime is asked for more shared memory than there is.
bool g_refuse_clusters = false;

// How many clusters of CL blocks run at a time on the current device (any number
// with CL = 1), and the kernel made ready for that much shared memory.  Clusters
// that the runtime refuses do not run: 0, and its error is taken back, since the
// call goes on with other sizes; a single block that it refuses: -1, an error.
template <typename T, int ARRAYS, int CL, auto kernel>
int resident() {
  static std::atomic<int> known[kDeviceSlots];   // (+ 1)
  std::atomic<int>& here = known[current_device()];
  const bool refuse = CL > 1 && g_refuse_clusters;
  if (const int n = here.load(std::memory_order_acquire); n && !refuse) return n - 1;
  constexpr int bytes = kMostBytes<T, ARRAYS>;
  bool ok = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, refuse ? INT_MAX : bytes) ==
            cudaSuccess;
  if (CL > 8) ok = ok && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
  int n = INT_MAX - 1;
  if (CL > 1 && ok) {
    cudaLaunchAttribute size;
    size.id = cudaLaunchAttributeClusterDimension;
    size.val.clusterDim.x = CL;
    size.val.clusterDim.y = size.val.clusterDim.z = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(CL);
    config.blockDim = dim3(kWarps * 32);
    config.dynamicSmemBytes = bytes;
    config.attrs = &size;
    config.numAttrs = 1;
    ok = cudaOccupancyMaxActiveClusters(&n, kernel, &config) == cudaSuccess && n >= 0;
  }
  if (!ok) {
    if (CL == 1) return -1;
    cudaGetLastError();
    n = 0;
  }
  if (!refuse) here.store(n + 1, std::memory_order_release);
  return n;
}

// Blocks that share a sequence's chunks: as few as give the fewest rounds, of
// those whose clusters run all at once.  bf16, forward and backward, with 8 at
// most and powers of two only: 8 x 1500 x 513 23 us and 38, here (6) 16 and 27; 1 x
// 32749 x 64 61 and 91, here (16) 37 and 50.  Clusters that do not all fit: 3 x
// 10000 x 1024 61 and 94 (48 of 6), here (5) 46 and 69.  Sizes 9 and 11 to 15 are
// left out: each is eight kernels, and of the chunk and tile counts up to 256 and
// 152, evenly spread over their logarithms, 8 % would take fewer rounds with them.
template <typename Fit, typename Launch>
int with_cluster(const frnnt_recurrence_dims& d, int tile, Fit fit, Launch launch) {
  const long long tiles = (long long)((d.D + tile - 1) / tile) * d.B;
  const int nc = (d.T + kChunk - 1) / kChunk;
  auto rounds = [&](int cl) { return (nc + cl - 1) / cl; };
  int best = 1;
  auto may = [&](auto CL) {
    if (tiles * CL() <= 2 * 148 && rounds(CL()) < rounds(best) && tiles <= fit(CL)) best = CL();
  };
  using std::integral_constant;
  may(integral_constant<int, 2>());
  may(integral_constant<int, 3>());
  may(integral_constant<int, 4>());
  may(integral_constant<int, 5>());
  may(integral_constant<int, 6>());
  may(integral_constant<int, 7>());
  may(integral_constant<int, 8>());
  may(integral_constant<int, 10>());
  may(integral_constant<int, 16>());
  switch (best) {
    case 1: return launch(integral_constant<int, 1>());
    case 2: return launch(integral_constant<int, 2>());
    case 3: return launch(integral_constant<int, 3>());
    case 4: return launch(integral_constant<int, 4>());
    case 5: return launch(integral_constant<int, 5>());
    case 6: return launch(integral_constant<int, 6>());
    case 7: return launch(integral_constant<int, 7>());
    case 8: return launch(integral_constant<int, 8>());
    case 10: return launch(integral_constant<int, 10>());
    default: return launch(integral_constant<int, 16>());
  }
}

template <typename T, int TILE, int ARRAYS, int CL, auto kernel, typename... A>
int launch_scan(const frnnt_recurrence_dims& d, cudaStream_t st, A... args) {
  if (resident<T, ARRAYS, CL, kernel>() < 0) return FRNNT_ERR_CUDA;
  const int warps = d.T < kChunk ? (d.T + kSteps - 1) / kSteps : kWarps;
  const dim3 grid((d.D + TILE - 1) / TILE * CL, d.B);
  // as many stages as there are rounds (whole ones, however short the last chunk)
  const int rounds = ((d.T + kChunk - 1) / kChunk + CL - 1) / CL;
  const int bytes =
      rounds >= stages_of(ARRAYS) ? kMostBytes<T, ARRAYS> : rounds * (int)sizeof(Stage<T>) * ARRAYS + kSlack;
  launch_k(kernel, grid, dim3(warps * 32), bytes, st, CL, args...);
  note_launch();
  return FRNNT_OK;
}

// The trial that the next launch makes (see frnnt_test_lose_scan_maps).
int g_trials = 0;
Trial g_trial;
template <int CL>
Trial trial_of() {
  if (CL == 1 || g_trials == 0) return Trial();
  --g_trials;
  return g_trial;
}

// Rows of 16-byte vectors throughout, and chunks that 32-bit offsets span.
bool vectors_ok(const frnnt_recurrence_dims& d, std::initializer_list<const void*> ptrs,
                std::initializer_list<long long> seqs, std::initializer_list<long long> steps) {
  if (d.D % 2) return false;
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return false;
  for (long long v : seqs)
    if (d.B > 1 && v * size_of(d.dtype) % 16) return false;
  for (long long v : steps)
    if (d.T > 1 && (v * size_of(d.dtype) % 16 || v > (1LL << 31) / kChunk / 4)) return false;
  return true;
}

template <typename T, bool VEC, typename... A>
int scan_fwd(const frnnt_recurrence_dims& d, cudaStream_t st, A... args) {
  return with_cluster(
      d, kTile<T, VEC>,
      [](auto CL) { return resident<T, 2, CL(), scan_fwd_kernel<T, VEC, CL(), stages_of(2)>>(); },
      [&](auto CL) {
        return launch_scan<T, kTile<T, VEC>, 2, CL(), scan_fwd_kernel<T, VEC, CL(), stages_of(2)>>(d, st, d, args...,
                                                                                                   trial_of<CL()>());
      });
}

template <typename T, bool VEC, typename... A>
int scan_bwd(const frnnt_recurrence_dims& d, cudaStream_t st, A... args) {
  return with_cluster(
      d, kTile<T, VEC>,
      [](auto CL) { return resident<T, 3, CL(), scan_bwd_kernel<T, VEC, CL(), stages_of(3)>>(); },
      [&](auto CL) {
        return launch_scan<T, kTile<T, VEC>, 3, CL(), scan_bwd_kernel<T, VEC, CL(), stages_of(3)>>(d, st, d, args...,
                                                                                                   trial_of<CL()>());
      });
}

template <typename T>
int fwd_of(bool vec, const frnnt_recurrence_dims& d, const void* x, const void* gate, const int32_t* lengths,
           const float* h0, void* h, float* h_last, float* saved, int32_t* status, cudaStream_t st) {
  return (vec ? scan_fwd<T, true, const T*, const T*, const int32_t*, const float*, T*, float*, float*, int32_t*>
              : scan_fwd<T, false, const T*, const T*, const int32_t*, const float*, T*, float*, float*, int32_t*>)(
      d, st, (const T*)x, (const T*)gate, lengths, h0, (T*)h, h_last, saved, status);
}
template <typename T>
int bwd_of(bool vec, const frnnt_recurrence_dims& d, const void* x, const void* gate, const int32_t* lengths,
           const float* saved, const void* dh, const float* dh_last, void* dx, void* dgate, float* dh0,
           int32_t* status, cudaStream_t st) {
  return (vec ? scan_bwd<T, true, const T*, const T*, const int32_t*, const float*, const T*, const float*, T*, T*,
                         float*, int32_t*>
              : scan_bwd<T, false, const T*, const T*, const int32_t*, const float*, const T*, const float*, T*, T*,
                         float*, int32_t*>)(d, st, (const T*)x, (const T*)gate, lengths, saved, (const T*)dh, dh_last,
                                            (T*)dx, (T*)dgate, dh0, status);
}

}  // namespace

bool refuse_clusters(bool on) {
  const bool prev = g_refuse_clusters;
  g_refuse_clusters = on;
  return prev;
}

int lose_scan_maps(int n, int round, bool quit, int tries) {
  const int prev = g_trials;
  g_trials = n < 0 ? 0 : n;
  g_trial.kind = quit ? Trial::kQuit : Trial::kLose;
  g_trial.round = round;
  g_trial.tries = tries < 0 ? 0u : tries < (int)sm100::kMaxTries ? (uint32_t)tries : sm100::kMaxTries;
  return prev;
}

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
    const bool vec = vectors_ok(*d, {x, gate, h}, {d->x_sb, d->gate_sb, d->h_sb}, {d->x_st, d->gate_st, d->h_st});
    const int rc = (d->dtype == FRNNT_BF16 ? fwd_of<__nv_bfloat16> : fwd_of<float>)(
        vec, *d, x, gate, lengths, h0, h, h_last, saved, status, st);
    if (rc) return rc;
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
    const bool vec = vectors_ok(*d, {x, gate, dh, dx, dgate}, {d->x_sb, d->gate_sb, d->dh_sb, d->dx_sb, d->dgate_sb},
                                {d->x_st, d->gate_st, d->dh_st, d->dx_st, d->dgate_st});
    const int rc = (d->dtype == FRNNT_BF16 ? bwd_of<__nv_bfloat16> : bwd_of<float>)(
        vec, *d, x, gate, lengths, saved, dh, dh_last, dx, dgate, dh0, status, st);
    if (rc) return rc;
  }
  return cudaGetLastError() == cudaSuccess ? FRNNT_OK : FRNNT_ERR_CUDA;
}

extern "C" FRNNT_API int frnnt_recurrence_step(const frnnt_step_dims* d, const void* x, const void* gate,
                                               const float* state, const int32_t* parent, const uint8_t* advance,
                                               void* h, float* new_state, int32_t* status, void* stream) {
  if (!d) return FRNNT_ERR_NULL;
  if (!dtype_ok(d->dtype)) return FRNNT_ERR_UNSUPPORTED;
  if (d->N < 1 || d->N > 65535 || d->S < 1 || d->D < 1 || d->D > (1 << 30) || d->x_sn < 0 || d->gate_sn < 0 ||
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
    const bool four = d->D % 4 == 0 && d->x_sn % 4 == 0 && d->gate_sn % 4 == 0 && aligned(x, 4 * es) &&
                      aligned(gate, 4 * es) && aligned(h, 4 * es) && aligned(state, 16) && aligned(new_state, 16);
    const int each = kStepThreads * (four ? 4 : 1);
    auto go = [&](auto kernel, auto type) {
      using T = decltype(type);
      launch_k(kernel, dim3((d->D + each - 1) / each, d->N), dim3(kStepThreads), 0, st, 1, *d, (const T*)x,
               (const T*)gate, state, parent, advance, (T*)h, new_state, status);
    };
    if (d->dtype == FRNNT_BF16)
      go(four ? step_kernel<__nv_bfloat16, 4> : step_kernel<__nv_bfloat16, 1>, __nv_bfloat16());
    else
      go(four ? step_kernel<float, 4> : step_kernel<float, 1>, float());
    note_launch();
  }
  return cudaGetLastError() == cudaSuccess ? FRNNT_OK : FRNNT_ERR_CUDA;
}
