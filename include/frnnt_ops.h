/*
 * frnnt operators beside the transducer loss -- C ABI.
 *
 *   token log-probabilities   log-softmax values of given tokens, entropy and the best alternatives of rows
 *                             of logits, and the gradient of the logits
 *   gated linear recurrence   the time recurrence of a prediction network or encoder layer: forward,
 *                             backward, and one step of many hypotheses
 *   dropout                   from a counter-based generator; the mask is never stored
 *
 * Same manner as frnnt.h: device pointers on the current device, owned by the caller; nothing is allocated,
 * nothing is synchronised, no data is kept between calls; work is queued on `stream`; host-side errors are
 * FRNNT_ERR_* codes returned before any launch.  Calls may come from several host threads at once and may be
 * captured into CUDA graphs.  Differences, because these calls take views of larger arrays and can be a few
 * microseconds long:
 *   - rows may be strided (strides in elements); pointers need the alignment of their element type only.  Where a
 *     row does not start or end on a 16-byte boundary, the whole aligned 16-byte unit around that end may be read (up
 *     to 15 bytes before or behind the row, whose values do not matter); writes stay inside the rows;
 *   - no workspace is needed;
 *   - `status` may be NULL.  When given, invalid device-side values OR their FRNNT_STATUS_* bits into it: the
 *     call never clears it, the caller does.  After a bit was set the outputs of the rows concerned are
 *     unspecified; no access out of bounds happens either way (but for those units).  FRNNT_STATUS_TIMEOUT: a
 *     bounded wait of the recurrence's blocks for each other gave up (after about 2 s; the call then ends within a
 *     few seconds, and later calls are not concerned).
 * Outputs must not overlap inputs except where a call says so.
 */
#ifndef FRNNT_OPS_H
#define FRNNT_OPS_H

#include "frnnt.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FRNNT_MAX_TOKENS 32   /* given tokens per row */
#define FRNNT_MAX_TOP 32      /* best alternatives per row */
#define FRNNT_NO_TOKEN (-1)   /* a token position that is not given */
#define FRNNT_SCAN_CHUNK 128  /* time steps between two saved states of the recurrence */

enum {
  FRNNT_STATUS_INDEX = 16     /* frnnt_recurrence_step: parent[n] outside [0, S) */
};

/* ------------------------------------------------------------------ token log-probabilities */

typedef struct {
  int N, V;            /* rows (1 .. 2^27), vocabulary size (1 .. 2^30)                        */
  int K;               /* given tokens per row, 0 .. FRNNT_MAX_TOKENS                          */
  int top;             /* best alternatives per row, 0 .. min(V, FRNNT_MAX_TOP)                */
  frnnt_dtype dtype;   /* element type of logits and dlogits                                   */
  long long ld;        /* elements from one row of logits to the next, >= V                    */
  long long ldd;       /* the same for dlogits (backward only), >= V                           */
  float* lse_rest;     /* [N] fp32 on the device or NULL: written by the forward call, read by
                          the backward call (see there)                                        */
} frnnt_logprob_dims;

/* For every row z of logits [N, V], with lse = log sum_j exp(z_j) and log p_j = z_j - lse:
 *   logp     [N, K] fp32    log p_{tokens[n,k]}; 0 where tokens[n,k] is FRNNT_NO_TOKEN
 *   entropy  [N] fp32       -sum_j p_j log p_j  (natural logarithm; p log p = 0 at p = 0)
 *   lse      [N] fp32; lse_rest [N], where given, is what rounding to fp32 took from it
 *   top_logp [N, top] fp32, top_ids [N, top] int32   the `top` largest logits' log-probabilities, largest
 *                           first, and their columns; equal logits: the lowest column first
 * tokens [N, K] int32 (may be NULL with K = 0); the same token may be given more than once.  logp / top_logp /
 * top_ids may be NULL where K / top is 0.  Any other token outside [0, V) sets FRNNT_STATUS_LABEL.
 * Logits of -inf are allowed and have probability 0.  A row that holds nothing else has lse = -inf, logp and
 * top_logp = -inf, entropy = 0 and top_ids 0, 1, ...  A NaN or +inf in a row makes that row's values NaN (its
 * top_ids stay in range; NaN ranks last).
 * Sums are held in fp32.  Equal inputs give equal outputs, bit for bit. */
FRNNT_API int frnnt_token_logprobs(const frnnt_logprob_dims* d, const void* logits, const int32_t* tokens,
                                   float* logp, float* entropy, float* lse, float* top_logp, int32_t* top_ids,
                                   int32_t* status, void* stream);

/* The gradient of sum(logp * dlogp) + sum(entropy * dentropy) + sum(top_logp * dtop) for the logits:
 *   dz_j = sum_k dlogp_k ([j = token_k] - p_j) + sum_i dtop_i ([j = id_i] - p_j)
 *          - dentropy p_j (log p_j + entropy)
 * lse, entropy and top_ids are the forward call's; dlogp [N, K], dentropy [N] and dtop [N, top] are fp32 and may
 * each be NULL (no such term; tokens and top_ids are then not read, entropy only with dentropy).  A token that is
 * FRNNT_NO_TOKEN contributes nothing; a token or top id outside [0, V) otherwise sets FRNNT_STATUS_LABEL and
 * contributes nothing.  p_j comes from lse and, where given, lse_rest, as the forward call wrote them; without
 * lse_rest every p_j is off by a factor of exp(2^-24 |lse|) at most, and in a row of huge logits (all of them the
 * type's lowest value, say) p means nothing.  dlogits [N, ldd] has the type of the logits, rounded once; it may
 * be the logits' own memory (same address and ldd = ld).  A row of -inf only gets zeros, and so does a row without
 * any term (no given token, dtop and dentropy NULL) whatever it holds; elements of the rows past V are not
 * written. */
FRNNT_API int frnnt_token_logprobs_bwd(const frnnt_logprob_dims* d, const void* logits, const int32_t* tokens,
                                       const float* lse, const float* entropy, const int32_t* top_ids,
                                       const float* dlogp, const float* dentropy, const float* dtop, void* dlogits,
                                       int32_t* status, void* stream);

/* ------------------------------------------------------------------ gated linear recurrence */

typedef struct {
  int B, T, D;               /* sequences (1 .. 65535), steps, channels (1 .. 2^30)            */
  frnnt_dtype dtype;         /* element type of x, gate, h, dh, dx and dgate                   */
  /* strides in elements from one sequence (_sb) and one step (_st) to the next; channels are contiguous.
   * Inputs: any strides >= 0, a step at most 2^30 elements.  Outputs (h, dx, dgate): no two elements may
   * share an address.                                                                          */
  long long x_sb, x_st, gate_sb, gate_st, h_sb, h_st;
  long long dh_sb, dh_st, dx_sb, dx_st, dgate_sb, dgate_st;   /* backward only                  */
} frnnt_recurrence_dims;

/* With a_t = sigmoid(gate_t), per channel, from h_{-1} = h0 (zero when NULL):
 *   h_t = a_t h_{t-1} + (1 - a_t) x_t                                  0 <= t < lengths[b]
 *   lengths [B] int32 or NULL (= T): 0 is allowed; outside [0, T] sets FRNNT_STATUS_LENGTH
 *   h       [B, T, D]   rows t >= lengths[b] are written as 0; x and gate are not read there
 *   h_last  [B, D] fp32 the state after the sequence's last step (h0 for length 0), unrounded
 *   saved   [B, ceil(T / FRNNT_SCAN_CHUNK), D] fp32 or NULL: the states before steps 0, 128, 256, ... that the
 *           backward call starts from (those at or past lengths[b] are not written)
 *   h0      [B, D] fp32 or NULL
 * The state is carried in fp32 and rounded only where it is written to h; a and 1 - a are each good to a relative
 * 2^-21 + |gate| 2^-24 (the rounding of an fp32 gate costs them as much). */
FRNNT_API int frnnt_recurrence_fwd(const frnnt_recurrence_dims* d, const void* x, const void* gate,
                                   const int32_t* lengths, const float* h0, void* h, float* h_last, float* saved,
                                   int32_t* status, void* stream);

/* The gradients of sum(h * dh) + sum(h_last * dh_last), with g_t = dh_t + a_{t+1} g_{t+1}:
 *   dx_t = (1 - a_t) g_t,  dgate_t = a_t (1 - a_t) (h_{t-1} - x_t) g_t,  dh0 = a_0 g_0
 * x, gate, lengths as in the forward call, saved as it wrote them; the states between are computed again from
 * them, in fp32 (h is not read).  dh [B, T, D] (rows t >= lengths[b] are not read), dh_last [B, D] fp32 or NULL,
 * dh0 [B, D] fp32 output or NULL.  Rows t >= lengths[b] of dx and dgate are written as 0.  Inputs whose strides
 * repeat elements (stride 0) get one gradient row for every use. */
FRNNT_API int frnnt_recurrence_bwd(const frnnt_recurrence_dims* d, const void* x, const void* gate,
                                   const int32_t* lengths, const float* saved, const void* dh, const float* dh_last,
                                   void* dx, void* dgate, float* dh0, int32_t* status, void* stream);

typedef struct {
  int N, S, D;               /* rows (1 .. 65535), rows of state, channels (1 .. 2^30)        */
  frnnt_dtype dtype;         /* element type of x, gate and h                                  */
  long long x_sn, gate_sn;   /* elements from one row to the next (inputs: >= 0)               */
} frnnt_step_dims;

/* One step of N rows (the hypotheses of a beam): row n continues the state of its parent,
 *   new_state_n = a_n state_{parent[n]} + (1 - a_n) x_n,  a_n = sigmoid(gate_n)     where advance[n] != 0
 *   new_state_n = state_{parent[n]}                                                 where advance[n] == 0
 *   h_n = new_state_n, rounded to the input type
 *   parent  [N] int32 or NULL (row n; needs N <= S); several rows may share a parent
 *   advance [N] bytes or NULL (every row advances); x and gate are not read where it is 0
 *   state [S, D] fp32, new_state [N, D] fp32, h [N, D]
 * new_state may be state's own memory when parent is NULL. */
FRNNT_API int frnnt_recurrence_step(const frnnt_step_dims* d, const void* x, const void* gate, const float* state,
                                    const int32_t* parent, const uint8_t* advance, void* h, float* new_state,
                                    int32_t* status, void* stream);

/* ------------------------------------------------------------------ dropout */

typedef struct {
  long long R, C;            /* rows, elements per row (both >= 1)                             */
  frnnt_dtype dtype;
  long long x_ld, y_ld;      /* elements from one row to the next, >= C                        */
  double p;                  /* probability of dropping, 0 .. 1; used in 65536ths, rounded     */
  uint64_t seed, offset;     /* key, and first counter                                         */
} frnnt_dropout_dims;

/* y = x / (1 - p) where the element stays, 0 where it is dropped (also if x is NaN or infinite there).
 * Element e (row-major index r * C + c) takes 16 bits of the Philox4x32-10 block of key seed and counter
 * (offset + e / 8) mod 2^64, the counter's upper 64 bits 0 ("Parallel Random Numbers: As Easy as 1, 2, 3"):
 * half-word e % 8 of its four words, low halves first; it stays where those bits are >= P = round(65536 p), and is
 * scaled by 65536 / (65536 - P).  So the mask depends on seed, offset and the element's index alone: not on type, strides or device, and the same
 * call on dy gives dx.  Arrays that follow each other in one stream of numbers take offsets at least
 * ceil(R C / 8) apart.
 *   rng  [2] uint64 device array or NULL: when given, rng[0] replaces d->seed and rng[1] is added to d->offset (a
 *        captured graph draws new numbers at each replay that way)
 * y may be x's own memory (same address and y_ld = x_ld). */
FRNNT_API int frnnt_dropout(const frnnt_dropout_dims* d, const void* x, void* y, const uint64_t* rng, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FRNNT_OPS_H */
