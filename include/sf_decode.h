/*
 * sf_decode.h -- C ABI of decoding several tokens at a time on a pool of recurrent states:
 * the outputs of drafted tokens and the commit of those that were accepted, the
 * verification of drafts against the target's probabilities, and the pool's
 * housekeeping (copies, forks, compaction).
 *
 * A recurrent state cannot be taken back by shortening a length as a cache of keys
 * can.  So drafts are run from a state without advancing it, and the state is advanced
 * by the accepted ones afterwards: by sf_*_commit, or at the start of the next
 * sf_*_draft_step, which reads and writes each state once for both.
 *
 * Types, layouts, streams and errors are those of sf_gdn.h and sf_linattn.h: device
 * pointers, FP32 states [num_slots,H,V,K], BF16 or FP32 tokens, HK query/key heads that
 * divide H, no allocation, asynchronous on `stream`, no host synchronisation,
 * SF_ERR_UNSUPPORTED instead of another implementation.
 */
#ifndef SF_DECODE_H
#define SF_DECODE_H

#include "sf_linattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The most tokens of a sequence in one call of sf_*_draft_step (drafts, and pending
 * tokens) and sf_*_commit. */
#define SF_DRAFT_MAX 32

/* Accepted tokens that the states do not hold yet: of sequence n the first count[n] of P.
 * k [N,P,HK,K]; v [N,P,H,V]; gate, beta [N,P,H] FP32 (delta rule only); count int32 [N]
 * device, clamped into [0,P], or NULL: all P. */
typedef struct {
  int P;
  const void *k, *v;
  const float *gate, *beta;
  const int32_t *count;
} sf_pending;

/* ------------------------------------------------------------------------
 * Drafted tokens of N sequences.  Sequence n's state is first advanced by its pending
 * tokens and written back (pending NULL, or none of them: the state is only read).
 * From there the rule of sf_gdn_step (sf_linattn_step) runs over the first
 * num_tokens[n] of the T tokens on a copy that is not kept:
 *
 *     out_i = scale S_i q_i          S_i: the state after pending tokens and 0 .. i
 *
 *   shape          N, T (0 .. SF_DRAFT_MAX), H, HK, K == V (64 or 128), dtype, scale;
 *                  B is not used
 *   q, k [N,T,HK,K]; v, out [N,T,H,V] (dtype); gate, beta [N,T,H] FP32; decay [H]
 *   num_tokens     int32 [N] device, clamped into [0,T], or NULL: all T.  Rows of out
 *                  from num_tokens[n] on are zero, and nothing in the inputs' rows there
 *                  (NaN, infinities) reaches a result; the same for pending rows.
 *   state_cache, num_slots, state_indices: as sf_gdn_step.  Padding gives zero rows.
 * 16-byte aligned tensors, a 32-byte aligned state_cache; out overlaps no input.  The
 * tokens go through the chunk form (dot products with the state before eight tokens, and a
 * triangular solve over them), in FP32; BF16 outputs are rounded from that.  The state left
 * is to the bit that of sf_*_commit, and outputs are those of the step behind it to FP32's
 * rounding of the terms that they are summed from.
 * ---------------------------------------------------------------------- */
sf_status sf_gdn_draft_step(const sf_gdn_shape *shape, const void *q, const void *k, const void *v,
                            const float *gate, const float *beta, const int32_t *num_tokens,
                            const sf_pending *pending, float *state_cache, int num_slots,
                            const int32_t *state_indices, void *out, sf_stream_t stream);
sf_status sf_linattn_draft_step(const sf_gdn_shape *shape, const void *q, const void *k,
                                const void *v, const float *decay, const int32_t *num_tokens,
                                const sf_pending *pending, float *state_cache, int num_slots,
                                const int32_t *state_indices, void *out, sf_stream_t stream);

/* The pending tokens alone: advances each state by the first num_tokens[n] of its T
 * tokens (shape->T). */
sf_status sf_gdn_commit(const sf_gdn_shape *shape, const void *k, const void *v, const float *gate,
                        const float *beta, const int32_t *num_tokens, float *state_cache,
                        int num_slots, const int32_t *state_indices, sf_stream_t stream);
sf_status sf_linattn_commit(const sf_gdn_shape *shape, const void *k, const void *v,
                            const float *decay, const int32_t *num_tokens, float *state_cache,
                            int num_slots, const int32_t *state_indices, sf_stream_t stream);

/* ------------------------------------------------------------------------
 * Verification of drafted tokens.  With p_i the target's probabilities of token i of a
 * sequence, q_i the draft's and x_i the drafted token:
 *
 *     draft i is accepted if the ones before it are and  u_i q_i(x_i) < p_i(x_i);
 *     after a accepted drafts one token is drawn from  max(p_a - q_a, 0), from p_a if all
 *     num_drafts[n] are accepted or that is zero everywhere:
 *     the lowest y with  w(0) + ... + w(y) > u_T (w(0) + ... + w(V-1)).
 *
 * so that every token has the target's distribution.
 *   target_probs   [N,T+1,V]; draft_probs [N,T,V] of the same dtype (BF16 or FP32), or
 *                  NULL: a draft is certain of its token (q_i(x_i) = 1, others 0).  They
 *                  need not be normalised for the draw.  Rows are contiguous; the
 *                  strides are in elements, between sequences and between rows.
 *   draft_tokens   int32 [N,T]; one outside [0,V) is rejected
 *   uniforms       [N,T+1] FP32 in [0,1): T for the tests, one for the draw (below 0 it
 *                  draws the first token with weight, from 1 on and as a NaN the last)
 *   num_drafts     int32 [N] or NULL (T); at most T of them count; negative: padding
 *   tokens         int32 [N,T+1]: the accepted drafts, the drawn token, then -1.  The
 *                  drawn token is -1 where the weights' sum is not positive or not finite
 *                  in FP32.
 *   num_tokens     int32 [N]: accepted drafts + 1 (0 for padding): the tokens gained, and
 *                  the number to commit of [last token, draft 0, draft 1, ...].  -1: a
 *                  kernel's bounded internal wait expired (2 s; there is no workspace to
 *                  say so in), and the sequence's tokens are undefined
 * A negative weight or a NaN counts as zero.  The test's products are exact.  The draw's sums
 * are exact to 2^-38 of the weights' sum at every V, for draft probabilities that are not
 * negative and sums from 2^-100 on, so that a draw depends on how they are split only where
 * u_T times the sum lies that near a border between two tokens.
 * N >= 0, T >= 0 (T = 0: one token is drawn from p_0), V >= 1.  Outputs overlap no input.
 * ---------------------------------------------------------------------- */
typedef struct {
  int N, T, V;
  sf_dtype dtype;
  int64_t target_seq, target_row, draft_seq, draft_row;   /* strides, elements */
} sf_verify_shape;

sf_status sf_draft_verify(const sf_verify_shape *shape, const void *target_probs,
                          const int32_t *draft_tokens, const float *uniforms,
                          const void *draft_probs, const int32_t *num_drafts, int32_t *tokens,
                          int32_t *num_tokens, sf_stream_t stream);

/* Failure-detection testing only, as sf_testing_inject_timeout: in the next sf_draft_verify on
 * the calling host thread the first CTA of every sequence gives up its wait for the others'
 * sums at once.  num_tokens then reads -1 (0 for padding); later calls are normal. */
sf_status sf_testing_inject_verify_timeout(void);

/* ------------------------------------------------------------------------
 * The pool's slots.  The layers of a model keep one cache each, and a slot's states lie
 * at the same index of all of them.
 *   caches         host array of num_caches device pointers, 16-byte aligned: cache c is
 *                  [num_slots] slots of slot_bytes[c] bytes (a multiple of 16) of any type
 *   reserved       uint8 [num_slots] device or NULL: slots (non-zero) that are not
 *                  written, moved or given out: states kept for later, sequences that
 *                  state_indices does not name.  Slot 0 is never used (padding's index).
 *   workspace      sf_state_workspace(num_slots, rows) bytes, 16-byte aligned, no initial
 *                  contents; rows: M of a fork, N of a compaction.  May be NULL for up to
 *                  4096 slots, 1024 rows and 64 caches, unless new_indices overlaps an
 *                  input.  Up to 256 rows of those do not use it; more are faster with it.
 * An index outside [1, num_slots) is padding.  num_slots <= SF_MAX_SLOTS.
 *
 * sf_state_copy: dst[i] becomes a copy of src[i] (int32 [M] device each); a pair with
 *   padding in it is skipped.  The dst are distinct, and none is also a src (caller's
 *   responsibility).
 * sf_state_fork: row i continues sequence parents[i] of the N sequences state_indices.
 *   The first row of a slot keeps it, unless it is reserved; the others get a copy in the
 *   lowest slots that no row keeps and that are not reserved, in the rows' order.  So the
 *   slots of sequences without a row are free.  new_indices[i]: its slot; -1 where
 *   parents[i] is outside [0,N) or padding, or no slot is left.
 * sf_state_compact: the slots that state_indices names and that are not reserved, L of
 *   them, are brought into the lowest L that are not reserved: those above, in order, move
 *   into the gaps, in order.  new_indices[n]: where state_indices[n] is now (padding and
 *   reserved slots stay).  Sequences that name one slot go on sharing it.
 * new_indices may be state_indices (or parents), and overlaps no input otherwise.  Slots that
 * nothing moves into keep what they held.
 * ---------------------------------------------------------------------- */
#define SF_MAX_SLOTS (1 << 18)

typedef struct {
  int num_slots, num_caches;
  void *const *caches;
  const size_t *slot_bytes;
} sf_state_pool;

size_t sf_state_workspace(int num_slots, int rows);
sf_status sf_state_copy(const sf_state_pool *pool, const int32_t *src, const int32_t *dst, int M,
                        sf_stream_t stream);
sf_status sf_state_fork(const sf_state_pool *pool, const int32_t *state_indices, int N,
                        const int32_t *parents, int M, const uint8_t *reserved,
                        int32_t *new_indices, void *workspace, size_t ws_bytes,
                        sf_stream_t stream);
sf_status sf_state_compact(const sf_state_pool *pool, const int32_t *state_indices, int N,
                           const uint8_t *reserved, int32_t *new_indices, void *workspace,
                           size_t ws_bytes, sf_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SF_DECODE_H */
