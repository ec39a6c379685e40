/*
 * sf_linattn.h -- C ABI of the operators around the gated delta rule (sf_gdn.h):
 * linear attention with a decay for each head (chunked forward, paged prefill,
 * backward), the single-token steps of both rules on a paged state pool, and
 * the pass that makes queries and keys (norm of each head and rotary position).
 *
 * Types, layouts, workspaces, streams and errors are those of sf_gdn.h: device
 * pointers, FP32 states [N,H,V,K], BF16 or FP32 tokens, HK query/key heads that
 * divide H, int32 cu_seqlens, no allocation, asynchronous on `stream`, no host
 * synchronisation, SF_ERR_UNSUPPORTED instead of another implementation.
 */
#ifndef SF_LINATTN_H
#define SF_LINATTN_H

#include "sf_gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Linear attention with a decay for each head.  With lam_h = exp(decay[h]):
 *
 *     S_t   = lam S_{t-1} + outer(v_t, k_t)          S [V,K], FP32
 *     out_t = scale S_t q_t                          (the updated state is read)
 *
 *   decay          [H] FP32 natural log, finite or -inf; <= 0 in use (0: plain
 *                  linear attention; -inf: a token sees itself only).  It is a
 *                  fixed property of the head: no gradient of it is formed.
 *   shape, q, k, v, initial_state, cu_seqlens, out, final_state: as
 *                  sf_gdn_chunk_fwd.  K == V, either 64 or 128, BF16 or FP32.
 *   workspace      sf_linattn_fwd_workspace(shape, packed) bytes, 16-byte aligned,
 *                  its first 256 bytes zero before the first use; packed != 0
 *                  when cu_seqlens is given.
 * Outputs overlap no input and no workspace; final_state may be initial_state.
 * An empty sequence hands its initial state through.  Rows past cu_seqlens[N]
 * are never written, and nothing in them (NaN, infinities) reaches a result.
 * A NaN or infinity inside a sequence reaches that head's results from the
 * start of its block of 64 tokens on, counted from the sequence's start (the
 * products run over whole blocks); what the backward walks from the end (dk, dv,
 * d_initial_state) from the end of its block, counted from the sequence's end.
 * It reaches no other sequence or head.
 *
 * FP32 outputs and states carry FP32 accuracy.  With BF16 tokens, out (in the
 * backward dq, dk and dv) is rounded from FP32 sums of which two operands are
 * rounded to BF16 before: the masked products of q and k, and the state (the
 * cotangent) as a token reads it.  Its error is 1.4 times that of rounding the
 * result alone, 2.4e-3 in the 2-norm.  Sequences of up to 64 tokens keep 16 bits
 * of the products, so that with no initial state theirs is the result's rounding
 * alone.  The state is carried and returned with FP32 accuracy; a call that
 * returns none (no final state, no d_initial_state) adds to it rows of 16 bits.
 * FP32 tokens have none of these roundings.
 * ---------------------------------------------------------------------- */
size_t sf_linattn_fwd_workspace(const sf_gdn_shape *shape, int packed);
sf_status sf_linattn_chunk_fwd(const sf_gdn_shape *shape, const void *q, const void *k,
                               const void *v, const float *decay, const float *initial_state,
                               const int32_t *cu_seqlens, int output_final_state, void *out,
                               float *final_state, void *workspace, size_t ws_bytes,
                               sf_stream_t stream);

/* The forward advancing a pool of states [num_slots,H,V,K] in place; state_indices,
 * has_initial_state and padding as sf_gdn_paged_chunk_fwd. */
sf_status sf_linattn_paged_chunk_fwd(const sf_gdn_shape *shape, const void *q, const void *k,
                                     const void *v, const float *decay, float *state_cache,
                                     int num_slots, const int32_t *state_indices,
                                     const uint8_t *has_initial_state, const int32_t *cu_seqlens,
                                     void *out, void *workspace, size_t ws_bytes,
                                     sf_stream_t stream);

/* ------------------------------------------------------------------------
 * Backward of sf_linattn_chunk_fwd: gradients of <d_out, out> + <d_final_state,
 * final_state>.  With dS_t the cotangent of S_t from everything after token t:
 *
 *     D_t  = dS_t + scale outer(d_out_t, q_t)        dS_{t-1} = lam D_t
 *     dq_t = scale S_t^T d_out_t    dk_t = D_t^T v_t    dv_t = D_t k_t
 *
 *   d_out [B,T,H,V]; d_final_state [N,H,V,K] or NULL (zeros); dq, dk [B,T,HK,K]
 *   (sums over each block of H / HK value heads), dv [B,T,H,V];
 *   d_initial_state [N,H,V,K] or NULL (not computed).  Inactive rows of the
 *   gradients are not written.  Outputs overlap no input.  K == V, either 64 or
 *   128, BF16 or FP32.
 * ---------------------------------------------------------------------- */
size_t sf_linattn_bwd_workspace(const sf_gdn_shape *shape, int packed);
sf_status sf_linattn_chunk_bwd(const sf_gdn_shape *shape, const void *q, const void *k,
                               const void *v, const float *decay, const float *initial_state,
                               const int32_t *cu_seqlens, const void *d_out,
                               const float *d_final_state, void *dq, void *dk, void *dv,
                               float *d_initial_state, void *workspace, size_t ws_bytes,
                               sf_stream_t stream);

/* ------------------------------------------------------------------------
 * Decoding: one token of each of N sequences, on a pool of states that is read
 * and written in place.
 *   shape          N sequences, H, HK, K == V (64 or 128), dtype, scale; B and T
 *                  are not used
 *   q, k [N,HK,K]; v, out [N,H,V] (dtype); 16-byte aligned
 *   state_cache    [num_slots,H,V,K] FP32, 16-byte aligned; the pool may hold
 *                  more than 2^31 elements
 *   state_indices  int32 [N] device: sequence n's slot.  Positive indices are
 *                  unique (caller's responsibility); an index <= 0 or >=
 *                  num_slots is padding: zero output, the pool untouched.
 *                  NULL: sequence n owns slot n (num_slots >= N).
 * sf_linattn_step: the rule above with decay [H].
 * sf_gdn_step: the gated delta rule of sf_gdn.h with gate, beta [N,H] FP32.
 * Both compute in FP32.  N == 0 does nothing.
 * ---------------------------------------------------------------------- */
sf_status sf_linattn_step(const sf_gdn_shape *shape, const void *q, const void *k, const void *v,
                          const float *decay, float *state_cache, int num_slots,
                          const int32_t *state_indices, void *out, sf_stream_t stream);
sf_status sf_gdn_step(const sf_gdn_shape *shape, const void *q, const void *k, const void *v,
                      const float *gate, const float *beta, float *state_cache, int num_slots,
                      const int32_t *state_indices, void *out, sf_stream_t stream);

/* ------------------------------------------------------------------------
 * Norm of each query and key head, and the position rotation, in one pass.
 *
 *     y = x * r * w        r = rsqrt(mean(x^2) + eps)       SF_NORM_RMS
 *                          r = 1 / max(||x||, eps)          SF_NORM_L2
 *     (out_a, out_b) = (y_a c - y_b s, y_b c + y_a s)       for each rotary pair p
 *
 * over the heads q [rows,H,D] and k [rows,HK,D] (rows = tokens of all batch
 * rows).  Pair p < rotary_dim / 2 is the elements (p, p + rotary_dim / 2), or
 * (2p, 2p + 1) with interleaved != 0; the elements from rotary_dim on are not
 * rotated.  Its angle's (c, s) is cos_sin[position][p] with the position of its
 * axis: the first sections[0] pairs take positions[0][row], the next
 * sections[1] pairs positions[1][row], and so on (time, height and width of an
 * image or video patch; one axis for text).
 *
 *   rows_stride_q, rows_stride_k   elements between consecutive tokens of q and
 *       k (a multiple of 16 bytes; >= H D, HK D), so that both may be slices of
 *       one fused projection; a token's heads are contiguous.  q_out and k_out
 *       are contiguous and may be q and k themselves where those are.
 *   q_weight, k_weight  [D] FP32 or NULL (ones)
 *   cos_sin             [table_rows, rotary_dim / 2, 2] FP32
 *   positions           [axes, rows] int32; a value outside [0, table_rows) is
 *                       clamped into it
 *   D 64 or 128; rotary_dim a multiple of 8, at most D (0: no rotation, then
 *   cos_sin, positions and sections are not used); 1 to 4 axes whose sections
 *   sum to rotary_dim / 2.  All arithmetic is FP32, rounded once.  A NaN in a head
 *   gives NaN in all of that head (both norms, forward and backward), no other.
 * ---------------------------------------------------------------------- */
typedef enum { SF_NORM_RMS = 0, SF_NORM_L2 = 1 } sf_norm;

typedef struct {
  int64_t rows;
  int H, HK, D;
  sf_dtype dtype;
  sf_norm norm;
  float eps;
  int rotary_dim, interleaved, table_rows, axes;
  int sections[4];
  int64_t rows_stride_q, rows_stride_k;
} sf_qk_shape;

sf_status sf_qk_norm_rope_fwd(const sf_qk_shape *shape, const void *q, const void *k,
                              const float *q_weight, const float *k_weight, const float *cos_sin,
                              const int32_t *positions, void *q_out, void *k_out,
                              sf_stream_t stream);

/* Its backward: d_q_out, d_k_out contiguous -> dq, dk contiguous, dq_weight, dk_weight [D]
 * FP32 or NULL (each is computed only if given).  The weights' gradients are summed in a
 * fixed order.  workspace: sf_qk_norm_rope_bwd_workspace bytes, 16-byte aligned, no
 * initial contents. */
size_t sf_qk_norm_rope_bwd_workspace(const sf_qk_shape *shape);
sf_status sf_qk_norm_rope_bwd(const sf_qk_shape *shape, const void *q, const void *k,
                              const float *q_weight, const float *k_weight, const float *cos_sin,
                              const int32_t *positions, const void *d_q_out, const void *d_k_out,
                              void *dq, void *dk, float *dq_weight, float *dk_weight,
                              void *workspace, size_t ws_bytes, sf_stream_t stream);

/* Failure-detection testing only, as sf_testing_inject_timeout: in the next BF16 call of
 * sf_linattn_chunk_fwd, sf_linattn_paged_chunk_fwd or sf_linattn_chunk_bwd on the calling
 * host thread no CTA's table of factors is ever announced, and every internal wait gives up
 * after `tries` (1 .. 10000) tries of 20 us at the most each.  The status word then reads
 * SF_ERR_TIMEOUT, and the call's outputs are undefined; later calls are normal. */
sf_status sf_testing_inject_linattn_timeout(int tries);

#ifdef __cplusplus
}
#endif
#endif /* SF_LINATTN_H */
