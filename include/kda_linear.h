/*
 * kda_linear.h -- a linear-attention layer with ONE decay a head, beside the
 * KDA core (whose decay is per key channel and whose write is a delta rule), and
 * the head norm and position rotation in front of it and of the latent layer.
 *
 * Per (sequence, head), with an fp32 K x V state S and a log-decay g that is a
 * number a head or a number a token and head:
 *
 *     S   <- exp(g_t) S + k_t v_t^T          decay, write
 *     o_t  = scale * S^T q_t                 read-out, updated state
 *
 * q and k are taken as they are (kda_head_norm_rope normalises and rotates
 * them); kda_output_gate_norm (kda.h) is the layer's epilogue as it is KDA's.
 * As in KDA there is a chunked form for prompts and a token step for decode, on
 * the same pools of states.
 *
 * Conventions are those of kda.h: device pointers, nothing allocated, nothing
 * kept between calls, work enqueued on `stream` without synchronising,
 * arguments validated before anything is enqueued, status codes of kda_status.
 *
 * Layouts (T = tokens, H = heads of v and o, Hk = heads of q and k, Hk | H):
 *   q, k    [T, Hk, K]   head h reads q and k of head h / (H / Hk)
 *   v, o    [T, H, V]
 *   g       fp32, element h of token t at g[t * g_stride + h]: g_stride = 0 is
 *           one fixed decay a head, otherwise at least H.  g <= 0; -inf clears the
 *           state.  Positive values are accepted while their sum over any 128
 *           tokens stays below 40.
 *   states  [N, H, V, K] fp32, key dim contiguous, as in kda.h
 * q, k and v have token strides of their own (*_stride, elements, multiples of
 * 8, at least heads * 128: slices of a fused projection); o is dense.
 * q, k, v, o are `dtype` (kda_dtype).  K = V = 128.  Rows are 16-byte aligned.
 */
#ifndef KDA_LINEAR_H_
#define KDA_LINEAR_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_ROPE_MAX_AXES 4

/*
 * RMS norm of each head and rotation by the token's position, of q and (if Hk > 0)
 * of k, in one pass:
 *   y = x / sqrt(mean(x^2) + eps) * weight      over the head's D channels, if norm
 *   pairs (a, b) of the rot_dim channels from rot_offset on:
 *     (a cos t - b sin t, b cos t + a sin t),   t = positions[axis(i)][token] * inv_freq[i]
 *   q       [T, Hq, D] dtype, q_stride elements between tokens; k [T, Hk, D] likewise
 *   q_weight, k_weight  fp32 [D], 16-byte aligned, or NULL: ones; not looked at without the norm
 *   positions  int32 [n_axes, T]; a token whose position on axis 0 is negative is
 *           padding: its rows of q_out and k_out are left as they were.  NULL
 *           with rot_dim = 0: every token is real
 *   sections   HOST int [n_axes]: the first sections[0] of the rot_dim / 2 pairs turn
 *           by axis 0, the next sections[1] by axis 1, ... (their sum is rot_dim / 2);
 *           NULL with n_axes = 1
 *   inv_freq   fp32 [rot_dim / 2]
 *   interleaved  0: pair i is channels (i, i + rot_dim / 2) of the rotated part;
 *           1: channels (2 i, 2 i + 1)
 *   q_out, k_out  like q and k, with strides of their own; q_out may be q and k_out
 *           may be k (in place, with the same stride), and share no memory otherwise
 * D is a multiple of 16 up to 256, rot_dim a multiple of 16 up to D (0: no rotation),
 * rot_offset a multiple of 8 up to D - rot_dim, strides multiples of 8.  Everything
 * is computed in fp32 and rounded once; angles are reduced to a turn before they
 * are rounded (a position of 2^24 costs no accuracy; of 2^31, 2^-17 of a radian).
 * T = 0 is a no-op.
 */
int kda_head_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                       const float *q_weight, const float *k_weight, float eps, int norm,
                       const int32_t *positions, const int *sections, int n_axes,
                       const float *inv_freq, int rot_offset, int rot_dim, int interleaved,
                       void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride,
                       int64_t n_tokens, int Hq, int Hk, int D, int dtype, void *stream);

/* Device workspace (256-byte aligned) of kda_linear_chunk_fwd: the states between the
 * parts that long sequences are cut into, and lists of several sequences.  0: none is needed; 0 on invalid sizes. */
size_t kda_linear_chunk_workspace_bytes(int64_t total_tokens, int n_seqs, int H, int dtype);

/*
 * Chunked forward over N packed sequences (prompts).
 *   cu_seqlens     int32 [N+1], non-decreasing from 0 to at most T; NULL = N sequences of
 *                  equal length T / N (N divides T)
 *   state_indices, n_slots, initial_state, final_state  as in kda_chunk_fwd:
 *                  [N, H, V, K], or pools of n_slots states indexed by
 *                  state_indices (distinct); initial_state NULL = zeros,
 *                  final_state NULL = not written, final_state may be initial_state
 *   o              shares no memory with the inputs or the states
 * bf16 runs on the tensor cores: chunks of 128 tokens, fp32 accumulation and states;
 * the scores and the state enter the products that give o as bf16 (two roundings
 * beside o's own; the scores of a sequence's first 128 tokens as two terms, 16 bits); what is written to the state is
 * split into three bf16 terms, so that the states are as exact as fp32 sums.  fp32 runs on the CUDA cores, token by
 * token.  Long sequences are cut into segments that are worked on at the same time.
 * A zero-length sequence hands back its initial state (or zeros).  A slot outside
 * [0, n_slots) gives NaN in that sequence's rows of o and leaves the pools alone.
 * Tokens of a sequence whose offsets are decreasing or out of range are not written,
 * nor is its state.  (Offsets that step back make sequences overlap: which of them are
 * then computed is not defined, nothing outside the buffers is read or written.)
 * Values that are not finite reach the rows behind them of their own
 * sequence and no other: a NaN or an infinity in v of token j makes that channel NaN
 * (fp32 inputs: NaN or infinite) from row j on, and in the state.  Results do not depend on
 * timing; where a sequence is cut, and with it the rounding, follows from T, H and
 * the offsets.  A bounded wait of a kernel that gave up (a copy that never landed)
 * gives NaN in what that part had to write.
 *
 * Limits: N <= 65535, H <= 65535, T < 2^31, T / 128 * H and N * H < 2^30.
 */
int kda_linear_chunk_fwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                         const void *v, int64_t v_stride, const float *g, int64_t g_stride,
                         const float *initial_state, float *final_state,
                         const int32_t *state_indices, int64_t n_slots, void *o,
                         const int32_t *cu_seqlens, int n_seqs, int64_t total_tokens, int H,
                         int Hk, int K, int V, float scale, int dtype, void *workspace,
                         size_t workspace_bytes, void *stream);

/*
 * One token for each of N sequences on a pooled state, in place.
 *   q, k [N, Hk, K]   v, o [N, H, V]   g as above (token n)
 *   state_pool  [n_slots, H, V, K] fp32; state_indices int32 [N], distinct, NULL =
 *               slot n (then n_slots >= N).  A slot outside [0, n_slots) leaves the
 *               pool alone and gives NaN in that sequence's o.
 * The decay is applied as the sum of two floats, so that a slow one does not add up its rounding over
 * the steps (an infinity in the state may become NaN by it).
 * N = 0 is a no-op.
 */
int kda_linear_step(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                    const void *v, int64_t v_stride, const float *g, int64_t g_stride,
                    float *state_pool, const int32_t *state_indices, int64_t n_slots, void *o,
                    int N, int H, int Hk, int K, int V, float scale, int dtype, void *stream);

/*
 * S tokens a sequence (speculative verify): q, k [N, S, Hk, K], v, o [N, S, H, V], token
 * n S + t at n S + t strides.  Slots and counts as for kda_recurrent_multi_step: the
 * state after token t goes to slot state_indices[n][t]; the first token starts from slot
 * state_indices[n][num_accepted[n] - 1] (num_accepted NULL: [n][0]).  A count outside
 * [1, S] or a slot outside [0, n_slots) leaves the sequence's slots alone and gives
 * NaN in its o; slots of different sequences must not overlap.
 */
int kda_linear_multi_step(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                          const void *v, int64_t v_stride, const float *g, int64_t g_stride,
                          float *state_pool, const int32_t *state_indices,
                          const int32_t *num_accepted, int64_t n_slots, void *o, int N, int S,
                          int H, int Hk, int K, int V, float scale, int dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LINEAR_H_ */
