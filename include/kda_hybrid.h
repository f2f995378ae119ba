/*
 * kda_hybrid.h -- the operators around the KDA core in a hybrid decoder's
 * serving step: the norm in front of every layer, and the latent-attention
 * layers that alternate with the KDA layers, with their paged cache.
 *
 * A latent-attention layer keeps ONE vector per token for all heads: a
 * normalised latent c of KDA_LATENT_DIM = 512 values and a positional key r of
 * KDA_ROPE_DIM = 64 values (stored as given: rotated by the caller, if the
 * model rotates it).  Head h's key and value are linear in c,
 *     k_h = [ U_h c ; r ]   (128 + 64)        v_h = W_h c   (128)
 * so attention has two forms:
 *   expanded  (kda_latent_prefill)  k_h, v_h are multiplied out first (a plain
 *             GEMM of the caller) and 192-wide scores are taken: the cheaper
 *             form for a prompt, whose keys are each read by many queries.
 *   absorbed  (kda_latent_decode)  U_h is multiplied into the query instead,
 *             q' = [ U_h^T q_nope ; q_rope ] (512 + 64), scores and sums are
 *             taken on the cached vectors themselves, and W_h is applied to
 *             the 512-wide result: the cheaper form for a few new tokens, which
 *             reads 1152 bytes a cached token whatever the number of heads.
 *
 * Conventions are those of kda.h: device pointers, nothing allocated, nothing
 * kept between calls, work enqueued on `stream` without synchronising,
 * arguments validated before anything is enqueued, status codes of kda_status.
 * Attention and the cache are bf16 (fp32 scores, softmax statistics and sums);
 * statistics of the norms are fp32.
 *
 * Paged cache: cache [n_pages, page_size, 576] bf16, page_size a power of two
 * from 16 to 256, n_pages * page_size < 2^31.  Token position p of request n
 * lives in page block_table[n][p / page_size], row p % page_size.  Rows past a
 * request's length may hold anything (NaN included).
 */
#ifndef KDA_HYBRID_H_
#define KDA_HYBRID_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_LATENT_DIM 512
#define KDA_ROPE_DIM 64
#define KDA_LATENT_ROW 576 /* one cached token: latent, then positional key */
#define KDA_NOPE_DIM 128   /* the expanded key's part from the latent, per head */
#define KDA_PAGE_TABLES_MAX_SEQS 16384

/*
 * Block tables and slot maps of one step, from request lengths on the device.
 *
 *   ctx_lens    int32 [N]  tokens of each request already in the cache
 *   new_lens    int32 [N]  tokens it adds in this step
 *   free_pages  int32 [n_free]  page ids not in use, taken from the front
 *   free_start  int32 [1] or NULL (0): where in free_pages this step begins (the
 *               status[0] of the step before, kept apart from this one's status)
 *   block_table int32 [N, max_pages], in and out: entries of the ctx_lens[n]
 *               tokens are kept, the pages that the new tokens need beyond them
 *               are taken from free_pages in request order and appended;
 *               entries past those are left alone
 *   cu_seqlens  int32 [N+1] out: offsets of the requests' new tokens in the
 *               packed batch (negative new_lens count as 0)
 *   seq_lens    int32 [N] out: ctx + new
 *   slots       int32 [max_tokens] out: cache row (page * page_size + offset)
 *               of each packed new token, -1 past the last one
 *   positions   int32 [max_tokens] out: position in its request, -1 likewise
 *   status      int32 [2] out: {position in free_pages after this step, number
 *               of requests refused}
 *
 * A request is refused when a length is negative, when its length would pass
 * 2^31 - 1 or need more than max_pages pages, or when its pages pass the end of
 * free_pages.  A refused request takes no page (one refused by a length or by
 * max_pages moves no other request's pages), its tokens get slot and position -1, and its
 * seq_lens is its ctx_lens (0 if that is negative).  A token whose
 * page id is outside [0, n_pages) gets slot and position -1.
 * N = 0 or max_tokens = 0 is allowed (max_tokens less than the packed batch:
 * only the first max_tokens entries are written).  No output may share memory
 * with an input or with block_table (seq_lens is not ctx_lens: keep two and
 * exchange them).
 */
int kda_page_tables(const int32_t *ctx_lens, const int32_t *new_lens, const int32_t *free_pages,
                    int64_t n_free, const int32_t *free_start, int32_t *block_table,
                    int32_t *cu_seqlens, int32_t *seq_lens, int32_t *slots, int32_t *positions,
                    int32_t *status, int n_seqs, int64_t max_tokens, int max_pages, int page_size,
                    int64_t n_pages, void *stream);

/* kda_rms_norm: the type of y */
#define KDA_QUANT_NONE 0  /* y in dtype, no scales */
#define KDA_QUANT_ROW 1   /* y in e4m3, scales fp32 [rows] */
#define KDA_QUANT_BLOCK 2 /* y in e4m3, scales fp32 [rows, D / 128] */

/*
 * RMS norm with the residual's addition:
 *   h = x + residual        (fp32; h = x without a residual)
 *   y = h / sqrt(mean(h^2) + eps) * weight
 *   residual_out = h rounded to dtype
 * x, residual, residual_out [rows, D] dtype, weight fp32 [D] (NULL = ones).
 * The statistics and y are taken from the unrounded h.  residual and
 * residual_out may each be NULL; residual_out may be residual or x.  With an
 * e4m3 output, y / scale is stored, saturating, with
 *   scale = max(amax |y|, 1e-30) / 448
 * over the row or over each 128 channels (so an all-zero group has a valid
 * scale); a NaN in the group makes its scale NaN.
 * D is a multiple of 8 up to 32768, of 128 for KDA_QUANT_BLOCK.  Rows are
 * 16-byte aligned (y: 8-byte aligned in e4m3).  rows = 0 is a no-op.
 */
int kda_rms_norm(const void *x, const void *residual, const float *weight, void *y,
                 float *scales, void *residual_out, float eps, int64_t rows, int D, int quant,
                 int dtype, void *stream);

/*
 * Append a step's tokens to the latent cache: for token t with slot
 * slots[t] in [0, n_pages * page_size),
 *   cache row slots[t] = [ rms_norm(kv[t, :512]) * weight ; kv[t, 512:576] ]
 *   kv      [T, 576] bf16, rows kv_stride elements apart (a multiple of 8, at
 *           least 576: a slice of a fused projection), 16-byte aligned
 *   weight  fp32 [512], or NULL: the latent is stored as it is (eps unused)
 *   slots   int32 [T], distinct where valid; others (padding: -1) are skipped
 * T = 0 is a no-op.
 */
int kda_latent_cache_write(const void *kv, int64_t kv_stride, const float *weight, float eps,
                           void *cache, const int32_t *slots, int64_t n_tokens, int64_t n_pages,
                           int page_size, void *stream);

/* Device workspace (256-byte aligned) of kda_latent_decode: partial results of
 * requests that several CTAs share.  0 on invalid sizes. */
size_t kda_latent_decode_workspace_bytes(int n_seqs, int S, int H);

/*
 * Absorbed latent attention of S new tokens a request (S = 1: plain decode;
 * S > 1: speculative verify) over the paged cache.
 *
 *   q           [N, S, H, 576] bf16, absorbed queries (16-byte aligned)
 *   cache       [n_pages, page_size, 576] bf16 (16-byte aligned)
 *   block_table int32 [N, max_pages]
 *   seq_lens    int32 [N]: cached tokens of each request, its S new ones among
 *               them
 *   o           [N, S, H, 512] bf16; lse fp32 [N, S, H] or NULL: natural
 *               logarithm of the sum of exp(scale * score)
 *
 * New token s of request n sees positions p < seq_lens[n] - S + 1 + s.  A row
 * that sees nothing (seq_lens[n] <= S - 1 - s) gives o = 0 and lse = -inf.  A
 * request with a negative length, a length beyond max_pages * page_size, or a
 * page id it needs outside [0, n_pages) gives NaN (nothing outside the buffers
 * is read).  The probabilities enter the second product as bf16; their sum is
 * taken in fp32 before that rounding.
 *
 * Limits: S * H <= 4096, N <= 65535, N * max_pages * page_size < 2^36.
 *
 * The cached tokens are split evenly over the GPU's SMs from the lengths on
 * the device, so that one long request fills the GPU as many short ones do.
 * Results do not depend on timing: parts are joined in a fixed order.
 */
int kda_latent_decode(const void *q, const void *cache, const int32_t *block_table,
                      const int32_t *seq_lens, void *o, float *lse, int n_seqs, int S, int H,
                      int64_t n_pages, int page_size, int max_pages, float scale, void *workspace,
                      size_t workspace_bytes, void *stream);

/* Device workspace (256-byte aligned) of kda_latent_prefill: partial results,
 * where there are too few queries to fill the GPU and so many keys that they are
 * split (for queries that see KDA_LATENT_PREFILL_SPLIT_KEYS of them; the split,
 * and with it the rounding, follows from the arguments n_seqs, total_q, total_k, H
 * and the lengths).  Whether keys are split is decided by total_k / n_seqs: one long
 * sequence among many short ones is better given a call of its own.  0: none is needed, as always where total_k is less than
 * KDA_LATENT_PREFILL_SPLIT_KEYS; 0 on invalid sizes. */
#define KDA_LATENT_PREFILL_SPLIT_KEYS 1024
size_t kda_latent_prefill_workspace_bytes(int n_seqs, int64_t total_q, int64_t total_k, int H);

/*
 * Expanded latent attention over packed sequences (prefill).
 *
 *   q       [Tq, H, 192] bf16: per head 128 (no position) then 64 (positional)
 *   kv      [Tk, H, 256] bf16: per head the key's 128 then the value's 128, as
 *           the up-projection writes them
 *   k_rope  [Tk, 64] bf16: the positional key, shared by the heads
 *   o       [Tq, H, 128] bf16; lse fp32 [Tq, H] or NULL
 *   cu_seqlens_q, cu_seqlens_k  int32 [N+1], non-decreasing from 0 to at most
 *           Tq and Tk; cu_seqlens_k NULL = cu_seqlens_q
 *   causal  query i of a sequence with lq queries and lk keys sees keys
 *           j <= i + lk - lq (the last query sees the last key: lk > lq is a
 *           prompt behind a cached prefix); 0 = every key
 *   *_stride  elements between tokens (multiples of 8): q at least 192 H,
 *           kv at least 256 H, k_rope at least 64
 *
 * A query that sees no key gives o = 0 and lse = -inf.  The probabilities enter
 * the second product as bf16; their sum is taken in fp32 before that rounding.
 * Tokens of a sequence whose offsets are decreasing or out of range are not
 * written.  Pointers are 16-byte aligned.  Tq = 0 is a no-op.  Results do not
 * depend on timing: parts are joined in a fixed order.
 *
 * Limits: N <= 65535, H <= 65535, H * ((Tq + 255 min(N, Tq)) / 256) < 2^31 (blocks of
 * 256 queries of a head; beyond them KDA_ERR_UNSUPPORTED).
 */
int kda_latent_prefill(const void *q, int64_t q_stride, const void *kv, int64_t kv_stride,
                       const void *k_rope, int64_t rope_stride, void *o, float *lse,
                       const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int n_seqs,
                       int64_t total_q, int64_t total_k, int H, int causal, float scale,
                       void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_HYBRID_H_ */
