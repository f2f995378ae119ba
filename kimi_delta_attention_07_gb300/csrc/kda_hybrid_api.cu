// C ABI of the operators around the KDA core (kda_hybrid.h): argument checks.
#include "kda_hybrid.cuh"

using namespace kda;

namespace {

// log2 of a page size, -1 if it is not a power of two from 16 to 256
inline int page_shift(int page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

inline bool pool_ok(int64_t n_pages, int shift) {
    return shift >= 0 && n_pages > 0 && n_pages < ((int64_t)1 << (31 - shift));
}

}  // namespace

extern "C" {

int kda_page_tables(const int32_t *ctx_lens, const int32_t *new_lens, const int32_t *free_pages,
                    int64_t n_free, const int32_t *free_start, int32_t *block_table,
                    int32_t *cu_seqlens, int32_t *seq_lens, int32_t *slots, int32_t *positions,
                    int32_t *status, int n_seqs, int64_t max_tokens, int max_pages, int page_size,
                    int64_t n_pages, void *stream) {
    const int shift = page_shift(page_size);
    if (n_seqs < 0 || max_tokens < 0 || max_tokens > INT32_MAX || n_free < 0 || n_free > INT32_MAX ||
        max_pages <= 0 || !pool_ok(n_pages, shift))
        return KDA_ERR_INVALID_ARG;
    if (n_seqs > KDA_PAGE_TABLES_MAX_SEQS) return KDA_ERR_UNSUPPORTED;
    if (!cu_seqlens || !status || (n_free > 0 && !free_pages) ||
        (n_seqs > 0 && (!ctx_lens || !new_lens || !block_table || !seq_lens)) ||
        (max_tokens > 0 && (!slots || !positions)))
        return KDA_ERR_INVALID_ARG;
    // every CTA reads the inputs (the table's held entries among them) while others write the outputs
    struct Ints {
        const int32_t *p;
        int64_t n;
        bool meets(const Ints &o) const {
            return p && o.p && n > 0 && o.n > 0 && (uintptr_t)p < (uintptr_t)(o.p + o.n) &&
                   (uintptr_t)o.p < (uintptr_t)(p + n);
        }
    };
    const Ints table = {block_table, (int64_t)n_seqs * max_pages};
    const Ints inputs[] = {{ctx_lens, n_seqs}, {new_lens, n_seqs}, {free_pages, n_free}, {free_start, 1}};
    const Ints outputs[] = {{cu_seqlens, (int64_t)n_seqs + 1}, {seq_lens, n_seqs}, {slots, max_tokens},
                            {positions, max_tokens}, {status, 2}};
    for (const Ints &in : inputs)
        if (in.meets(table)) return KDA_ERR_INVALID_ARG;
    for (const Ints &out : outputs) {
        if (out.meets(table)) return KDA_ERR_INVALID_ARG;
        for (const Ints &in : inputs)
            if (in.meets(out)) return KDA_ERR_INVALID_ARG;
    }
    for (const void *p : {(const void *)ctx_lens, (const void *)new_lens, (const void *)free_pages,
                          (const void *)free_start, (const void *)block_table,
                          (const void *)cu_seqlens, (const void *)seq_lens, (const void *)slots,
                          (const void *)positions, (const void *)status})
        if (!aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const PageTablesArgs a{ctx_lens, new_lens,  free_pages, free_start, block_table, cu_seqlens,
                           seq_lens, slots,     positions,  status,     n_free,      max_tokens,
                           n_pages,  n_seqs,    max_pages,  shift,
                           aligned(slots, 16) && aligned(positions, 16)};
    return launched([&] { return launch_page_tables(a, (cudaStream_t)stream); });
}

int kda_rms_norm(const void *x, const void *residual, const float *weight, void *y,
                 float *scales, void *residual_out, float eps, int64_t rows, int D, int quant,
                 int dtype, void *stream) {
    if ((dtype != KDA_F32 && dtype != KDA_BF16) || quant < KDA_QUANT_NONE ||
        quant > KDA_QUANT_BLOCK || rows < 0 || rows > INT32_MAX || D <= 0 || D % 8 != 0 ||
        (quant == KDA_QUANT_BLOCK && D % 128 != 0) || !isfinite(eps) || eps < 0.0f)
        return KDA_ERR_INVALID_ARG;
    if (D > 32768) return KDA_ERR_UNSUPPORTED;
    if (rows == 0) return KDA_OK;
    if (!x || !y || (quant != KDA_QUANT_NONE && !scales) || !aligned(x, 16) ||
        !aligned(residual, 16) || !aligned(residual_out, 16) || !aligned(weight, 16) ||
        !aligned(y, quant == KDA_QUANT_NONE ? 16 : 8) || !aligned(scales, 4))
        return KDA_ERR_INVALID_ARG;
    const RmsNormArgs a{x, residual, weight, y, scales, residual_out, eps, rows, D};
    return launched([&] { return launch_rms_norm(a, quant, dtype, (cudaStream_t)stream); });
}

int kda_latent_cache_write(const void *kv, int64_t kv_stride, const float *weight, float eps,
                           void *cache, const int32_t *slots, int64_t n_tokens, int64_t n_pages,
                           int page_size, void *stream) {
    const int shift = page_shift(page_size);
    if (n_tokens < 0 || n_tokens > INT32_MAX || kv_stride < kLatentRow || kv_stride % 8 != 0 ||
        !pool_ok(n_pages, shift) || (weight && (!isfinite(eps) || eps < 0.0f)))
        return KDA_ERR_INVALID_ARG;
    if (n_tokens == 0) return KDA_OK;
    if (!kv || !cache || !slots || !aligned(kv, 16) || !aligned(cache, 16) || !aligned(weight, 16) ||
        !aligned(slots, 4))
        return KDA_ERR_INVALID_ARG;
    const CacheWriteArgs a{(const __nv_bfloat16 *)kv, kv_stride, weight,   eps,
                           (__nv_bfloat16 *)cache,    slots,     n_tokens, n_pages << shift};
    return launched([&] { return launch_latent_cache_write(a, (cudaStream_t)stream); });
}

size_t kda_latent_decode_workspace_bytes(int n_seqs, int S, int H) {
    if (n_seqs < 0 || S <= 0 || H <= 0 || (int64_t)S * H > 4096) return 0;
    return latent_decode_workspace_bytes(n_seqs, S, H);
}

int kda_latent_decode(const void *q, const void *cache, const int32_t *block_table,
                      const int32_t *seq_lens, void *o, float *lse, int n_seqs, int S, int H,
                      int64_t n_pages, int page_size, int max_pages, float scale, void *workspace,
                      size_t workspace_bytes, void *stream) {
    const int shift = page_shift(page_size);
    if (n_seqs < 0 || S <= 0 || H <= 0 || max_pages <= 0 || !pool_ok(n_pages, shift) ||
        !isfinite(scale))
        return KDA_ERR_INVALID_ARG;
    // tiles are counted in 32 bits
    if ((int64_t)S * H > 4096 || n_seqs > 65535 ||
        (((int64_t)max_pages << shift) * n_seqs) >> 36 != 0)
        return KDA_ERR_UNSUPPORTED;
    if (n_seqs == 0) return KDA_OK;
    if (!q || !cache || !block_table || !seq_lens || !o || !aligned(q, 16) || !aligned(cache, 16) ||
        !aligned(o, 16) || !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
        return KDA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < latent_decode_workspace_bytes(n_seqs, S, H))
        return KDA_ERR_WORKSPACE;
    const LatentDecodeArgs a{(const __nv_bfloat16 *)q, (const __nv_bfloat16 *)cache, block_table,
                             seq_lens, (__nv_bfloat16 *)o, lse, n_seqs, S, H, n_pages, shift,
                             max_pages, scale, workspace};
    return launched([&] { return launch_latent_decode(a, (cudaStream_t)stream); });
}

size_t kda_latent_prefill_workspace_bytes(int n_seqs, int64_t total_q, int64_t total_k, int H) {
    if (n_seqs <= 0 || H <= 0 || H > 65535 || n_seqs > 65535 || total_q < 0 || total_q > INT32_MAX || total_k < 0 ||
        total_k > INT32_MAX)
        return 0;
    return latent_prefill_workspace_bytes(n_seqs, total_q, total_k, H);
}

int kda_latent_prefill(const void *q, int64_t q_stride, const void *kv, int64_t kv_stride,
                       const void *k_rope, int64_t rope_stride, void *o, float *lse,
                       const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int n_seqs,
                       int64_t total_q, int64_t total_k, int H, int causal, float scale, void *workspace,
                       size_t workspace_bytes, void *stream) {
    if (n_seqs <= 0 || H <= 0 || total_q < 0 || total_q > INT32_MAX || total_k < 0 ||
        total_k > INT32_MAX || !isfinite(scale) || q_stride < (int64_t)kQk * H || q_stride % 8 != 0 ||
        kv_stride < (int64_t)kKvRow * H || kv_stride % 8 != 0 || rope_stride < kRope ||
        rope_stride % 8 != 0)
        return KDA_ERR_INVALID_ARG;
    if (H > 65535 || n_seqs > 65535 || latent_prefill_items(n_seqs, total_q, H) > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (total_q == 0) return KDA_OK;
    if (!q || !o || !cu_seqlens_q || (total_k > 0 && (!kv || !k_rope)) || !aligned(q, 16) ||
        !aligned(kv, 16) || !aligned(k_rope, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
        !aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4))
        return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens_k && total_k != total_q) return KDA_ERR_INVALID_ARG;
    const size_t need = latent_prefill_workspace_bytes(n_seqs, total_q, total_k, H);
    if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    const LatentPrefillArgs a{(const __nv_bfloat16 *)q, (const __nv_bfloat16 *)kv,
                              (const __nv_bfloat16 *)k_rope, q_stride, kv_stride, rope_stride,
                              (__nv_bfloat16 *)o, lse, cu_seqlens_q,
                              cu_seqlens_k ? cu_seqlens_k : cu_seqlens_q, n_seqs, total_q, total_k,
                              H, causal != 0, scale, workspace};
    return launched([&] { return launch_latent_prefill(a, (cudaStream_t)stream); });
}

}  // extern "C"
