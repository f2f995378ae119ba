// C ABI of the linear-attention layer with one decay a head (kda_linear.h): argument checks.
#include "kda_linear.cuh"

using namespace kda;

namespace {

inline bool dtype_ok(int dtype) { return dtype == KDA_F32 || dtype == KDA_BF16; }

// A token stride for `heads` heads of `width`: a slice of a wider row, 16-byte aligned.
inline bool stride_ok(int64_t stride, int64_t heads, int width) {
    return stride >= heads * width && stride % 8 == 0 && stride < ((int64_t)1 << 31);
}

// What the chunked form and the steps have in common, but for the pointers.
int check_layer(int64_t tokens, int H, int Hk, int K, int V, float scale, int dtype, int64_t q_stride,
                int64_t k_stride, int64_t v_stride, int64_t g_stride, int64_t n_slots) {
    if (H <= 0 || Hk <= 0 || H % Hk != 0 || K <= 0 || V <= 0 || tokens < 0 || tokens > INT32_MAX || n_slots < 0 ||
        !dtype_ok(dtype) || !isfinite(scale))
        return KDA_ERR_INVALID_ARG;
    if (K != kHeadDim || V != kHeadDim || H > 65535) return KDA_ERR_UNSUPPORTED;
    if (!stride_ok(q_stride, Hk, K) || !stride_ok(k_stride, Hk, K) || !stride_ok(v_stride, H, V) ||
        (g_stride != 0 && g_stride < H) || g_stride >= ((int64_t)1 << 31))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

int linear_step(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                const float *g, int64_t g_stride, float *state_pool, const int32_t *state_indices,
                const int32_t *num_accepted, int64_t n_slots, void *o, int N, int S, int H, int Hk, int K, int V,
                float scale, int dtype, void *stream) {
    if (N < 0 || S <= 0) return KDA_ERR_INVALID_ARG;
    const int st = check_layer((int64_t)N * S, H, Hk, K, V, scale, dtype, q_stride, k_stride, v_stride, g_stride, n_slots);
    if (st != KDA_OK) return st;
    if ((int64_t)N * H > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (N == 0) return KDA_OK;
    if (!q || !k || !v || !g || !state_pool || !o || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(o, 16) || !aligned(state_pool, 16) || !aligned(g, 4) || !aligned(state_indices, 4) ||
        !aligned(num_accepted, 4) || (!state_indices && n_slots < N))
        return KDA_ERR_INVALID_ARG;
    const LinearStepArgs a{q, k, v, q_stride, k_stride, v_stride, g, g_stride, state_pool, state_indices, num_accepted,
                           n_slots, o, N, S, H, H / Hk, scale};
    return launched([&] { return launch_linear_step(a, dtype, (cudaStream_t)stream); });
}

}  // namespace

extern "C" {

int kda_head_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                       const float *q_weight, const float *k_weight, float eps, int norm,
                       const int32_t *positions, const int *sections, int n_axes,
                       const float *inv_freq, int rot_offset, int rot_dim, int interleaved,
                       void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride,
                       int64_t n_tokens, int Hq, int Hk, int D, int dtype, void *stream) {
    if (!dtype_ok(dtype) || n_tokens < 0 || n_tokens > INT32_MAX || Hq <= 0 || Hk < 0 || D <= 0 || D % 16 != 0 ||
        rot_dim < 0 || rot_dim % 16 != 0 || rot_offset < 0 || rot_offset % 8 != 0 || rot_dim > D ||
        rot_offset > D - rot_dim || (norm && (!isfinite(eps) || eps < 0.0f)) || n_axes < 1 ||
        n_axes > KDA_ROPE_MAX_AXES || (n_axes > 1 && !sections))
        return KDA_ERR_INVALID_ARG;
    if (D > 256 || Hq > 65535 || Hk > 65535 || n_tokens * (Hq + Hk) > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (!stride_ok(q_stride, Hq, D) || !stride_ok(q_out_stride, Hq, D) ||
        (Hk > 0 && (!stride_ok(k_stride, Hk, D) || !stride_ok(k_out_stride, Hk, D))))
        return KDA_ERR_INVALID_ARG;
    HeadRopeArgs a{{q, k}, {q_out, k_out}, {q_stride, k_stride}, {q_out_stride, k_out_stride}, {q_weight, k_weight},
                   {Hq, Hk}, eps, positions, inv_freq, {}, rot_offset, rot_dim, D, n_tokens};
    int64_t pairs = 0;
    for (int i = 0; i < KDA_ROPE_MAX_AXES; ++i) {
        const int own = i >= n_axes ? 0 : sections ? sections[i] : rot_dim / 2;
        if (own < 0) return KDA_ERR_INVALID_ARG;
        pairs += own;
        a.section_end[i] = (int)(pairs < INT32_MAX ? pairs : INT32_MAX);
    }
    if (pairs != rot_dim / 2) return KDA_ERR_INVALID_ARG;
    if (n_tokens == 0) return KDA_OK;
    if (!q || !q_out || (rot_dim > 0 && (!positions || !inv_freq)) || !aligned(q, 16) || !aligned(q_out, 16) || (q == q_out && q_stride != q_out_stride) ||
        (Hk > 0 && (!k || !k_out || !aligned(k, 16) || !aligned(k_out, 16) || (k == k_out && k_stride != k_out_stride))) ||
        !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(positions, 4) || !aligned(inv_freq, 4))
        return KDA_ERR_INVALID_ARG;
    return launched([&] { return launch_head_norm_rope(a, norm != 0, interleaved != 0, dtype, (cudaStream_t)stream); });
}

size_t kda_linear_chunk_workspace_bytes(int64_t total_tokens, int n_seqs, int H, int dtype) {
    if (total_tokens < 0 || total_tokens > INT32_MAX || n_seqs <= 0 || n_seqs > 65535 || H <= 0 || H > 65535 ||
        !dtype_ok(dtype))
        return 0;
    return dtype == KDA_BF16 ? linear_chunk_tc_workspace_bytes(total_tokens, n_seqs, H)
                             : linear_chunk_f32_workspace_bytes(total_tokens, n_seqs, H);
}

int kda_linear_chunk_fwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                         const void *v, int64_t v_stride, const float *g, int64_t g_stride,
                         const float *initial_state, float *final_state,
                         const int32_t *state_indices, int64_t n_slots, void *o,
                         const int32_t *cu_seqlens, int n_seqs, int64_t total_tokens, int H,
                         int Hk, int K, int V, float scale, int dtype, void *workspace,
                         size_t workspace_bytes, void *stream) {
    if (n_seqs <= 0) return KDA_ERR_INVALID_ARG;
    const int st = check_layer(total_tokens, H, Hk, K, V, scale, dtype, q_stride, k_stride, v_stride, g_stride, n_slots);
    if (st != KDA_OK) return st;
    if (n_seqs > 65535 || total_tokens / 128 * H >= (1 << 30) || (int64_t)n_seqs * H >= (1 << 30))
        return KDA_ERR_UNSUPPORTED;
    if ((total_tokens > 0 && (!q || !k || !v || !g || !o)) || (!cu_seqlens && total_tokens % n_seqs != 0) ||
        !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(g, 4) ||
        !aligned(initial_state, 16) || !aligned(final_state, 16) || !aligned(state_indices, 4) || !aligned(cu_seqlens, 4))
        return KDA_ERR_INVALID_ARG;
    const size_t need = kda_linear_chunk_workspace_bytes(total_tokens, n_seqs, H, dtype);
    if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    const LinearChunkArgs a{q, k, v, q_stride, k_stride, v_stride, g, g_stride, initial_state, final_state,
                            state_indices, n_slots, o, cu_seqlens, n_seqs, total_tokens, H, H / Hk, scale, workspace,
                            (int)(total_tokens / n_seqs)};
    return launched([&] {
        return dtype == KDA_BF16 ? launch_linear_chunk_tc(a, (cudaStream_t)stream) : launch_linear_chunk_f32(a, (cudaStream_t)stream);
    });
}

int kda_linear_step(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                    const void *v, int64_t v_stride, const float *g, int64_t g_stride,
                    float *state_pool, const int32_t *state_indices, int64_t n_slots, void *o,
                    int N, int H, int Hk, int K, int V, float scale, int dtype, void *stream) {
    return linear_step(q, q_stride, k, k_stride, v, v_stride, g, g_stride, state_pool, state_indices, nullptr, n_slots, o,
                       N, 1, H, Hk, K, V, scale, dtype, stream);
}

int kda_linear_multi_step(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                          const void *v, int64_t v_stride, const float *g, int64_t g_stride,
                          float *state_pool, const int32_t *state_indices,
                          const int32_t *num_accepted, int64_t n_slots, void *o, int N, int S,
                          int H, int Hk, int K, int V, float scale, int dtype, void *stream) {
    if (N > 0 && !state_indices) return KDA_ERR_INVALID_ARG;
    return linear_step(q, q_stride, k, k_stride, v, v_stride, g, g_stride, state_pool, state_indices, num_accepted,
                       n_slots, o, N, S, H, Hk, K, V, scale, dtype, stream);
}

}  // extern "C"
