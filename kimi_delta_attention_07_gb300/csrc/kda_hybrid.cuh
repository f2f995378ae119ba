// Launchers and helpers of the operators around the KDA core (kda_hybrid.h).
#pragma once

#include "kda_hybrid.h"
#include "kda_internal.cuh"

namespace kda {

constexpr int kLatent = KDA_LATENT_DIM;
constexpr int kRope = KDA_ROPE_DIM;
constexpr int kLatentRow = KDA_LATENT_ROW;
constexpr int kNope = KDA_NOPE_DIM;
constexpr int kQk = kNope + kRope;      // expanded query / key width
constexpr int kKvRow = kNope + kHeadDim;  // expanded kv row of a head: key part, value

// 8 consecutive elements as fp32 (p 16-byte aligned)
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    const float4 b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 raw = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // a bf16 is the upper half of the fp32 of the same value
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

struct PageTablesArgs {
    const int32_t *ctx_lens, *new_lens, *free_pages, *free_start;
    int32_t *block_table, *cu_seqlens, *seq_lens, *slots, *positions, *status;
    int64_t n_free, max_tokens, n_pages;
    int n_seqs, max_pages, page_shift;
    bool vector_stores;  // slots and positions are 16-byte aligned
};
cudaError_t launch_page_tables(const PageTablesArgs &a, cudaStream_t stream);

struct RmsNormArgs {
    const void *x, *residual;
    const float *weight;
    void *y;
    float *scales;
    void *residual_out;
    float eps;
    int64_t rows;
    int D;
};
cudaError_t launch_rms_norm(const RmsNormArgs &a, int quant, int dtype, cudaStream_t stream);

struct CacheWriteArgs {
    const __nv_bfloat16 *kv;
    int64_t kv_stride;
    const float *weight;
    float eps;
    __nv_bfloat16 *cache;
    const int32_t *slots;
    int64_t n_tokens, n_rows;
};
cudaError_t launch_latent_cache_write(const CacheWriteArgs &a, cudaStream_t stream);

struct LatentDecodeArgs {
    const __nv_bfloat16 *q, *cache;
    const int32_t *block_table, *seq_lens;
    __nv_bfloat16 *o;
    float *lse;
    int n_seqs, S, H;
    int64_t n_pages;
    int page_shift, max_pages;
    float scale;
    void *workspace;
};
size_t latent_decode_workspace_bytes(int n_seqs, int S, int H);
cudaError_t launch_latent_decode(const LatentDecodeArgs &a, cudaStream_t stream);

struct LatentPrefillArgs {
    const __nv_bfloat16 *q, *kv, *k_rope;
    int64_t q_stride, kv_stride, rope_stride;
    __nv_bfloat16 *o;
    float *lse;
    const int32_t *cu_q, *cu_k;
    int n_seqs;
    int64_t total_q, total_k;
    int H, causal;
    float scale;
    void *workspace;
};
// Blocks of queries times heads, at most: the grid without a split.
int64_t latent_prefill_items(int n_seqs, int64_t total_q, int H);
size_t latent_prefill_workspace_bytes(int n_seqs, int64_t total_q, int64_t total_k, int H);
cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, cudaStream_t stream);

}  // namespace kda
