// Launchers of the linear-attention layer with one decay a head (kda_linear.h).
#pragma once

#include "kda_hybrid.cuh"
#include "kda_linear.h"

namespace kda {

// Two fp32 as one operand of the packed instructions.
typedef uint64_t F2;
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unf2(F2 x, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// Two bf16 of a register as fp32.
__device__ __forceinline__ F2 wide(uint32_t two) {
    return f2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
}
__device__ __forceinline__ uint32_t narrow(F2 x) {
    float lo, hi;
    unf2(x, lo, hi);
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// e^g as the sum of two floats.  As one, a decay near one that is applied again and again (token by token,
// chunk by chunk, segment by segment) brings its rounding error back each time: with a fixed decay of 2^-8 a token,
// 1e-5 in the state of a thousand tokens.  (d - 1 is exact from 1/2 to 2; smaller decays leave nothing for
// their error to come back in.)
__device__ __forceinline__ float2 decay_of(float g) {
    const float d = expf(g);
    return make_float2(d, d > 0.5f && d < 2.0f ? expm1f(g) - (d - 1.0f) : 0.0f);
}
// 2^x, likewise (the product's rounding is relative to x, and so is its effect over the decay's memory)
__device__ __forceinline__ float2 decay_of_log2(float x) {
    const float d = exp2f(x);
    return make_float2(d, d > 0.5f && d < 2.0f ? expm1f(x * 0.6931471805599453f) - (d - 1.0f) : 0.0f);
}

struct HeadRopeArgs {
    const void *x[2];  // q, k
    void *y[2];
    int64_t x_stride[2], y_stride[2];
    const float *weight[2];
    int heads[2];
    float eps;
    const int32_t *positions;
    const float *inv_freq;
    int section_end[KDA_ROPE_MAX_AXES];  // pairs below it turn by this axis or one before
    int rot_offset, rot_dim, D;
    int64_t n_tokens;
};
cudaError_t launch_head_norm_rope(const HeadRopeArgs &a, bool norm, bool interleaved, int dtype, cudaStream_t stream);

struct LinearChunkArgs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const float *g;
    int64_t g_stride;
    const float *initial_state;
    float *final_state;
    const int32_t *state_indices;
    int64_t n_slots;
    void *o;
    const int32_t *cu_seqlens;
    int n_seqs;
    int64_t total_tokens;
    int H, group;  // group: heads that share q and k
    float scale;
    void *workspace;
    int equal_len;  // of each sequence, without cu_seqlens
};
size_t linear_chunk_tc_workspace_bytes(int64_t total_tokens, int n_seqs, int H);
size_t linear_chunk_f32_workspace_bytes(int64_t total_tokens, int n_seqs, int H);
// bf16 on the tensor cores; fp32 on the CUDA cores
cudaError_t launch_linear_chunk_tc(const LinearChunkArgs &a, cudaStream_t stream);
cudaError_t launch_linear_chunk_f32(const LinearChunkArgs &a, cudaStream_t stream);

struct LinearStepArgs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const float *g;
    int64_t g_stride;
    float *pool;
    const int32_t *state_indices, *num_accepted;
    int64_t n_slots;
    void *o;
    int N, S, H, group;
    float scale;
};
cudaError_t launch_linear_step(const LinearStepArgs &a, int dtype, cudaStream_t stream);

// Sequence n's tokens [first, first + len); len < 0 where its offsets are decreasing or out of range.
struct Span {
    int first, len;
};
__device__ __forceinline__ Span span_of(const LinearChunkArgs &a, int n) {
    if (!a.cu_seqlens) {
        return {n * a.equal_len, a.equal_len};
    }
    const int from = a.cu_seqlens[n], to = a.cu_seqlens[n + 1];
    const bool ok = from >= 0 && to >= from && to <= a.total_tokens;
    return {from, ok ? to - from : -1};
}
// The slot of sequence n's states, -1 where it lies outside the pool.
__device__ __forceinline__ int64_t slot_of(const LinearChunkArgs &a, int n) {
    if (!a.state_indices) return n;
    const int s = a.state_indices[n];
    return s >= 0 && s < a.n_slots ? s : -1;
}

}  // namespace kda
