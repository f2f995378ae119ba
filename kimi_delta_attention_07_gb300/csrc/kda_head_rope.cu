// RMS norm of each head of q and k, and rotation of channel pairs by the token's
// position, in one pass over both:
//   y = x / sqrt(mean(x^2) + eps) * weight,  (a, b) -> (a cos t - b sin t, b cos t + a sin t)
//
// HBM bound: each element is read and written once.  Four to sixteen lanes take a
// head, two vectors of eight channels a lane, chosen so that a lane holds both
// members of its pairs; the sum of squares is the lanes' only exchange.  A CTA takes a
// run of (token, head) pairs in the order of memory and computes the angles of its tokens
// once for all their heads, while the first rows are on their way.
//
// Angles: t / 2 pi = p f / 2 pi, taken modulo 1 before it is rounded.  f / 2 pi is held as
// the sum c + d of two floats, p as the sum of two parts of 16 bits; p c is split by an fma
// into its rounding and the rest, whose integer part costs nothing.
#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 32;  // of a CTA: rows of the table of angles
constexpr float kTurnHi = 0.15915494f;  // 1 / 2 pi
constexpr float kTurnLo = (float)(0.15915494309189533577 - (double)kTurnHi);

// x * (c + d) modulo 1, for an integer x that a float holds
__device__ __forceinline__ float turns(float x, float c, float d) {
    const float a = x * c;
    return (a - rintf(a)) + fmaf(x, d, fmaf(x, c, -a));
}

template <typename T>
struct Vec {  // eight channels as they lie in memory
    uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T *p) {
    Vec<T> r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.v[i] = reinterpret_cast<const uint4 *>(p)[i];
    return r;
}

// LANES: lanes of a head.  PASSES: heads that a thread group takes, all requested at once.
template <typename T, int LANES, int PASSES, bool NORM, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) head_norm_rope_kernel(const HeadRopeArgs a, int per_cta) {
    extern __shared__ float2 table[];  // [tokens of this CTA][rot_dim / 2]: cos, sin
    __shared__ bool padding[kMaxTokens];
    constexpr int kGroups = kThreads / LANES;
    griddep_wait();
    griddep_launch_dependents();
    const int heads = a.heads[0] + a.heads[1], half = a.rot_dim / 2;
    const int64_t begin = (int64_t)blockIdx.x * per_cta, total = a.n_tokens * heads;
    const int64_t end = begin + per_cta < total ? begin + per_cta : total;
    const int t0 = (int)(begin / heads), tokens = (int)((end - 1) / heads) - t0 + 1;
    const int group = threadIdx.x / LANES, l = threadIdx.x % LANES;

    // the two vectors of this lane: of pairs, or of channels that do not turn
    const int turning = a.rot_dim / 16, off = a.rot_offset / 8;
    const bool active = l < a.D / 16, turns_here = l < turning;
    int at[2];
    if (turns_here) {
        at[0] = off + (INTERLEAVED ? 2 * l : l);
        at[1] = INTERLEAVED ? at[0] + 1 : at[0] + turning;
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int u = 2 * (l - turning) + i;
            at[i] = u < off ? u : u + a.rot_dim / 8;
        }
    }
    Vec<T> raw[PASSES][2];
    int token[PASSES], head[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int64_t item = begin + group + p * kGroups;
        token[p] = item < end && active ? (int)(item / heads) : -1;
        if (token[p] < 0) continue;
        head[p] = (int)(item - (int64_t)token[p] * heads);
        const int which = head[p] >= a.heads[0];
        if (which) head[p] -= a.heads[0];
        const T *x = (const T *)a.x[which] + token[p] * a.x_stride[which] + (int64_t)head[p] * a.D;
        if (which) head[p] = ~head[p];
        raw[p][0] = load_vec(x + 8 * at[0]);
        raw[p][1] = load_vec(x + 8 * at[1]);
    }
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int t = i / half, pair = i - t * half;
        int axis = 0;
#pragma unroll
        for (int j = 0; j < KDA_ROPE_MAX_AXES - 1; ++j) axis += pair >= a.section_end[j];
        const int pos = a.positions[axis * a.n_tokens + t0 + t];
        const float f = a.inv_freq[pair], c = f * kTurnHi, d = fmaf(f, kTurnLo, fmaf(f, kTurnHi, -c));
        float r = turns((float)(pos & ~0xffff), c, d) + turns((float)(pos & 0xffff), c, d);
        r -= rintf(r);
        float sn, cs;
        sincospif(2.0f * r, &sn, &cs);
        table[i] = make_float2(cs, sn);
    }
    for (int t = threadIdx.x; t < tokens; t += kThreads) padding[t] = a.positions && a.positions[t0 + t] < 0;
    __syncthreads();
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int which = token[p] >= 0 && head[p] < 0;
        float x[2][8];
        if (token[p] >= 0) {
            load8((const T *)raw[p][0].v, x[0]);
            load8((const T *)raw[p][1].v, x[1]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[0][j] = x[1][j] = 0.0f;
        }
        if (NORM) {
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += x[0][j] * x[0][j] + x[1][j] * x[1][j];
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float rn = 1.0f / sqrtf(sum / a.D + a.eps);
            const float *weight = a.weight[which];
            if (weight && active) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float w[8];
                    load8(weight + 8 * at[i], w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[i][j] *= rn * w[j];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[i][j] *= rn;
            }
        }
        if (token[p] < 0 || padding[token[p] - t0]) continue;
        if (turns_here) {
            const float2 *cs = table + (token[p] - t0) * half + 8 * l;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float &u = INTERLEAVED ? x[j >> 2][2 * (j & 3)] : x[0][j];
                float &w = INTERLEAVED ? x[j >> 2][2 * (j & 3) + 1] : x[1][j];
                const float2 t = cs[j];
                const float b = w * t.x + u * t.y;
                u = u * t.x - w * t.y;
                w = b;
            }
        }
        T *y = (T *)a.y[which] + token[p] * a.y_stride[which] + (int64_t)(which ? ~head[p] : head[p]) * a.D;
        store8(y + 8 * at[0], x[0]);
        store8(y + 8 * at[1], x[1]);
    }
}

template <typename T, int LANES, int PASSES>
cudaError_t launch(const HeadRopeArgs &a, bool norm, bool interleaved, cudaStream_t stream) {
    const int64_t heads = a.heads[0] + a.heads[1], total = a.n_tokens * heads;
    // a run of pairs touches at most two tokens more than it holds whole ones
    const int64_t most = heads * (kMaxTokens - 2), want = (kThreads / LANES) * PASSES;
    const int per_cta = (int)(want < most ? want : most);
    const int64_t tokens = per_cta / heads + 2 < a.n_tokens ? per_cta / heads + 2 : a.n_tokens;
    const size_t smem = (size_t)tokens * (a.rot_dim / 2) * sizeof(float2);
    auto kern = norm ? interleaved ? head_norm_rope_kernel<T, LANES, PASSES, true, true>
                                   : head_norm_rope_kernel<T, LANES, PASSES, true, false>
                     : interleaved ? head_norm_rope_kernel<T, LANES, PASSES, false, true>
                                   : head_norm_rope_kernel<T, LANES, PASSES, false, false>;
    const cudaError_t e = launch_dependent(kern, dim3((unsigned)((total + per_cta - 1) / per_cta)), dim3(kThreads), smem,
                                           stream, a, per_cta);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int LANES>
cudaError_t launch(const HeadRopeArgs &a, bool norm, bool interleaved, cudaStream_t stream) {
    return launch<T, LANES, 2>(a, norm, interleaved, stream);
}

template <typename T>
cudaError_t launch(const HeadRopeArgs &a, bool norm, bool interleaved, cudaStream_t stream) {
    return a.D <= 64    ? launch<T, 4>(a, norm, interleaved, stream)
           : a.D <= 128 ? launch<T, 8>(a, norm, interleaved, stream)
                        : launch<T, 16>(a, norm, interleaved, stream);
}

}  // namespace

cudaError_t launch_head_norm_rope(const HeadRopeArgs &a, bool norm, bool interleaved, int dtype, cudaStream_t stream) {
    return dtype == KDA_BF16 ? launch<__nv_bfloat16>(a, norm, interleaved, stream)
                             : launch<float>(a, norm, interleaved, stream);
}

}  // namespace kda
