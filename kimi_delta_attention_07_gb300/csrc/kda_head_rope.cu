// RMS norm of each head of q and k, and rotation of channel pairs by the token's
// position, in one pass over both:
//   y = x / sqrt(mean(x^2) + eps) * weight,  (a, b) -> (a cos t - b sin t, b cos t + a sin t)
//
// HBM bound: each element is read and written once.  Four to sixteen lanes take a
// head, two vectors of eight channels a lane, chosen so that a lane holds both
// members of its pairs; the sum of squares is the lanes' only exchange.  A CTA takes some
// tokens (and, where there are few, a part of their heads), computes their angles once for all
// heads while the first rows are on their way, and requests each thread's next row
// before it works on the last one.  What then bounds it is instructions, some 200 a warp and rows of two
// vectors a lane: fp32 in pairs, indices without a division, weights and angles in shared
// memory in the order of the lanes (4096 tokens of 64 heads: 25.4 us, 5.3 TB/s; one token a CTA and
// scalar arithmetic, 38 us; a thread that keeps to a head, with its weights in registers, 27; two
// rows ahead with 24 warps a SM, 30).
//
// Angles: t / 2 pi = p f / 2 pi, taken modulo 1 before it is rounded.  f / 2 pi is held as
// the sum c + d of two floats, p as the sum of two parts of 16 bits; p c is split by an fma
// into its rounding and the rest, whose integer part costs nothing.
#include <algorithm>

#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 64;        // of a CTA
constexpr int kTableBytes = 32768;    // of a CTA's angles, at most (a single token's may be as many as 2 KB)
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
__device__ __forceinline__ void unpack(const Vec<__nv_bfloat16> &r, F2 (&x)[4]) {
    x[0] = wide(r.v[0].x), x[1] = wide(r.v[0].y), x[2] = wide(r.v[0].z), x[3] = wide(r.v[0].w);
}
__device__ __forceinline__ void unpack(const Vec<float> &r, F2 (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x[2 * i] = f2(__uint_as_float(r.v[i].x), __uint_as_float(r.v[i].y));
        x[2 * i + 1] = f2(__uint_as_float(r.v[i].z), __uint_as_float(r.v[i].w));
    }
}
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const F2 (&x)[4]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(narrow(x[0]), narrow(x[1]), narrow(x[2]), narrow(x[3]));
}
__device__ __forceinline__ void store_vec(float *p, const F2 (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float4 y;
        unf2(x[2 * i], y.x, y.y);
        unf2(x[2 * i + 1], y.z, y.w);
        reinterpret_cast<float4 *>(p)[i] = y;
    }
}

struct HeadRopeParams {
    HeadRopeArgs a;
    int tokens;  // of a CTA
    int heads;   // of a CTA, of q's and k's together
};

// LANES: lanes of a head.
template <typename T, int LANES, bool NORM, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 4) head_norm_rope_kernel(const HeadRopeParams p) {
    // Angles, [token][four][lane], entry i of lane l: half layout, (cos, cos, sin, sin) of pairs 8 l + 2 i and the one
    // after; interleaved [token][eight][lane], (cos, cos, -sin, sin) of pair 8 l + i.
    // Behind them the weights, [q, k][four][lane]: four channels each.
    extern __shared__ __align__(16) float4 table[];
    __shared__ bool padding[kMaxTokens];
    constexpr int kGroups = kThreads / LANES, kEntries = INTERLEAVED ? 8 : 4;
    const HeadRopeArgs &a = p.a;
    const int turning = a.rot_dim / 16, off = a.rot_offset / 8;
    const int t0 = blockIdx.x * p.tokens, tokens = min(p.tokens, (int)a.n_tokens - t0);
    const int all = a.heads[0] + a.heads[1], h0 = blockIdx.y * p.heads, heads = min(p.heads, all - h0);
    const int group = threadIdx.x / LANES, l = threadIdx.x % LANES;
    float4 *weights = table + p.tokens * turning * kEntries;
    griddep_wait();
    griddep_launch_dependents();

    // the two vectors of this lane: of pairs, or of channels that do not turn
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
    // this thread's next (token, head)
    const int step_tokens = (unsigned)kGroups / (unsigned)heads, step_heads = kGroups - step_tokens * heads;
    int token = (unsigned)group / (unsigned)heads, head = group - token * heads;
    Vec<T> raw[2];
    auto request = [&] {
        if (token >= tokens || !active) return;
        const int h = h0 + head, which = h >= a.heads[0];
        const T *x = (const T *)a.x[which] + (t0 + token) * a.x_stride[which] + (which ? h - a.heads[0] : h) * a.D;
        raw[0] = load_vec(x + 8 * at[0]);
        raw[1] = load_vec(x + 8 * at[1]);
    };
    request();
    for (int i = threadIdx.x; i < tokens * turning * 8; i += kThreads) {
        const int t = i / (8 * turning), pair = i - t * (8 * turning);
        int axis = 0;
#pragma unroll
        for (int j = 0; j < KDA_ROPE_MAX_AXES - 1; ++j) axis += pair >= a.section_end[j];
        const int pos = a.positions[axis * a.n_tokens + t0 + t];
        const float f = a.inv_freq[pair], c = f * kTurnHi, d = fmaf(f, kTurnLo, fmaf(f, kTurnHi, -c));
        float r = turns((float)(pos & ~0xffff), c, d) + turns((float)(pos & 0xffff), c, d);
        r -= rintf(r);
        float sn, cs;
        sincospif(2.0f * r, &sn, &cs);
        const int lane = pair >> 3, j = pair & 7;
        if (INTERLEAVED) {
            table[(t * kEntries + j) * turning + lane] = make_float4(cs, cs, -sn, sn);
        } else {
            float *e = (float *)&table[(t * kEntries + (j >> 1)) * turning + lane] + (j & 1);
            e[0] = cs, e[2] = sn;
        }
    }
    for (int t = threadIdx.x; t < tokens; t += kThreads) padding[t] = a.positions && a.positions[t0 + t] < 0;
    if (NORM && threadIdx.x < 2 * LANES && active) {  // this lane's channels, of q's weight or k's
        const float *w = a.weight[threadIdx.x / LANES];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            weights[(threadIdx.x / LANES * 4 + j) * LANES + l] =
                w ? *(const float4 *)(w + 8 * at[j >> 1] + 4 * (j & 1)) : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    }
    __syncthreads();
    const float mean = 1.0f / a.D;
    const int steps = (tokens * heads + kGroups - 1) / kGroups;  // (the same for all: lanes exchange)
    for (int n = 0; n < steps; ++n) {
        const int t = token, h = h0 + head, which = h >= a.heads[0];
        const bool here = token < tokens && active;
        F2 x[2][4];
        if (here) {
            unpack(raw[0], x[0]);
            unpack(raw[1], x[1]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[0][j] = x[1][j] = 0;
        }
        token += step_tokens, head += step_heads;
        if (head >= heads) head -= heads, ++token;
        request();
        if (NORM) {
            F2 sum = mul2(x[0][0], x[0][0]);
#pragma unroll
            for (int j = 1; j < 8; ++j) sum = fma2(x[j >> 2][j & 3], x[j >> 2][j & 3], sum);
            float lo, hi;
            unf2(sum, lo, hi);
            lo += hi;
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) lo += __shfl_xor_sync(0xffffffffu, lo, o);
            const float rn = rsqrtf(fmaf(lo, mean, a.eps));
            const float4 *w = weights + which * 4 * LANES + l;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 v = w[j * LANES];
                F2 &y = x[j >> 1][2 * (j & 1)], &z = x[j >> 1][2 * (j & 1) + 1];
                y = mul2(y, mul2(f2(v.x, v.y), f2(rn, rn)));
                z = mul2(z, mul2(f2(v.z, v.w), f2(rn, rn)));
            }
        }
        if (!here || padding[t]) continue;
        if (turns_here) {
            const float4 *e = table + t * kEntries * turning + l;
            if (INTERLEAVED) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    F2 &y = x[j >> 2][j & 3];
                    const float4 r = e[j * turning];
                    float u, v;
                    unf2(y, u, v);
                    y = fma2(y, f2(r.x, r.y), mul2(f2(v, u), f2(r.z, r.w)));
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 r = e[j * turning];
                    const F2 c = f2(r.x, r.y), s = f2(r.z, r.w), y = x[0][j], z = x[1][j];
                    x[0][j] = fma2(y, c, mul2(z, f2(-r.z, -r.w)));
                    x[1][j] = fma2(z, c, mul2(y, s));
                }
            }
        }
        T *y = (T *)a.y[which] + (t0 + t) * a.y_stride[which] + (which ? h - a.heads[0] : h) * a.D;
        store_vec(y + 8 * at[0], x[0]);
        store_vec(y + 8 * at[1], x[1]);
    }
}

template <typename T, int LANES>
cudaError_t launch(const HeadRopeArgs &a, bool norm, bool interleaved, cudaStream_t stream) {
    constexpr int kGroups = kThreads / LANES;
    const int64_t heads = a.heads[0] + a.heads[1], T_ = a.n_tokens;
    // A CTA's rows are eight times its groups (4096 tokens of 64 heads: 24.1 us of the device; four times 24.6, sixteen 27.6),
    // fewer where that leaves SMs idle: four CTAs a SM (4096 of 9 heads of 256: 9.4 us; two 12.3), but a row for each group
    // while every SM has a CTA (777 of 32 heads of 64: 3.3 us; 4.3 without), and at last heads apart
    // (8 tokens of 40 heads: 2.2 us; 2.6 without).
    const int64_t token_bytes = std::max(1, a.rot_dim / 2 * (interleaved ? 16 : 8));
    int64_t tokens = std::min<int64_t>({std::max<int64_t>(1, 8 * kGroups / heads), kMaxTokens, std::max<int64_t>(1, kTableBytes / token_bytes),
                                        std::max<int64_t>({1, T_ / (4 * sm_count()), std::min<int64_t>(kGroups / heads, T_ / sm_count())})});
    int64_t split = 1;
    while (heads / split > kGroups && (T_ + tokens - 1) / tokens * split < 2 * sm_count()) split *= 2;
    HeadRopeParams p{a, (int)tokens, (int)((heads + split - 1) / split)};
    const size_t smem = (size_t)(tokens * (a.rot_dim ? token_bytes : 0)) + (norm ? 2 * 4 * LANES * sizeof(float4) : 0);
    auto kern = norm ? interleaved ? head_norm_rope_kernel<T, LANES, true, true> : head_norm_rope_kernel<T, LANES, true, false>
                     : interleaved ? head_norm_rope_kernel<T, LANES, false, true> : head_norm_rope_kernel<T, LANES, false, false>;
    const cudaError_t e = launch_dependent(kern, dim3((unsigned)((T_ + tokens - 1) / tokens), (unsigned)((heads + p.heads - 1) / p.heads)),
                                           dim3(kThreads), smem, stream, p);
    return e != cudaSuccess ? e : cudaGetLastError();
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
