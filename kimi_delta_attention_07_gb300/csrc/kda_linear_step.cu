// One or a few tokens of linear attention with one decay a head, on a pooled fp32 state:
//   S <- e^g S + k v^T,  o = scale S^T q = scale (e^g S_old^T q + v (k . q))
//
// HBM bound: a head's 64 KB state is read once and written once a token.  The pool keeps
// S^T ([V][K]): a warp owns whole rows, a lane four key channels of each; all rows of a warp
// are requested before the first is used.  The rows' dot products with q are summed over
// the lanes together, by a reduce-scatter: RPW rows cost RPW shuffles where a
// reduction of each would take five times as many.  Rows of a head are split over CTAs
// where there are few heads.  With several tokens the rows stay in registers between them.
//
// The decay is the sum of two floats (decay_of): a state lives through thousands of steps (error behind 1024 of
// them at 2^-8 a token 3e-7; with one float 1.3e-5, and 64 x 4 tokens 106.8 us of the device instead of 109.3).
//
// 256 sequences of 32 heads: 156 us, 6.9 TB/s of states read and written; 64 sequences of 32 heads, 4 tokens each: 109 us,
// 6.1 TB/s; 4 sequences of 8 heads: 1.9 us of the device.
#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The sums over the lanes of RPW values a lane: lane l gets that of value l % RPW.
template <int RPW>
__device__ __forceinline__ float scatter_sums(float (&p)[RPW], int lane) {
#pragma unroll
    for (int m = RPW / 2; m > 0; m >>= 1) {
        const bool hi = (lane & m) != 0;
#pragma unroll
        for (int i = 0; i < m; ++i) {
            const float send = hi ? p[i] : p[i + m];
            p[i] = (hi ? p[i + m] : p[i]) + __shfl_xor_sync(0xffffffffu, send, m);
        }
    }
    float x = p[0];
#pragma unroll
    for (int o = RPW; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// RPW: rows of a warp; a CTA takes 8 RPW rows of one head, row j of a warp being warp + 8 j.
template <typename T, int RPW, bool MULTI>
__global__ void __launch_bounds__(kThreads, 2) linear_step_kernel(const LinearStepArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int n = blockIdx.x / a.H, h = blockIdx.x - n * a.H;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row0 = blockIdx.y * (kWarps * RPW) + warp;
    const int S = MULTI ? a.S : 1;
    const int hk = h / a.group;
    const int64_t token0 = (int64_t)n * S;
    T *o = (T *)a.o + (token0 * a.H + h) * kHeadDim + row0;
    auto slot_after = [&](int t) { return a.state_indices ? (int64_t)a.state_indices[token0 + t] : (int64_t)n; };

    int64_t slot = 0;
    bool valid = true;
    if (MULTI) {
        // every slot of the sequence and its count are looked at before anything is written
        const int accepted = a.num_accepted ? a.num_accepted[n] : 1;
        valid = accepted >= 1 && accepted <= S;
        for (int t = 0; t < S && valid; ++t) {
            const int64_t s = slot_after(t);
            valid = s >= 0 && s < a.n_slots;
        }
        if (valid) slot = slot_after(accepted - 1);
    } else {
        slot = slot_after(0);
        valid = slot >= 0 && slot < a.n_slots;
    }
    if (!valid) {
        if (lane < RPW)
            for (int t = 0; t < S; ++t) o[(int64_t)t * a.H * kHeadDim + kWarps * lane] = from_f32<T>(__int_as_float(0x7fc00000));
        return;
    }
    const int64_t row_at = (int64_t)row0 * kHeadDim + 4 * lane;
    const float *src = a.pool + (slot * a.H + h) * (int64_t)(kHeadDim * kHeadDim) + row_at;
    struct Token {
        float4 q, k;
        float v, g;  // v: of row `lane` of the warp
    };
    auto fetch = [&](int t) {
        const int64_t at = token0 + t;
        Token x;
        x.q = load4((const T *)a.q + at * a.q_stride + hk * kHeadDim + 4 * lane);
        x.k = load4((const T *)a.k + at * a.k_stride + hk * kHeadDim + 4 * lane);
        x.v = to_f32(((const T *)a.v)[at * a.v_stride + (int64_t)h * kHeadDim + row0 + kWarps * (lane % RPW)]);
        x.g = a.g[at * a.g_stride + h];
        return x;
    };
    Token next = fetch(0);
    float4 s[RPW];
#pragma unroll
    for (int j = 0; j < RPW; ++j) s[j] = *(const float4 *)(src + j * kWarps * kHeadDim);
    for (int t = 0; t < S; ++t) {
        const Token x = next;
        if (MULTI && t + 1 < S) next = fetch(t + 1);
        const float2 decay = decay_of(x.g);
        const F2 hi = f2(decay.x, decay.x), lo = f2(decay.y, decay.y);
        float p[RPW];
#pragma unroll
        for (int j = 0; j < RPW; ++j) {
            const F2 x01 = f2(s[j].x, s[j].y), x23 = f2(s[j].z, s[j].w);
            unf2(fma2(hi, x01, mul2(lo, x01)), s[j].x, s[j].y);
            unf2(fma2(hi, x23, mul2(lo, x23)), s[j].z, s[j].w);
            p[j] = s[j].x * x.q.x + s[j].y * x.q.y + s[j].z * x.q.z + s[j].w * x.q.w;
        }
        const float kq = warp_sum(x.k.x * x.q.x + x.k.y * x.q.y + x.k.z * x.q.z + x.k.w * x.q.w);
        const float before = scatter_sums<RPW>(p, lane);
        float *dst = a.pool + (slot_after(t) * a.H + h) * (int64_t)(kHeadDim * kHeadDim) + row_at;
#pragma unroll
        for (int j = 0; j < RPW; ++j) {
            const float v = __shfl_sync(0xffffffffu, x.v, j);
            s[j].x = fmaf(v, x.k.x, s[j].x), s[j].y = fmaf(v, x.k.y, s[j].y);
            s[j].z = fmaf(v, x.k.z, s[j].z), s[j].w = fmaf(v, x.k.w, s[j].w);
            *(float4 *)(dst + j * kWarps * kHeadDim) = s[j];
        }
        if (lane < RPW) o[(int64_t)t * a.H * kHeadDim + kWarps * lane] = from_f32<T>(a.scale * fmaf(x.v, kq, before));
    }
}

template <typename T, int RPW>
void launch(const LinearStepArgs &a, cudaStream_t stream, cudaError_t *e) {
    const dim3 grid((unsigned)((int64_t)a.N * a.H), kHeadDim / (kWarps * RPW));
    *e = launch_dependent(a.S == 1 && !a.num_accepted ? linear_step_kernel<T, RPW, false> : linear_step_kernel<T, RPW, true>,
                          grid, dim3(kThreads), 0, stream, a);
}

template <typename T>
cudaError_t launch(const LinearStepArgs &a, cudaStream_t stream) {
    cudaError_t e;
    // a head's rows go to several CTAs until there are some eight a SM (one sequence of 8 heads: 1.7 us of the device with 2 rows
    // a warp, 3.0 with 16; 32 of 16 heads: 7.2 with 4, 8.1 with 16, 9.0 with 2; 256 of 32 heads: 154 with 16, 175 with 2)
    int64_t ctas = (int64_t)a.N * a.H;
    int rpw = 16;
    while (rpw > 2 && ctas < 8 * sm_count()) rpw /= 2, ctas *= 2;
    switch (rpw) {
        case 16: launch<T, 16>(a, stream, &e); break;
        case 8: launch<T, 8>(a, stream, &e); break;
        case 4: launch<T, 4>(a, stream, &e); break;
        default: launch<T, 2>(a, stream, &e);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_step(const LinearStepArgs &a, int dtype, cudaStream_t stream) {
    return dtype == KDA_BF16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
}

}  // namespace kda
