// Expanded latent attention over packed sequences: per (query i, head h) with
// keys k_j = [kv[j,h,:128] ; k_rope[j]] and values v_j = kv[j,h,128:],
//   x_j = scale * q . k_j over visible j,  o = sum_j softmax(x)_j v_j
//
// The simplest form: a warp takes four queries of one head and runs over the
// keys with a running maximum and sum.
#include "kda_hybrid.cuh"

namespace kda {
namespace {

constexpr int kRows = 4, kWarps = 8;

__global__ void __launch_bounds__(kWarps * 32) latent_prefill_kernel(const LatentPrefillArgs a) {
    const int lane = threadIdx.x & 31, h = blockIdx.y;
    const int64_t t0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRows;
    float q[kRows][6], o[kRows][4], m[kRows], l[kRows];
    int64_t k0 = 0, limit[kRows], most = 0;
    int last = -1;
    for (int r = 0; r < kRows; ++r) {
        limit[r] = -1;
        const int64_t t = t0 + r;
        m[r] = -INFINITY, l[r] = 0.0f;
        for (int i = 0; i < 4; ++i) o[r][i] = 0.0f;
        if (t >= a.total_q) continue;
        for (int n = 0; n < a.n_seqs; ++n) {
            const int64_t qa = a.cu_q[n], qb = a.cu_q[n + 1], ka = a.cu_k[n], kb = a.cu_k[n + 1];
            if (qa < 0 || qb > a.total_q || ka < 0 || kb < ka || kb > a.total_k || t < qa || t >= qb) continue;
            const int64_t vis = a.causal ? min(kb - ka, t - qa + 1 + (kb - ka) - (qb - qa)) : kb - ka;
            limit[r] = max(vis, (int64_t)0);
            if (last >= 0 && n != last) limit[r] = -2 - limit[r];  // a row of another sequence: alone
            else last = n, k0 = ka;
            break;
        }
        for (int i = 0; i < 6; ++i) q[r][i] = to_f32(a.q[t * a.q_stride + (int64_t)h * kQk + lane + 32 * i]);
        if (limit[r] >= 0) most = max(most, limit[r]);
    }
    for (int pass = 0; pass < kRows; ++pass) {
        for (int64_t j = 0; j < most; ++j) {
            const __nv_bfloat16 *kv = a.kv + (k0 + j) * a.kv_stride + (int64_t)h * kKvRow;
            float k[6], v[4];
            for (int i = 0; i < 4; ++i) {
                k[i] = to_f32(kv[lane + 32 * i]);
                v[i] = to_f32(kv[kNope + lane + 32 * i]);
            }
            for (int i = 0; i < 2; ++i) k[4 + i] = to_f32(a.k_rope[(k0 + j) * a.rope_stride + lane + 32 * i]);
            for (int r = 0; r < kRows; ++r) {
                float x = 0.0f;
                for (int i = 0; i < 6; ++i) x += q[r][i] * k[i];
                x = warp_sum(x) * a.scale;
                if (j >= limit[r]) continue;
                const float mn = fmaxf(m[r], x), f = m[r] == -INFINITY ? 0.0f : expf(m[r] - mn), e = expf(x - mn);
                l[r] = l[r] * f + e;
                for (int i = 0; i < 4; ++i) o[r][i] = o[r][i] * f + e * v[i];
                m[r] = mn;
            }
        }
        // write the rows of this pass's sequence, then take the next sequence among the four rows
        most = 0;
        int next = -1;
        for (int r = 0; r < kRows; ++r) {
            const int64_t t = t0 + r;
            if (limit[r] >= 0) {
                for (int i = 0; i < 4; ++i)
                    a.o[(t * a.H + h) * kHeadDim + lane + 32 * i] =
                        __float2bfloat16_rn(l[r] > 0.0f ? o[r][i] / l[r] : o[r][i]);
                if (a.lse && lane == 0)
                    a.lse[t * a.H + h] = m[r] == -INFINITY ? -INFINITY : m[r] + logf(l[r]);
                limit[r] = -1;
            } else if (limit[r] <= -2) {
                int n = 0;
                while (!(a.cu_q[n] <= t && t < a.cu_q[n + 1])) ++n;
                if (next < 0 || n == next) {
                    next = n;
                    k0 = a.cu_k[n];
                    limit[r] = -2 - limit[r];
                    most = max(most, limit[r]);
                }
            }
        }
        if (next < 0) break;
    }
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, cudaStream_t stream) {
    const int64_t blocks = (a.total_q + kWarps * kRows - 1) / (kWarps * kRows);
    latent_prefill_kernel<<<dim3((unsigned)blocks, a.H), kWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
