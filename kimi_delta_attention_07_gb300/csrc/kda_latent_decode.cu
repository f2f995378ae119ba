// Absorbed latent attention over the paged cache: per query row (request n,
// new token s, head h), with rows c_p of 576 values (latent 512, key 64),
//   x_p = scale * q . c_p,  o = sum_p softmax(x)_p c_p[:512]
//
// The simplest form: a CTA per query row, each warp takes every eighth token
// with its own running maximum and sum, and the eight parts are joined in
// shared memory.
#include "kda_hybrid.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8;

__global__ void __launch_bounds__(kWarps * 32) latent_decode_kernel(const LatentDecodeArgs a) {
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kLatent];
    __shared__ int bad;
    const int h = blockIdx.x % a.H, s = (blockIdx.x / a.H) % a.S, n = blockIdx.x / (a.H * a.S);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    const int64_t len = a.seq_lens[n], cap = (int64_t)a.max_pages << a.page_shift;
    const bool len_ok = len >= 0 && len <= cap;
    const int64_t visible = len_ok ? len - a.S + 1 + s : 0;
    const int64_t row = (int64_t)blockIdx.x;
    float q[18], o[16], m = -INFINITY, l = 0.0f;
    for (int i = 0; i < 18; ++i) q[i] = to_f32(a.q[row * kLatentRow + lane + 32 * i]);
    for (int i = 0; i < 16; ++i) o[i] = 0.0f;
    if (len_ok)
        for (int64_t j = threadIdx.x; (j << a.page_shift) < len; j += blockDim.x) {
            const int p = a.block_table[(int64_t)n * a.max_pages + j];
            if (p < 0 || p >= a.n_pages) bad = 1;
        }
    else
        bad = 1;
    __syncthreads();
    const bool refused = bad != 0;
    for (int64_t p = wid; p < (refused ? 0 : visible); p += kWarps) {
        const int64_t page = a.block_table[(int64_t)n * a.max_pages + (p >> a.page_shift)];
        const __nv_bfloat16 *c =
            a.cache + ((page << a.page_shift) + (p & ((1 << a.page_shift) - 1))) * kLatentRow;
        float v[18], x = 0.0f;
        for (int i = 0; i < 18; ++i) {
            v[i] = to_f32(c[lane + 32 * i]);
            x += q[i] * v[i];
        }
        x = warp_sum(x) * a.scale;
        const float mn = fmaxf(m, x);
        const float f = m == -INFINITY ? 0.0f : expf(m - mn), e = expf(x - mn);
        l = l * f + e;
        for (int i = 0; i < 16; ++i) o[i] = o[i] * f + e * v[i];
        m = mn;
    }
    if (lane == 0) sm[wid] = m, sl[wid] = l;
    for (int i = 0; i < 16; ++i) so[wid][lane + 32 * i] = o[i];
    __syncthreads();
    m = -INFINITY;
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm[w]);
    l = 0.0f;
    for (int w = 0; w < kWarps; ++w) l += sm[w] == -INFINITY ? 0.0f : sl[w] * expf(sm[w] - m);
    for (int d = threadIdx.x; d < kLatent; d += blockDim.x) {
        float v = 0.0f;
        for (int w = 0; w < kWarps; ++w) v += sm[w] == -INFINITY ? 0.0f : so[w][d] * expf(sm[w] - m);
        v = l > 0.0f ? v / l : v;
        a.o[row * kLatent + d] = __float2bfloat16_rn(refused ? NAN : v);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[row] = refused ? NAN : m == -INFINITY ? -INFINITY : m + logf(l);
}

}  // namespace

size_t latent_decode_workspace_bytes(int n_seqs, int S, int H) { return 256; }

cudaError_t launch_latent_decode(const LatentDecodeArgs &a, cudaStream_t stream) {
    latent_decode_kernel<<<dim3((unsigned)(a.n_seqs * a.S * a.H)), kWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
