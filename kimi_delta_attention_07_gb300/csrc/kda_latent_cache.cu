// Append tokens to the paged latent cache: row = [ rms_norm(latent) * w ; key ].
//
// A warp per token: 576 bf16 are 72 vectors of 16 bytes, two latent vectors a
// lane and one positional vector for lanes 0..7, all requested before the slot is
// known to be valid and before the norm's shuffle reduction.  HBM bound: 1152
// bytes read and written a token; 16384 tokens take 7.5 us (5.1 TB/s), 8.0 us if
// the slot is waited for first.
#include "kda_hybrid.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;

__global__ void __launch_bounds__(kThreads) latent_cache_write_kernel(const CacheWriteArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (t >= a.n_tokens) return;
    const int64_t slot = a.slots[t];
    const __nv_bfloat16 *src = a.kv + t * a.kv_stride;
    __nv_bfloat16 *dst = a.cache + slot * kLatentRow;
    float c[2][8];
    load8(src + 8 * lane, c[0]);
    load8(src + 8 * lane + 256, c[1]);
    uint4 key;
    if (lane < kRope / 8) key = *reinterpret_cast<const uint4 *>(src + kLatent + 8 * lane);
    if (a.weight) {
        float w[2][8];
        load8(a.weight + 8 * lane, w[0]);
        load8(a.weight + 8 * lane + 256, w[1]);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += c[i][j] * c[i][j];
        const float rn = 1.0f / sqrtf(warp_sum(sum) * (1.0f / kLatent) + a.eps);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) c[i][j] *= rn * w[i][j];
    }
    if (slot < 0 || slot >= a.n_rows) return;
    store8(dst + 8 * lane, c[0]);
    store8(dst + 8 * lane + 256, c[1]);
    if (lane < kRope / 8) *reinterpret_cast<uint4 *>(dst + kLatent + 8 * lane) = key;
}

}  // namespace

cudaError_t launch_latent_cache_write(const CacheWriteArgs &a, cudaStream_t stream) {
    const int64_t grid = (a.n_tokens + kThreads / 32 - 1) / (kThreads / 32);
    const cudaError_t e = launch_dependent(latent_cache_write_kernel, dim3((unsigned)grid),
                                           dim3(kThreads), 0, stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kda
