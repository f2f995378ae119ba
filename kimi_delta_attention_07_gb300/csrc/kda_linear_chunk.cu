// Linear attention with one decay a head over packed sequences, token by token on the CUDA
// cores: the path of fp32 inputs.
//   S <- e^g S + k v^T,  o = scale S^T q
//
// 3 * 128 * 128 fp32 operations a token and head.  A CTA takes sixteen rows of S^T (value
// channels) of one (sequence, head), eight lanes a row and sixteen key channels a lane in
// registers, so that the only exchange is the sum of eight lanes for o.  Tokens come through shared
// memory in blocks of sixteen, the next block requested while one is worked on.
#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int kRows = 16;  // of S^T, a CTA
constexpr int kLanes = 8;  // of a row
constexpr int kThreads = kRows * kLanes;
constexpr int kPer = kHeadDim / kLanes;  // key channels of a lane: four times four, 32 apart
constexpr int kBlock = 16;               // tokens in shared memory at a time

__global__ void __launch_bounds__(kThreads) linear_chunk_f32_kernel(const LinearChunkArgs a) {
    __shared__ __align__(16) float sq[kBlock][kHeadDim], sk[kBlock][kHeadDim];
    __shared__ float sv[kBlock][kRows], sg[kBlock];
    griddep_wait();
    griddep_launch_dependents();
    const int n = blockIdx.x / a.H, h = blockIdx.x - n * a.H, row0 = blockIdx.y * kRows;
    const int tid = threadIdx.x, row = tid / kLanes, l = tid % kLanes;
    const Span span = span_of(a, n);
    if (span.len < 0) return;
    const int64_t slot = slot_of(a, n);
    const int64_t first = span.first;
    float *o = (float *)a.o + h * kHeadDim + row0;
    if (slot < 0) {
        for (int64_t i = tid; i < (int64_t)span.len * kRows; i += kThreads)
            o[(first + i / kRows) * a.H * kHeadDim + i % kRows] = (__int_as_float(0x7fc00000));
        return;
    }
    const int64_t state_at = (slot * a.H + h) * (int64_t)(kHeadDim * kHeadDim) + (int64_t)(row0 + row) * kHeadDim + 4 * l;
    float4 s[kPer / 4];
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i)
        s[i] = a.initial_state ? *(const float4 *)(a.initial_state + state_at + 32 * i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float *q = (const float *)a.q + h / a.group * kHeadDim, *k = (const float *)a.k + h / a.group * kHeadDim,
            *v = (const float *)a.v + h * kHeadDim + row0;
    constexpr int kVecs = kBlock * kHeadDim / 4 / kThreads;  // of four channels, of q (and of k) a thread
    float4 rq[kVecs], rk[kVecs];
    float rv[kBlock * kRows / kThreads], rg = 0.0f;
    auto request = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int t = t0 + tid / 32 + i * (kThreads / 32);
            if (t >= span.len) continue;
            rq[i] = load4(q + (first + t) * a.q_stride + 4 * (tid % 32));
            rk[i] = load4(k + (first + t) * a.k_stride + 4 * (tid % 32));
        }
#pragma unroll
        for (int i = 0; i < kBlock * kRows / kThreads; ++i) {
            const int t = t0 + (tid + i * kThreads) / kRows;
            if (t < span.len) rv[i] = (v[(first + t) * a.v_stride + tid % kRows]);
        }
        if (tid < kBlock && t0 + tid < span.len) rg = a.g[(first + t0 + tid) * a.g_stride + h];
    };
    request(0);
    for (int t0 = 0; t0 < span.len; t0 += kBlock) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            *(float4 *)&sq[tid / 32 + i * (kThreads / 32)][4 * (tid % 32)] = rq[i];
            *(float4 *)&sk[tid / 32 + i * (kThreads / 32)][4 * (tid % 32)] = rk[i];
        }
#pragma unroll
        for (int i = 0; i < kBlock * kRows / kThreads; ++i) sv[(tid + i * kThreads) / kRows][tid % kRows] = rv[i];
        if (tid < kBlock) sg[tid] = expf(rg);
        __syncthreads();
        request(t0 + kBlock);
        const int block = min(kBlock, span.len - t0);
        for (int t = 0; t < block; ++t) {
            const float decay = sg[t], vt = sv[t][row];
            float sum[kPer / 4];
#pragma unroll
            for (int i = 0; i < kPer / 4; ++i) {
                const float4 kk = *(const float4 *)&sk[t][4 * l + 32 * i], qq = *(const float4 *)&sq[t][4 * l + 32 * i];
                s[i].x = fmaf(decay, s[i].x, vt * kk.x), s[i].y = fmaf(decay, s[i].y, vt * kk.y);
                s[i].z = fmaf(decay, s[i].z, vt * kk.z), s[i].w = fmaf(decay, s[i].w, vt * kk.w);
                sum[i] = s[i].x * qq.x + s[i].y * qq.y + s[i].z * qq.z + s[i].w * qq.w;
            }
            float x = (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
            for (int m = 1; m < kLanes; m <<= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
            if (l == 0) o[(first + t0 + t) * a.H * kHeadDim + row] = (a.scale * x);
        }
    }
    if (a.final_state)
#pragma unroll
        for (int i = 0; i < kPer / 4; ++i) *(float4 *)(a.final_state + state_at + 32 * i) = s[i];
}

}  // namespace

cudaError_t launch_linear_chunk_f32(const LinearChunkArgs &a, cudaStream_t stream) {
    const cudaError_t e = launch_dependent(linear_chunk_f32_kernel, dim3((unsigned)(a.n_seqs * a.H), kHeadDim / kRows),
                                           dim3(kThreads), 0, stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kda
