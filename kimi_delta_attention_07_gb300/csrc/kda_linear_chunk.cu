// Linear attention with one decay a head over packed fp32 sequences, token by token on the CUDA cores:
//   S <- e^g S + k v^T,  o = scale S^T q
//
// 6 * 128 * 128 fp32 operations a token and head.  A CTA takes sixteen rows of S^T (value
// channels) of one (segment, head), eight lanes a row and sixteen key channels a lane in
// registers.  Tokens come through shared memory in blocks of sixteen, the next block requested
// while one is worked on; four tokens share the lanes' exchange for o.  What bounds it is the chain of
// a token's instructions, so that long sequences are cut into segments (kda_linear_segments.cuh):
// two sequences of 1001 and 500 tokens, 16 heads, @ us, 252 us uncut and with an exchange a token.
//
// A decay near one is the sum of two floats: as one, its rounding error would come back in every
// token that it is applied to (a fixed decay of 2^-8 a token: 1e-5 in the state).
#include <algorithm>

#include "kda_linear_segments.cuh"

namespace kda {
namespace {

constexpr int kRows = 16;  // of S^T, a CTA
constexpr int kLanes = 8;  // of a row
constexpr int kThreads = kRows * kLanes;
constexpr int kBlock = 16;  // tokens in shared memory at a time

// OUTPUT: o and final states, from the states in front of the segments; else a segment's own state.
template <bool OUTPUT>
__global__ void __launch_bounds__(kThreads) linear_chunk_f32_kernel(const ChunkParams p) {
    // (a row of 128 channels as 8 lanes of 16: channel 32 i + 4 l + j is lane l's)
    __shared__ __align__(16) float sq[OUTPUT ? kBlock : 1][kHeadDim], sk[kBlock][kHeadDim];
    __shared__ float sv[kBlock][kRows];
    __shared__ float2 sg[kBlock];
    griddep_wait();
    griddep_launch_dependents();
    const LinearChunkArgs &a = p.a;
    const int row0 = blockIdx.y * kRows, tid = threadIdx.x, row = tid / kLanes, l = tid % kLanes;
    for_segments<OUTPUT>(p, blockIdx.x, gridDim.x, [&](const Item &seg) {
        const int h = head_of(seg), len = seg.y;
        const int64_t first = seg.x;
        float *o = (float *)a.o + h * kHeadDim + row0;
        if (seg.w & kNoSlot) {
            for (int64_t i = tid; i < (int64_t)len * kRows; i += kThreads)
                o[(first + i / kRows) * a.H * kHeadDim + i % kRows] = __int_as_float(0x7fc00000);
            return;
        }
        const int place = (row0 + row) * kHeadDim + 4 * l;  // of this thread's part of a state
        F2 s[8];
        const float *init = OUTPUT ? state_before(p, seg) : nullptr;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 x = init ? *(const float4 *)(init + place + 32 * i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            s[2 * i] = f2(x.x, x.y), s[2 * i + 1] = f2(x.z, x.w);
        }
        const float *q = (const float *)a.q + h / a.group * kHeadDim, *k = (const float *)a.k + h / a.group * kHeadDim,
                    *v = (const float *)a.v + h * kHeadDim + row0;
        constexpr int kVecs = kBlock * kHeadDim / 4 / kThreads;  // of four channels, of q (and of k) a thread
        float4 rq[kVecs], rk[kVecs];
        float rv[kBlock * kRows / kThreads], rg = 0.0f, total = 0.0f;
        auto request = [&](int t0) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int t = t0 + tid / 32 + i * (kThreads / 32);
                if (t >= len) continue;
                if (OUTPUT) rq[i] = *(const float4 *)(q + (first + t) * a.q_stride + 4 * (tid % 32));
                rk[i] = *(const float4 *)(k + (first + t) * a.k_stride + 4 * (tid % 32));
            }
#pragma unroll
            for (int i = 0; i < kBlock * kRows / kThreads; ++i) {
                const int t = t0 + (tid + i * kThreads) / kRows;
                if (t < len) rv[i] = v[(first + t) * a.v_stride + tid % kRows];
            }
            if (tid < kBlock) rg = t0 + tid < len ? a.g[(first + t0 + tid) * a.g_stride + h] : 0.0f;
        };
        request(0);
        for (int t0 = 0; t0 < len; t0 += kBlock) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int t = tid / 32 + i * (kThreads / 32);
                if (OUTPUT) *(float4 *)&sq[t][4 * (tid % 32)] = rq[i];
                *(float4 *)&sk[t][4 * (tid % 32)] = rk[i];
            }
#pragma unroll
            for (int i = 0; i < kBlock * kRows / kThreads; ++i) sv[(tid + i * kThreads) / kRows][tid % kRows] = rv[i];
            if (tid < kBlock) {
                const float d = expf(rg);
                // (d - 1 is exact from 1/2 to 2; smaller decays leave nothing for their error to come back in)
                sg[tid] = make_float2(d, d > 0.5f && d < 2.0f ? expm1f(rg) - (d - 1.0f) : 0.0f);
                total += rg;
            }
            __syncthreads();
            request(t0 + kBlock);
            const int block = min(kBlock, len - t0);
            auto step = [&](int t) {  // this lane's part of row . q
                const float2 d = sg[t];
                const float vt = sv[t][row];
                F2 sum = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 kk = *(const float4 *)&sk[t][4 * l + 32 * i];
                    const F2 k2[2] = {f2(kk.x, kk.y), f2(kk.z, kk.w)};
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        s[2 * i + j] = fma2(f2(d.x, d.x), s[2 * i + j], fma2(f2(d.y, d.y), s[2 * i + j], mul2(f2(vt, vt), k2[j])));
                    if (OUTPUT) {
                        const float4 qq = *(const float4 *)&sq[t][4 * l + 32 * i];
                        sum = fma2(s[2 * i], f2(qq.x, qq.y), sum);
                        sum = fma2(s[2 * i + 1], f2(qq.z, qq.w), sum);
                    }
                }
                float lo, hi;
                unf2(sum, lo, hi);
                return lo + hi;
            };
            int t = 0;
            for (; t + 4 <= block; t += 4) {
                float x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = step(t + i);
                if (OUTPUT) {
                    // the sums over eight lanes of four tokens: lane l gets token l % 4's
#pragma unroll
                    for (int m = 2; m > 0; m >>= 1) {
                        const bool hi = l & m;
#pragma unroll
                        for (int i = 0; i < m; ++i) {
                            const float send = hi ? x[i] : x[i + m];
                            x[i] = (hi ? x[i + m] : x[i]) + __shfl_xor_sync(0xffffffffu, send, m);
                        }
                    }
                    x[0] += __shfl_xor_sync(0xffffffffu, x[0], 4);
                    if (l < 4) o[(first + t0 + t + l) * a.H * kHeadDim + row] = a.scale * x[0];
                }
            }
            for (; t < block; ++t) {
                float x = step(t);
                if (OUTPUT) {
#pragma unroll
                    for (int m = 1; m < kLanes; m <<= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
                    if (l == 0) o[(first + t0 + t) * a.H * kHeadDim + row] = a.scale * x;
                }
            }
        }
        float *out = OUTPUT ? state_after(p, seg) : p.states + entry_of(p, seg) * kState;
        if (out)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float4 x;
                unf2(s[2 * i], x.x, x.y), unf2(s[2 * i + 1], x.z, x.w);
                *(float4 *)(out + place + 32 * i) = x;
            }
        if (!OUTPUT && blockIdx.y == 0 && tid < 32) {
            total = warp_sum(tid < kBlock ? total : 0.0f);
            if (tid == 0) p.decay[entry_of(p, seg)] = expf(total);
        }
    });
}

// Tokens of a segment: so many that there are some four CTAs a SM, and no fewer than cost what the cut costs.
inline int64_t segment_of(int64_t total_tokens, int H) {
    constexpr int64_t kLeast = 128;
    const int64_t each = std::max<int64_t>(1, 4 * sm_count() / (H * (kHeadDim / kRows)));
    return kLeast * std::max<int64_t>(1, (total_tokens + each * kLeast - 1) / (each * kLeast));
}

}  // namespace

size_t linear_chunk_f32_workspace_bytes(int64_t total_tokens, int n_seqs, int H) {
    return segments_workspace_bytes(total_tokens, n_seqs, H, segment_of(total_tokens, H));
}

cudaError_t launch_linear_chunk_f32(const LinearChunkArgs &a, cudaStream_t stream) {
    const ChunkParams p = plan_segments(a, segment_of(a.total_tokens, a.H));
    auto launch = [&](auto kernel, int64_t items) {
        return launch_dependent(kernel, dim3((unsigned)items, kHeadDim / kRows), dim3(kThreads), 0, stream, p);
    };
    cudaError_t e = launch_segment_lists(p, stream);
    if (e == cudaSuccess && p.entries > 0) {
        e = launch(linear_chunk_f32_kernel<false>, (int64_t)p.entries * a.H);
        if (e == cudaSuccess) e = launch_segment_join(p, stream);
    }
    if (e == cudaSuccess) e = launch(linear_chunk_f32_kernel<true>, ((int64_t)p.entries + a.n_seqs) * a.H);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kda
