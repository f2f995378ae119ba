// Linear attention with one decay a head over packed fp32 sequences, token by token on the CUDA cores:
//   S <- e^g S + k v^T,  o = scale S^T q
//
// A CTA takes 64 rows of S^T (value channels) of one (segment, head), eight lanes for four rows and sixteen key
// channels a lane, in registers.  Tokens come through shared memory in blocks of sixteen, the next block
// requested while one is worked on; two tokens share the lanes' exchange for o.
//
// Eight tokens at a time with G_t the decays since their first one: S_t = e^{G_t} (S_0 + sum_j e^{-G_j} k_j v_j^T), so
// that an element of the state costs one fma a token, and one for o, and e^{G_8} once in eight;
// in fp32 while |G| < 8 (2^-22 in e^{G_t - G_j}), else token by token.  Sequences are cut into
// segments (kda_linear_segments.cuh).
//
// Two sequences of 1001 and 500 tokens, 16 heads: 91 us; 135 with two rows a thread, 196 with
// a product for each decay and one row a thread, 252 uncut and with an exchange a token.  What bounds it: 12 warps
// a SM (their registers hold the state), whose fma and shared-memory pipes are each half busy (4096 tokens of
// 32 heads: 369 us, of which 174 are its fmas at the pipe's rate).
//
// A decay near one is the sum of two floats (decay_of).
#include <algorithm>
#include <type_traits>

#include "kda_linear_segments.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kRows = 64;   // of S^T, a CTA
constexpr int kLanes = 8;   // of a row
constexpr int kOwn = 4;     // rows of a thread, next to one another
constexpr int kThreads = kRows / kOwn * kLanes;
constexpr int kBlock = 16;  // tokens in shared memory at a time, twice
constexpr int kSub = 8;     // tokens that share a reference for their decays
constexpr float kMostDecay = 8.0f;

__device__ __forceinline__ void copy16(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(to)), "l"(from) : "memory");
}

// OUTPUT: o and final states, from the states in front of the segments; else a segment's own state.
template <bool OUTPUT, Source SOURCE>
__global__ void __launch_bounds__(kThreads, 3) linear_chunk_f32_kernel(const ChunkParams p) {
    // (a row of 128 channels as 8 lanes of 16: channel 32 i + 4 l + j is lane l's)
    __shared__ __align__(16) float sq[OUTPUT ? 2 : 1][OUTPUT ? kBlock : 1][kHeadDim], sk[2][kBlock][kHeadDim], sv[2][kBlock][kRows];
    __shared__ float2 sg[2][kBlock];          // a token's decay
    __shared__ float2 su[2][kBlock];          // e^{G_t}, e^{-G_t}
    __shared__ float2 se[2][kBlock / kSub];   // e^{G_8}
    __shared__ bool strong[2][kBlock / kSub]; // |G| >= kMostDecay
    griddep_wait();
    griddep_launch_dependents();
    const LinearChunkArgs &a = p.a;
    const int row0 = blockIdx.y * kRows, tid = threadIdx.x, row = tid / kLanes * kOwn, l = tid % kLanes;
    for_segments<OUTPUT, SOURCE>(p, blockIdx.x, gridDim.x, [&](const Item &seg) {
        const int h = head_of(seg), len = seg.y;
        const int64_t first = seg.x;
        float *o = (float *)a.o + h * kHeadDim + row0;
        if (seg.w & kNoSlot) {
            for (int64_t i = tid; i < (int64_t)len * kRows; i += kThreads)
                o[(first + i / kRows) * a.H * kHeadDim + i % kRows] = __int_as_float(0x7fc00000);
            return;
        }
        const float *q = (const float *)a.q + h / a.group * kHeadDim, *k = (const float *)a.k + h / a.group * kHeadDim,
                    *v = (const float *)a.v + h * kHeadDim + row0;
        float rg = 0.0f, total = 0.0f;
        auto request = [&](int t0, int buf) {
#pragma unroll
            for (int i = 0; i < kBlock * kHeadDim / 4 / kThreads; ++i) {
                const int t = tid / 32 + i * (kThreads / 32);
                if (t0 + t >= len) continue;
                if (OUTPUT) copy16(&sq[buf][t][4 * (tid % 32)], q + (first + t0 + t) * a.q_stride + 4 * (tid % 32));
                copy16(&sk[buf][t][4 * (tid % 32)], k + (first + t0 + t) * a.k_stride + 4 * (tid % 32));
            }
#pragma unroll
            for (int i = 0; i < kBlock * kRows / 4 / kThreads; ++i) {
                const int t = tid / (kRows / 4) + i * (4 * kThreads / kRows), at = 4 * (tid % (kRows / 4));
                if (t0 + t < len) copy16(&sv[buf][t][at], v + (first + t0 + t) * a.v_stride + at);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (tid < kBlock) rg = t0 + tid < len ? a.g[(first + t0 + tid) * a.g_stride + h] : 0.0f;
        };
        __syncthreads();  // (the segment before it is done with the buffers)
        request(0, 0);
        const int place = (row0 + row) * kHeadDim + 4 * l;  // of this thread's part of a state
        F2 s[kOwn][8];
        const float *init = OUTPUT ? state_before(p, seg) : nullptr;
#pragma unroll
        for (int i = 0; i < 4 * kOwn; ++i) {
            const float4 x = init ? *(const float4 *)(init + place + (i >> 2) * kHeadDim + 32 * (i & 3)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            s[i >> 2][2 * (i & 3)] = f2(x.x, x.y), s[i >> 2][2 * (i & 3) + 1] = f2(x.z, x.w);
        }
        // where lane l's share of two tokens' o goes: row l % 4 of token l / 4
        const int64_t o_step = (int64_t)a.H * kHeadDim;
        float *o_at = o + (first + (l >> 2)) * o_step + row + (l & 3);
        for (int t0 = 0, buf = 0; t0 < len; t0 += kBlock, buf ^= 1) {
            if (tid < 32) {
                const float g = tid < kBlock ? rg : 0.0f;
                float G = g;
#pragma unroll
                for (int m = 1; m < kSub; m <<= 1) {
                    const float x = __shfl_up_sync(0xffffffffu, G, m);
                    if (tid % kSub >= m) G += x;
                }
                const uint32_t weak = __ballot_sync(0xffffffffu, fabsf(G) < kMostDecay);
                if (tid < kBlock) {
                    sg[buf][tid] = decay_of(g);
                    su[buf][tid] = make_float2(expf(G), expf(-G));
                    if (tid % kSub == kSub - 1) {
                        se[buf][tid / kSub] = decay_of(G);
                        strong[buf][tid / kSub] = ((weak >> (tid - (kSub - 1))) & 0xff) != 0xff;
                    }
                    total += g;
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();
            request(t0 + kBlock, buf ^ 1);
            // the sums over eight lanes of eight values (four rows of two tokens): lane l gets that of value l
            auto reduce = [&](float (&x)[8]) {
#pragma unroll
                for (int m = 4; m > 0; m >>= 1) {
                    const bool hi = l & m;
#pragma unroll
                    for (int i = 0; i < m; ++i) {
                        const float send = hi ? x[i] : x[i + m];
                        x[i] = (hi ? x[i + m] : x[i]) + __shfl_xor_sync(0xffffffffu, send, m);
                    }
                }
                return x[0];
            };
            // one token: S += k v^T, behind a product with its decay where the tokens have no reference; x: this lane's parts of S^T q
            auto step = [&](int t, auto decays, float *x) {
                const float2 d = decays ? sg[buf][t] : su[buf][t];
                const float4 vt = *(const float4 *)&sv[buf][t][row];
                const float scale = decays ? 1.0f : d.y;
                const float vs[kOwn] = {vt.x * scale, vt.y * scale, vt.z * scale, vt.w * scale};
                F2 sum[kOwn] = {};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 kk = *(const float4 *)&sk[buf][t][4 * l + 32 * i];
                    const F2 k2[2] = {f2(kk.x, kk.y), f2(kk.z, kk.w)};
                    F2 q2[2];
                    if (OUTPUT) {
                        const float4 qq = *(const float4 *)&sq[buf][t][4 * l + 32 * i];
                        q2[0] = f2(qq.x, qq.y), q2[1] = f2(qq.z, qq.w);
                    }
#pragma unroll
                    for (int r = 0; r < kOwn; ++r)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            F2 &y = s[r][2 * i + j];
                            if (decays) y = fma2(f2(d.x, d.x), y, fma2(f2(d.y, d.y), y, mul2(f2(vs[r], vs[r]), k2[j])));
                            else y = fma2(f2(vs[r], vs[r]), k2[j], y);
                            if (OUTPUT) sum[r] = fma2(y, q2[j], sum[r]);
                        }
                }
#pragma unroll
                for (int r = 0; r < kOwn; ++r) {
                    float lo, hi;
                    unf2(sum[r], lo, hi);
                    x[r] = (lo + hi) * (decays ? 1.0f : d.x);
                }
            };
            auto tokens = [&](int begin, int end, auto decays) {
#pragma unroll 1
                for (int t = begin; t < end; t += 2) {
                    float x[8] = {};
                    step(t, decays, x);
                    if (t + 1 < end) step(t + 1, decays, x + 4);
                    if (OUTPUT) {
                        const float sum = reduce(x);
                        if (t + (l >> 2) < end) o_at[(int64_t)(t0 + t) * o_step] = a.scale * sum;
                    }
                }
            };
            const int block = min(kBlock, len - t0);
#pragma unroll 1
            for (int b = 0; b * kSub < block; ++b) {
                const int end = min((b + 1) * kSub, block);
                if (strong[buf][b]) {
                    tokens(b * kSub, end, std::true_type());
                } else {
                    tokens(b * kSub, end, std::false_type());
                    const float2 d = se[buf][b];
#pragma unroll
                    for (int i = 0; i < 8 * kOwn; ++i) {
                        F2 &y = s[i >> 3][i & 7];
                        y = fma2(f2(d.x, d.x), y, mul2(f2(d.y, d.y), y));
                    }
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        float *out = OUTPUT ? state_after(p, seg) : p.states + entry_of(p, seg) * kState;
        if (out)
#pragma unroll
            for (int i = 0; i < 4 * kOwn; ++i) {
                float4 x;
                unf2(s[i >> 2][2 * (i & 3)], x.x, x.y), unf2(s[i >> 2][2 * (i & 3) + 1], x.z, x.w);
                *(float4 *)(out + place + (i >> 2) * kHeadDim + 32 * (i & 3)) = x;
            }
        if (!OUTPUT && blockIdx.y == 0 && tid < 32) {
            total = warp_sum(tid < kBlock ? total : 0.0f);
            if (tid == 0) p.decay[entry_of(p, seg)] = decay_of(total);
        }
    });
}

// Tokens of a segment: so many that there are some twelve CTAs a SM, of which three are resident (4096 tokens of 16 heads:
// 210 us; six 220, sixteen 220), and 64 at least (two sequences of 1001 and 500 tokens: 94 us; 32 100, 96 111).
inline Cut cut_of(int64_t total_tokens, int n_seqs, int H) {
    constexpr int64_t kLeast = 64, kStep = 2 * kBlock;
    const int64_t each = std::max<int64_t>(1, 12 * sm_count() / (H * (kHeadDim / kRows)));
    const int64_t segment = std::max(kLeast, kStep * ((total_tokens + each * kStep - 1) / (each * kStep)));
    // Three CTAs of an SM share its fma pipe: with nothing but one sequence to fill the SMs, segments and heads go at the rate of
    // 0.7 an SM (1024 tokens of 64 heads: 196 us cut, 212 uncut), and two more launches count like 64 tokens.
    if (n_seqs == 1) return {segment, 7 * sm_count() / 10, 64};
    return {segment, 3 * sm_count() / (kHeadDim / kRows), 24};
}

}  // namespace

size_t linear_chunk_f32_workspace_bytes(int64_t total_tokens, int n_seqs, int H) {
    return segments_workspace_bytes(total_tokens, n_seqs, H, cut_of(total_tokens, n_seqs, H));
}

cudaError_t launch_linear_chunk_f32(const LinearChunkArgs &a, cudaStream_t stream) {
    const ChunkParams p = plan_segments(a, cut_of(a.total_tokens, a.n_seqs, a.H));
    const Source source = source_of(p);
    auto launch = [&](auto kernel, int64_t items) {
        return launch_dependent(kernel, dim3((unsigned)items, kHeadDim / kRows), dim3(kThreads), 0, stream, p);
    };
    cudaError_t e = launch_segment_lists(p, stream);
    if (e == cudaSuccess && p.entries > 0) {
        e = launch(source == kOne ? linear_chunk_f32_kernel<false, kOne> : linear_chunk_f32_kernel<false, kListed>, (int64_t)p.entries * a.H);
        if (e == cudaSuccess) e = launch_segment_join(p, stream);
    }
    if (e == cudaSuccess)
        e = launch(source == kOne     ? linear_chunk_f32_kernel<true, kOne>
                   : source == kWhole ? linear_chunk_f32_kernel<true, kWhole>
                                      : linear_chunk_f32_kernel<true, kListed>,
                   ((int64_t)p.entries + a.n_seqs) * a.H);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kda
