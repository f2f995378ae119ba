// Linear attention with one decay a head over packed bf16 sequences, on the tensor cores.
//
// A chunk of 128 tokens of a head, with G_i the sum of its decays up to token i, S the state
// in front of it:
//   o_i = scale (sum_{j<=i} e^{G_i - G_j} (q_i . k_j) v_j + e^{G_i} S^T q_i)
//   S  <- e^{G_127} S + sum_j e^{G_127 - G_j} k_j v_j^T
// as four products of 128 x 128 x 128:
//   X  [i x j] = Q . K^T     shared memory, both K-major
//   O  [i x e] = Q . S       S as bf16 in shared memory, [key][value]; then rows times e^{G_i}
//   O          += P . V      P = X times its decays, bf16 in TMEM over X
//   D  [d x e] = Kt . V      Kt = K^T times e^{G_127 - G_j}, in TMEM: lane = key channel
// S stays in registers (fp32, lane = key channel) for as long as a CTA works on a sequence:
// S = e^{G_127} S + D, which the tensor core could not scale.
//
// What is rounded: P and the copy of S that O is taken from, to bf16 (as o itself is, so that o's
// rounding variance doubles; both are read once and kept nowhere).  Kt enters the states, which
// are fp32 and live on: it is split into three bf16 terms that hold all 24 bits, three products
// instead of one.  With two terms the states would be off by 2.3e-6, with one by 1.6e-3.
//
// Decays are taken inside blocks of 32 tokens: a prefix sum, a suffix sum and the blocks'
// totals, so that every exponent that matters is a short sum of its own terms; between
// blocks e^{G_i - G_j} is a product of a factor of row i and one of column j, both <= 1,
// which leaves 32 exponentials a row instead of 128.
//
// Long sequences of few heads are cut into segments (a whole number of chunks each, so
// many that a GPU is filled): a first kernel takes every segment's own state from zero (all but
// each sequence's last), a second one joins them to the states in front of the segments, a
// third one computes the outputs.  Two instantiations of one kernel are the first and
// the third.
//
// Masked places: rows of a tile past the sequence's end are emptied (V) or taken as 0 (K).  A
// value that is not finite would reach rows before it as 0 times it: V is looked through,
// such values become 0 and their channel NaN from their row on, in o and in S.
//
// Warps: 0 TMA, 1 MMA of X and O, 2 MMA of D, 3 decays, 4..7 Kt, 8..11 check of V and P,
// 12..19 the state and the outputs, 64 value channels each half.
#include <algorithm>

#include "kda_attn.cuh"
#include "kda_linear.cuh"

namespace kda {

using namespace tc;

namespace {

constexpr int kTok = 128;  // tokens of a chunk
constexpr int kThreads = 640;
constexpr uint32_t kTile = 32768;        // 128 tokens x 128 channels: two blocks of 64 channels
constexpr uint32_t kHalf = kTile / 2;
constexpr int kState = kHeadDim * kHeadDim;

// shared memory (from a 1024-byte boundary): two stages of K, Q, V; the copy of S
constexpr uint32_t kSmK = 0, kSmQ = 2 * kTile, kSmV = 4 * kTile, kSmS = 6 * kTile, kSmShared = 7 * kTile;

// TMEM columns: X and P, O, D, two buffers of 32 tokens of Kt in three terms of 16 columns
constexpr uint32_t kTmO = 128, kTmD = 256, kTmK = 384, kTmTerm = 16, kTmBuf = 48;

struct Shared {
    uint64_t kq_full[2], v_full[2], k_empty[2], q_empty[2], v_empty[2], gates_full[2], gates_empty[2], v_ready[2],
        kt_full[2], kt_empty[2], x_full, p_full, qs_full, o_scaled, o_full, o_empty, s_full, d_full, d_empty;
    alignas(16) float lower[2][kTok];  // log2 decay of a token's block up to and with it
    float upper[2][kTok];   // decay of a token's block behind it
    float block[2][4];      // log2 decay of each block
    uint8_t odd[2][kTok];   // a value channel's first row that is not finite, if any_odd; else kTok
    volatile int any_odd[2], dead;
    uint32_t tmem_base;
};
constexpr uint32_t kSmemBytes = kSmShared + sizeof(Shared);
static_assert(kSmemBytes <= 232448, "shared memory");

struct ChunkParams {
    LinearChunkArgs a;
    int segment;     // tokens
    int entries;     // segments whose state the workspace holds, at most
    int64_t items;   // of the kernel with outputs: (segment, head)
    float *states;   // [entries][H][V][K]
    float *first;    // [entries][H][V][K]: copies of initial states (those that a later CTA may overwrite)
    float *decay;    // [entries][H]
};

__device__ __forceinline__ int offset_of(const LinearChunkArgs &a, int n) {
    return a.cu_seqlens ? a.cu_seqlens[n] : n * (int)(a.total_tokens / a.n_seqs);
}

// The last sequence n with bound(n) <= at, by the warp's 32 lanes together (bound(0) <= at).
template <typename F>
__device__ __forceinline__ int last_below(int n_seqs, int64_t at, F bound) {
    const int lane = threadIdx.x & 31;
    int lo = 0, span = n_seqs;  // in [lo, lo + span)
    while (span > 1) {
        const int step = (span + 31) / 32, n = lo + lane * step;
        const bool below = n < lo + span && (lane == 0 || bound(n) <= at);
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, below));
        lo += last * step;
        span = min(step, span - last * step);
    }
    return lo;
}

struct Item {
    int n, h, first, rows;  // first token, tokens (0: nothing to compute)
    int64_t slot;           // of the sequence's states, -1: none
    int entry;              // of this segment in the workspace
    bool begins, ends, cut; // the sequence's first and last segment; whether it has several
};

// Segment (and head) `i` of the kernel with outputs.  Sequence n's segments are numbered from
// floor(offset / segment) + n on, which leaves room for all of them whatever the lengths; false: no such segment.
__device__ __forceinline__ bool output_item(const ChunkParams &p, int64_t i, Item &s) {
    const LinearChunkArgs &a = p.a;
    const int64_t rank = i / a.H;
    s.h = (int)(i - rank * a.H);
    s.n = last_below(a.n_seqs, rank, [&](int n) { return (int64_t)(offset_of(a, n) / p.segment) + n; });
    const Span span = span_of(a, s.n);
    const int l = (int)(rank - span.first / p.segment - s.n);
    const int count = max(1, (span.len + p.segment - 1) / p.segment);
    if (span.len < 0 || l < 0 || l >= count) return false;
    s.first = span.first + l * p.segment;
    s.rows = min(p.segment, span.len - l * p.segment);
    s.slot = slot_of(a, s.n);
    s.entry = span.first / p.segment + l;
    s.begins = l == 0, s.ends = l == count - 1, s.cut = count > 1;
    return true;
}

// Segment of entry m, if it is one that others follow in its sequence: the one that token
// (m + 1) segment - 1 lies in, or ends with.
__device__ __forceinline__ bool state_item(const ChunkParams &p, int m, Item &s) {
    const LinearChunkArgs &a = p.a;
    const int64_t x = (int64_t)(m + 1) * p.segment;
    s.n = last_below(a.n_seqs, x, [&](int n) { return (int64_t)offset_of(a, n); });
    const Span span = span_of(a, s.n);
    if (span.len < 0 || x <= span.first) return false;
    const int64_t l = (x - span.first - 1) / p.segment;
    if ((l + 1) * p.segment >= span.len) return false;
    s.first = span.first + (int)l * p.segment;
    s.rows = p.segment;
    s.slot = slot_of(a, s.n);
    s.entry = m;
    s.begins = l == 0, s.ends = false, s.cut = true;
    return s.slot >= 0;
}

// OUTPUT: o and final states, from the states in front of the segments; else a segment's own state.
template <bool OUTPUT>
__global__ void __launch_bounds__(kThreads, 1)
    linear_chunk_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const ChunkParams p) {
    extern __shared__ __align__(1024) uint8_t sm[];
    Shared &sh = *reinterpret_cast<Shared *>(sm + kSmShared);
    volatile int &dead = sh.dead;
    const LinearChunkArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.kq_full[i], 1), mbar_init(&sh.v_full[i], 1);
            mbar_init(&sh.k_empty[i], OUTPUT ? 2 : 1), mbar_init(&sh.q_empty[i], 1), mbar_init(&sh.v_empty[i], OUTPUT ? 2 : 1);
            mbar_init(&sh.gates_full[i], 1), mbar_init(&sh.gates_empty[i], 16);
            mbar_init(&sh.v_ready[i], 128), mbar_init(&sh.kt_full[i], 128), mbar_init(&sh.kt_empty[i], 1);
        }
        mbar_init(&sh.x_full, 1), mbar_init(&sh.p_full, 128), mbar_init(&sh.qs_full, 1), mbar_init(&sh.o_scaled, 256);
        mbar_init(&sh.o_full, 1), mbar_init(&sh.o_empty, 256), mbar_init(&sh.s_full, 256);
        mbar_init(&sh.d_full, 1), mbar_init(&sh.d_empty, 256);
        fence_mbar_init();
        dead = 0;
    }
    if (wid == 1) tmem_alloc(&sh.tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    griddep_wait();
    griddep_launch_dependents();

    // a bounded wait; once one has given up, none waits any more
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!mbar_try_wait(bar, parity) && !dead && !mbar_wait(bar, parity)) dead = 1;
        __syncwarp();
    };
    auto gave_up = [&] { return __any_sync(0xffffffffu, dead); };
    // f(item, chunks) for each of this CTA's items, in the same order by every warp
    auto for_items = [&](auto f) {
        const int64_t items = OUTPUT ? p.items : (int64_t)p.entries * a.H;
        for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
            Item s;
            if (OUTPUT) {
                if (!output_item(p, i, s)) continue;
            } else {
                const int m = (int)(i / a.H);
                s.h = (int)(i - (int64_t)m * a.H);
                if (!state_item(p, m, s)) continue;
            }
            f(s, s.slot < 0 ? 0 : (s.rows + kTok - 1) / kTok);
        }
    };

    if (wid == 0) {
        // ---- TMA
        uint32_t c = 0;
        for_items([&](const Item &s, int chunks) {
            const int hk = s.h / a.group;
            for (int i = 0; i < chunks && !gave_up(); ++i, ++c) {
                const uint32_t st = c & 1, before = ((c >> 1) & 1) ^ 1;
                const int row = s.first + i * kTok;
                wait(&sh.k_empty[st], before);
                if (OUTPUT) wait(&sh.q_empty[st], before);
                if (elect_one()) {
                    mbar_arrive_expect_tx(&sh.kq_full[st], OUTPUT ? 2 * kTile : kTile);
                    for (int b = 0; b < 2; ++b) {
                        tma_load_3d(sm + kSmK + st * kTile + b * kHalf, &map_k, 64 * b, hk, row, &sh.kq_full[st]);
                        if (OUTPUT) tma_load_3d(sm + kSmQ + st * kTile + b * kHalf, &map_q, 64 * b, hk, row, &sh.kq_full[st]);
                    }
                }
                wait(&sh.v_empty[st], before);
                if (elect_one()) {
                    mbar_arrive_expect_tx(&sh.v_full[st], kTile);
                    for (int b = 0; b < 2; ++b)
                        tma_load_3d(sm + kSmV + st * kTile + b * kHalf, &map_v, 64 * b, s.h, row, &sh.v_full[st]);
                }
                __syncwarp();
            }
        });
    } else if (wid == 1 && OUTPUT) {
        // ---- MMA of X and O
        uint32_t c = 0;
        const uint32_t q0 = smem_u32(sm + kSmQ), k0 = smem_u32(sm + kSmK), s0 = smem_u32(sm + kSmS);
        const uint32_t v_lo = (smem_u32(sm + kSmV) >> 4) | ((kHalf >> 4) << 16);
        for_items([&](const Item &s, int chunks) {
            for (int i = 0; i < chunks && !gave_up(); ++i, ++c) {
                const uint32_t st = c & 1, full = (c >> 1) & 1;
                wait(&sh.kq_full[st], full);
                if (c > 0) wait(&sh.o_full, (c - 1) & 1);  // P of the chunk before is read
                tc_fence_after();
                if (elect_one()) {
                    mma_tile<kTok, kTok, kHeadDim, kTok, kTok>(tmem, q0 + st * kTile, k0 + st * kTile, false);
                    mma_commit(&sh.k_empty[st]);
                    mma_commit(&sh.x_full);
                }
                __syncwarp();
                wait(&sh.s_full, c & 1);
                if (c > 0) wait(&sh.o_empty, (c - 1) & 1);
                tc_fence_after();
                if (elect_one()) {
                    mma_tile<kTok, kTok, kHeadDim, kTok, kTok, false, true>(tmem + kTmO, q0 + st * kTile, s0, false);
                    mma_commit(&sh.q_empty[st]);
                    mma_commit(&sh.qs_full);
                }
                __syncwarp();
                wait(&sh.v_ready[st], full);
                wait(&sh.p_full, c & 1);
                wait(&sh.o_scaled, c & 1);
                tc_fence_after();
                if (elect_one()) {
                    constexpr uint32_t idesc = idesc_bf16(kTok, kTok) | (1u << 16);
#pragma unroll
                    for (int j = 0; j < kTok / 16; ++j)
                        mma_bf16_ts(tmem + kTmO, tmem + 8 * j,
                                    ((uint64_t)kDescHi << 32) | (uint64_t)(v_lo + st * (kTile >> 4) + 128 * j), idesc, 1);
                    mma_commit(&sh.v_empty[st]);
                    mma_commit(&sh.o_full);
                }
                __syncwarp();
            }
        });
    } else if (wid == 2) {
        // ---- MMA of D
        uint32_t c = 0, kt = 0;  // chunks and quarters of Kt so far
        const uint32_t v_lo = (smem_u32(sm + kSmV) >> 4) | ((kHalf >> 4) << 16);
        constexpr uint32_t idesc = idesc_bf16(kTok, kTok) | (1u << 16);
        for_items([&](const Item &s, int chunks) {
            for (int i = 0; i < chunks && !gave_up(); ++i, ++c) {
                const uint32_t st = c & 1, full = (c >> 1) & 1;
                const int quarters = (min(kTok, s.rows - i * kTok) + 31) / 32;
                wait(&sh.v_ready[st], full);
                if (c > 0) wait(&sh.d_empty, (c - 1) & 1);
                for (int b = 0; b < quarters; ++b, ++kt) {
                    wait(&sh.kt_full[kt & 1], (kt >> 1) & 1);
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t k_at = tmem + kTmK + (kt & 1) * kTmBuf, v_at = v_lo + st * (kTile >> 4) + 256 * b;
#pragma unroll
                        for (int term = 0; term < 3; ++term)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                mma_bf16_ts(tmem + kTmD, k_at + term * kTmTerm + 8 * j,
                                            ((uint64_t)kDescHi << 32) | (uint64_t)(v_at + 128 * j), idesc, b + term + j > 0);
                        mma_commit(&sh.kt_empty[kt & 1]);
                        if (b == quarters - 1) {
                            mma_commit(&sh.k_empty[st]);
                            mma_commit(&sh.v_empty[st]);
                            mma_commit(&sh.d_full);
                        }
                    }
                    __syncwarp();
                }
            }
        });
    } else if (wid == 3) {
        // ---- decays
        uint32_t c = 0;
        for_items([&](const Item &s, int chunks) {
            for (int i = 0; i < chunks && !gave_up(); ++i, ++c) {
                const uint32_t st = c & 1;
                float g[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int t = i * kTok + 32 * b + lane;
                    g[b] = t < s.rows ? a.g[(int64_t)(s.first + t) * a.g_stride + s.h] * kLog2e : 0.0f;
                }
                wait(&sh.gates_empty[st], ((c >> 1) & 1) ^ 1);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    // (2^-160 is 0; -inf would leave no difference of two sums)
                    const float x = g[b] < -160.0f ? -160.0f : g[b];
                    float up = x, down = x;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const float y = __shfl_up_sync(0xffffffffu, up, o), z = __shfl_down_sync(0xffffffffu, down, o);
                        if (lane >= o) up += y;
                        if (lane + o < 32) down += z;
                    }
                    down = __shfl_down_sync(0xffffffffu, down, 1);
                    sh.lower[st][32 * b + lane] = up;
                    sh.upper[st][32 * b + lane] = lane < 31 ? exp2f(down) : 1.0f;
                    if (lane == 31) sh.block[st][b] = up;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.gates_full[st]);
            }
        });
    } else if (wid >= 4 && wid < 8) {
        // ---- Kt: a thread takes a key channel, 32 tokens at a time
        uint32_t c = 0, kt = 0;
        const int d = tid - 128;
        const uint32_t lanes = (uint32_t)((wid & 3) * 32) << 16;
        const uint32_t at = (d >> 6) * kHalf + (d & 7) * 2, chunk16 = (d & 63) >> 3;
        for_items([&](const Item &s, int chunks) {
            for (int i = 0; i < chunks && !gave_up(); ++i, ++c) {
                const uint32_t st = c & 1, full = (c >> 1) & 1;
                const int rows = min(kTok, s.rows - i * kTok), quarters = (rows + 31) / 32;
                wait(&sh.gates_full[st], full);
                wait(&sh.kq_full[st], full);
                const uint8_t *k = sm + kSmK + st * kTile + at;
                float behind = 0.0f;  // log2 decay of the blocks behind
                for (int b = 1; b < 4; ++b) behind += sh.block[st][b];
                for (int b = 0; b < quarters; ++b, ++kt) {
                    const float f = exp2f(behind);
                    if (b < 3) behind = b == 0 ? sh.block[st][2] + sh.block[st][3] : b == 1 ? sh.block[st][3] : 0.0f;
                    wait(&sh.kt_empty[kt & 1], ((kt >> 1) & 1) ^ 1);
                    tc_fence_after();
                    uint32_t term[3][16];
#pragma unroll
                    for (int m = 0; m < 16; ++m) {
                        float y[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int j = 2 * m + e;
                            const uint32_t u = *(const uint16_t *)(k + (32 * b + j) * 128 + ((chunk16 ^ (j & 7)) << 4));
                            y[e] = __uint_as_float(u << 16) * (f * sh.upper[st][32 * b + j]);
                            if (32 * b + j >= rows) y[e] = 0.0f;
                        }
#pragma unroll
                        for (int t = 0; t < 3; ++t) {
                            const uint32_t w = pack2(y[0], y[1]);
                            term[t][m] = w;
                            y[0] -= __uint_as_float(w << 16), y[1] -= __uint_as_float(w & 0xffff0000u);
                        }
                    }
                    const uint32_t to = tmem + kTmK + (kt & 1) * kTmBuf + lanes;
#pragma unroll
                    for (int t = 0; t < 3; ++t) tmem_st16(to + t * kTmTerm, term[t]);
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(&sh.kt_full[kt & 1]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.gates_empty[st]);
            }
        });
    } else if (wid >= 8 && wid < 12) {
        // ---- check of V; P: a thread takes a row (token i of the chunk)
        uint32_t c = 0;
        const int row = tid - 256, w = wid & 3;
        const uint32_t lanes = (uint32_t)(w * 32) << 16;
        for_items([&](const Item &s, int chunks) {
            for (int i = 0; i < chunks; ++i, ++c) {  // (not left early: its four warps meet at a barrier)
                const uint32_t st = c & 1, full = (c >> 1) & 1;
                const int rows = min(kTok, s.rows - i * kTok);
                wait(&sh.gates_full[st], full);  // (the chunk two before is done with `odd`)
                wait(&sh.v_full[st], full);
                uint8_t *v = sm + kSmV + st * kTile;
                uint32_t ones = 0;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    uint4 *x = (uint4 *)(v + (j >> 3) * kHalf + row * 128 + (((j & 7) ^ (row & 7)) << 4));
                    if (row < rows) ones |= exponent_of_ones(*x);
                    else *x = make_uint4(0, 0, 0, 0);
                }
                if (!named_bar_and(1, 128, ones == 0)) {
                    // this thread's channel: its first such row, and zeros in the place of all of them
                    uint8_t *x = v + (row >> 6) * kHalf + (row & 7) * 2;
                    int first = kTok;
                    for (int j = rows - 1; j >= 0; --j) {
                        uint16_t *u = (uint16_t *)(x + j * 128 + ((((row & 63) >> 3) ^ (j & 7)) << 4));
                        if ((*u & 0x7f80) == 0x7f80) first = j, *u = 0;
                    }
                    sh.odd[st][row] = (uint8_t)first;
                    if (row == 0) sh.any_odd[st] = 1;
                } else if (row == 0) {
                    sh.any_odd[st] = 0;
                }
                fence_async_smem();
                mbar_arrive(&sh.v_ready[st]);
                if (OUTPUT) {
                    const float own = sh.lower[st][row];
                    wait(&sh.x_full, c & 1);
                    tc_fence_after();
#pragma unroll 1
                    for (int b = 0; b < 4; ++b) {
                        uint32_t u[16];
                        if (b < w) {
                            float x[32];
                            tmem_ld32(tmem + lanes + 32 * b, x);
                            float before = own;  // log2 decay from the end of block b to this row
                            for (int j = b + 1; j < w; ++j) before += sh.block[st][j];
                            const float f = exp2f(before);
                            tmem_ld_wait_for(x);
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                const float4 y = *(const float4 *)&sh.upper[st][32 * b + j];
                                u[j / 2] = pack2(x[j] * (f * y.x), x[j + 1] * (f * y.y));
                                u[j / 2 + 1] = pack2(x[j + 2] * (f * y.z), x[j + 3] * (f * y.w));
                            }
                        } else if (b == w) {
                            float x[32];
                            tmem_ld32(tmem + lanes + 32 * b, x);
                            tmem_ld_wait_for(x);
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                const float4 y = *(const float4 *)&sh.lower[st][32 * b + j];
                                x[j] = j <= lane ? x[j] * exp2_sfu(own - y.x) : 0.0f;
                                x[j + 1] = j + 1 <= lane ? x[j + 1] * exp2_sfu(own - y.y) : 0.0f;
                                x[j + 2] = j + 2 <= lane ? x[j + 2] * exp2_sfu(own - y.z) : 0.0f;
                                x[j + 3] = j + 3 <= lane ? x[j + 3] * exp2_sfu(own - y.w) : 0.0f;
                                u[j / 2] = pack2(x[j], x[j + 1]);
                                u[j / 2 + 1] = pack2(x[j + 2], x[j + 3]);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) u[j] = 0;
                        }
                        tmem_st16(tmem + lanes + 16 * b, u);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(&sh.p_full);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.gates_empty[st]);
            }
        });
    } else if (wid >= 12) {
        // ---- the state (a thread takes a key channel) and the outputs (a token), 64 value channels each
        uint32_t c = 0;
        const int half = (wid - 12) >> 2, w = wid & 3, row = 32 * w + lane;
        const uint32_t lanes = (uint32_t)(w * 32) << 16;
        const uint32_t to = tmem + kTmO + 64 * half + lanes, td = tmem + kTmD + 64 * half + lanes;
        for_items([&](const Item &s, int chunks) {
            const int64_t place = (int64_t)(64 * half) * kHeadDim + row;  // of this thread's part of a state
            if (s.slot < 0) {
                for (int t = row; t < s.rows; t += kTok) {
                    uint32_t *o = (uint32_t *)((__nv_bfloat16 *)a.o + ((int64_t)(s.first + t) * a.H + s.h) * kHeadDim + 64 * half);
                    for (int j = 0; j < 32; ++j) o[j] = 0x7fc07fc0u;
                }
                return;
            }
            float S[64];
            const float *init = nullptr;
            if (OUTPUT) {
                const int64_t in_pool = (s.slot * a.H + s.h) * (int64_t)kState;
                if (!s.begins) init = p.states + ((int64_t)(s.entry - 1) * a.H + s.h) * kState;
                else if (a.initial_state) init = s.cut ? p.first + ((int64_t)s.entry * a.H + s.h) * kState : a.initial_state + in_pool;
            }
            if (init) {
#pragma unroll
                for (int e = 0; e < 64; ++e) S[e] = init[place + e * kHeadDim];
            } else {
#pragma unroll
                for (int e = 0; e < 64; ++e) S[e] = 0.0f;
            }
            float log_decay = 0.0f;
            auto publish = [&] {  // the copy of S that the next chunk's O is taken from
                uint8_t *to_s = sm + kSmS + half * kHalf + row * 128;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *(uint4 *)(to_s + ((j ^ (row & 7)) << 4)) =
                        make_uint4(pack2(S[8 * j], S[8 * j + 1]), pack2(S[8 * j + 2], S[8 * j + 3]),
                                   pack2(S[8 * j + 4], S[8 * j + 5]), pack2(S[8 * j + 6], S[8 * j + 7]));
                fence_async_smem();
                mbar_arrive(&sh.s_full);
            };
            if (OUTPUT && chunks > 0) publish();
            for (int i = 0; i < chunks; ++i, ++c) {
                const uint32_t st = c & 1, full = (c >> 1) & 1;
                const int rows = min(kTok, s.rows - i * kTok);
                wait(&sh.gates_full[st], full);
                wait(&sh.v_ready[st], full);
                float whole = 0.0f, upto = sh.lower[st][row];
                for (int b = 0; b < 4; ++b) {
                    if (b < w) upto += sh.block[st][b];
                    whole += sh.block[st][b];
                }
                if (OUTPUT) {
                    const float f = exp2f(upto);
                    wait(&sh.qs_full, c & 1);
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float x[16];
                        tmem_ld16(to + 16 * k, x);
                        tmem_ld_wait_for(x);
                        uint32_t u[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(x[j] * f);
                        tmem_st16(to + 16 * k, u);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(&sh.o_scaled);
                } else {
                    log_decay += whole;
                }
                const float decay = exp2f(whole);
                wait(&sh.d_full, c & 1);
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float x[16];
                    tmem_ld16(td + 16 * k, x);
                    tmem_ld_wait_for(x);
#pragma unroll
                    for (int j = 0; j < 16; ++j) S[16 * k + j] = fmaf(decay, S[16 * k + j], x[j]);
                }
                tc_fence_before();
                mbar_arrive(&sh.d_empty);
                const bool odd = sh.any_odd[st];
                if (odd) {
#pragma unroll
                    for (int e = 0; e < 64; ++e)
                        if (sh.odd[st][64 * half + e] < kTok) S[e] = NAN;
                }
                if (OUTPUT) {
                    if (i + 1 < chunks) publish();
                    wait(&sh.o_full, c & 1);
                    tc_fence_after();
                    const bool lost = gave_up();
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float x[32];
                        tmem_ld32(to + 32 * k, x);
                        tmem_ld_wait_for(x);
                        if (k == 1) {
                            tc_fence_before();
                            mbar_arrive(&sh.o_empty);
                        }
                        uint32_t u[4][4];
#pragma unroll
                        for (int j = 0; j < 16; ++j) u[j >> 2][j & 3] = pack2(x[2 * j] * a.scale, x[2 * j + 1] * a.scale);
                        if (odd) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (sh.odd[st][64 * half + 32 * k + j] <= row) u[j >> 3][(j >> 1) & 3] |= j & 1 ? 0x7fff0000u : 0x7fffu;
                        }
                        if (lost) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) u[j >> 2][j & 3] = 0x7fff7fffu;
                        }
                        // four lanes exchange their units of 16 bytes, so that a store writes 64 bytes of eight rows
#pragma unroll
                        for (int o = 1; o < 4; o <<= 1) {
                            const bool up = lane & o;
#pragma unroll
                            for (int m = 0; m < 4; ++m)
                                if (!(m & o))
#pragma unroll
                                    for (int j = 0; j < 4; ++j) {
                                        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? u[m][j] : u[m | o][j], o);
                                        if (up) u[m][j] = got; else u[m | o][j] = got;
                                    }
                        }
                        const int t0 = 32 * w + (lane & ~3);
                        __nv_bfloat16 *o = (__nv_bfloat16 *)a.o + ((int64_t)(s.first + i * kTok + t0) * a.H + s.h) * kHeadDim +
                                           64 * half + 32 * k + 8 * (lane & 3);
#pragma unroll
                        for (int m = 0; m < 4; ++m)
                            if (t0 + m < rows)
                                *(uint4 *)(o + (int64_t)m * a.H * kHeadDim) = make_uint4(u[m][0], u[m][1], u[m][2], u[m][3]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.gates_empty[st]);
            }
            if (gave_up()) {
#pragma unroll
                for (int e = 0; e < 64; ++e) S[e] = NAN;
            }
            float *out = nullptr;
            if (!OUTPUT) out = p.states + ((int64_t)s.entry * a.H + s.h) * kState;
            else if (s.ends && a.final_state) out = a.final_state + (s.slot * a.H + s.h) * (int64_t)kState;
            if (out) {
#pragma unroll
                for (int e = 0; e < 64; ++e) out[place + e * kHeadDim] = S[e];
            }
            if (!OUTPUT && half == 0 && row == 0) p.decay[(int64_t)s.entry * a.H + s.h] = exp2f(log_decay);
        });
    }
    tc_fence_before();
    __syncthreads();
    if (dead) {  // copies still in flight land before the memory is given up
        const long long t0 = clock64();
        while (clock64() - t0 < 100000000LL) __nanosleep(1000);
    }
    if (wid == 1) tmem_dealloc(tmem, 512);
}

// The states in front of the segments of each sequence that is cut, in place of the segments' own: entry l gets
// that in front of segment l + 1.  A sequence's initial state is copied, because its last segment may
// overwrite it while the first one still reads.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) linear_join_kernel(const ChunkParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const LinearChunkArgs &a = p.a;
    const int h = blockIdx.y;
    Item s;
    if (!state_item(p, blockIdx.x, s) || !s.begins) return;
    const Span span = span_of(a, s.n);
    const int count = (span.len - 1) / p.segment;  // entries
    const int64_t at = (int64_t)blockIdx.z * kJoinThreads + threadIdx.x;
    const int64_t step = (int64_t)a.H * kState;
    float x = 0.0f;
    const int64_t own = ((int64_t)s.entry * a.H + h) * kState + at;
    if (a.initial_state) {
        x = a.initial_state[(s.slot * a.H + h) * (int64_t)kState + at];
        p.first[own] = x;
    }
    float *state = p.states + own;
    const float *decay = p.decay + (int64_t)s.entry * a.H + h;
    constexpr int kAhead = 8;
    for (int l = 0; l < count; l += kAhead) {
        float y[kAhead], d[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (l + j < count) y[j] = state[(l + j) * step], d[j] = decay[(int64_t)(l + j) * a.H];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (l + j < count) state[(l + j) * step] = x = fmaf(d[j], x, y[j]);
    }
}

// Tokens of a segment: so many that the segments of all heads are about as many as SMs.
inline int64_t segment_of(int64_t total_tokens, int H) {
    const int64_t chunks = (total_tokens + kTok - 1) / kTok, each = std::max<int64_t>(1, sm_count() / H);
    return kTok * std::max<int64_t>(1, (chunks + each - 1) / each);
}
inline int64_t entries_of(int64_t total_tokens, int H) {
    return total_tokens > 0 ? (total_tokens - 1) / segment_of(total_tokens, H) : 0;
}

}  // namespace

size_t linear_chunk_workspace_bytes(int64_t total_tokens, int n_seqs, int H) {
    const int64_t entries = entries_of(total_tokens, H) * H;
    return (size_t)entries * 2 * kState * sizeof(float) + align_up((size_t)entries * sizeof(float), 256);
}

cudaError_t launch_linear_chunk_tc(const LinearChunkArgs &a, cudaStream_t stream) {
    const int64_t T = a.total_tokens, rows = std::max<int64_t>(T, 1);
    const int hk = a.H / a.group;
    CUtensorMap map_q, map_k, map_v;
    // (without a token there is no copy, and maybe no pointer)
    const void *none = a.final_state ? (const void *)a.final_state : a.initial_state;
    if (T == 0 && !none) return cudaSuccess;
    if (!encode_heads64(&map_q, T ? a.q : none, kHeadDim, hk, rows, a.q_stride, kTok) ||
        !encode_heads64(&map_k, T ? a.k : none, kHeadDim, hk, rows, a.k_stride, kTok) ||
        !encode_heads64(&map_v, T ? a.v : none, kHeadDim, a.H, rows, a.v_stride, kTok))
        return cudaErrorUnknown;
    ChunkParams p{a};
    const int64_t segment = segment_of(T, a.H), entries = entries_of(T, a.H);
    p.segment = (int)segment;
    p.entries = (int)entries;
    p.items = (T / segment + a.n_seqs) * a.H;
    p.states = (float *)a.workspace;
    p.first = p.states + entries * a.H * kState;
    p.decay = p.first + entries * a.H * kState;
    auto launch = [&](auto kernel, int64_t items) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
        return e != cudaSuccess ? e
                                : launch_dependent(kernel, dim3((unsigned)std::min<int64_t>(items, sm_count())), dim3(kThreads),
                                                   kSmemBytes, stream, map_q, map_k, map_v, p);
    };
    if (entries > 0) {
        cudaError_t e = launch(linear_chunk_kernel<false>, entries * a.H);
        if (e == cudaSuccess)
            e = launch_dependent(linear_join_kernel, dim3((unsigned)entries, (unsigned)a.H, kState / kJoinThreads),
                                 dim3(kJoinThreads), 0, stream, p);
        if (e != cudaSuccess) return e;
    }
    const cudaError_t e = launch(linear_chunk_kernel<true>, p.items);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kda
