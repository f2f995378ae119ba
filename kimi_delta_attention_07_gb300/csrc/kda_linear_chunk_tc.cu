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
// S = e^{G_127} S + D, which the tensor core could not scale.  e^{G_127}, and a segment's decay, is the sum of two
// floats (decay_of_log2): applied chunk by chunk, one near one would add up its rounding (131072 tokens of 2^-16 each:
// states off by 1.8e-6, now by the 3e-7 of their sums).
//
// What is rounded: P and the copy of S that O is taken from, to bf16 (as o itself is, so that o's
// rounding variance doubles; both are read once and kept nowhere).  In the chunk that a sequence begins with, P
// has a second term: a row of a few tokens may hang on one of its elements (error of o of 4 tokens: 1.4 times o's own
// rounding without, up to 2 for a row; 1.0 with).  It is a matter of the sequence alone, not of what else is in the call.  4096
// sequences of 40 tokens take 292 us with, 267 without, 131072 tokens 300 and 298; in every chunk, 331, for an
// error of 1.2 instead of 1.4 times o's rounding.  Kt enters the states, which
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
// the third (kda_linear_segments.cuh).
//
// Masked places: rows of a tile past the sequence's end are emptied (V) or taken as 0 (K).  A
// value that is not finite would reach rows before it as 0 times it: V is looked through,
// such values become 0 and their channel NaN from their row on, in o and in S.
//
// What bounds a chunk: not its products (half of its 6300 clocks; without them it took a tenth less) but
// the chain of instructions of a warp, each some seven clocks behind the last.  So the work is spread over
// as many warps as there are registers for (five groups of four with 128 registers: 9300 clocks).  With outputs, eight warps look through V and make Kt and
// run ahead, sixteen make P and hold the state, 32 value channels each, and take a chunk's outputs while the
// next one's scores are computed; without outputs, sixteen warps make a quarter of Kt each and update a
// quarter of the state while the next chunk's D runs.
//
// What a chunk waits for is ordered so that little waits: its outputs, then P while D's last quarters are made, the state
// while Q . S is computed (in front of P 313 us for 131072 tokens, behind the scaling of O 327, here 300), the copy of S
// while P . V is.
//
// 131072 tokens of 8 heads: 302 to 314 us, of which the segments' states take 105 (4.9 TB/s), the join 6 and the
// outputs 193 (5.5 TB/s); 4096 tokens of 32 heads: 64 us; 8 sequences of 333 to 4001 tokens, 32 heads, uncut: 133 us.
// (Decays as sums of two floats and the second terms of P are 3 to 4 % of that.)
//
// Warps: 0 TMA, 1 MMA of X and O, 2 MMA of D, 3 decays, 4..11 check of V and Kt, 12..27 P, the state
// and the outputs; without outputs 4..19 all of it.
#include <algorithm>
#include <type_traits>

#include "kda_attn.cuh"
#include "kda_linear_segments.cuh"

namespace kda {

using namespace tc;

namespace {

constexpr int kTok = 128;  // tokens of a chunk
constexpr uint32_t kTile = 32768;        // 128 tokens x 128 channels: two blocks of 64 channels
constexpr uint32_t kHalf = kTile / 2;

// shared memory (from a 1024-byte boundary): two stages of K, V, Q and the copy of S; without outputs three of K, V
constexpr uint32_t kSmQ = 4 * kTile, kSmS = 6 * kTile, kSmShared = 7 * kTile;
__device__ __forceinline__ constexpr uint32_t tile_k(uint32_t st) { return 2 * st * kTile; }
__device__ __forceinline__ constexpr uint32_t tile_v(uint32_t st) { return (2 * st + 1) * kTile; }

// TMEM columns: X and P (16 tokens of P over the first 8 columns of their scores, its second term over the next 8), O, D, buffers of 32 tokens of Kt in three
// terms of 16 columns.  Without outputs eight buffers, over X and O as well.
constexpr uint32_t kTmO = 128, kTmD = 384, kTmK = 256, kTmTerm = 16, kTmBuf = 48;

struct Shared {
    uint64_t k_full[3], v_full[3], k_empty[3], v_empty[3], v_ready[3], q_full[2], q_empty[2], gates_full[2], gates_empty[2], kt_full[2], kt_empty[2],
        x_full, qs_full, pv_ready, o_full, o_empty, d_full, d_empty;
    alignas(16) float lower[2][kTok];  // log2 decay of a token's block up to and with it
    float upper[2][kTok];              // decay of a token's block behind it
    float block[2][4];                 // log2 decay of each block
    float whole[4];                    // of a chunk; for four chunks, because they are read behind the arrival at gates_empty
    int early[4];                      // a sequence begins with the chunk: P has two terms
    float2 decay[4];                   // 2 to that, as the sum of two floats
    uint8_t odd[4][kTok];              // a value channel's first row that is not finite (kTok: none), if any_odd
    volatile int any_odd[4][4], dead;  // of a group of channels
    uint32_t tmem_base;
};
constexpr uint32_t kSmemBytes = kSmShared + sizeof(Shared);
static_assert(kSmemBytes <= 232448, "shared memory");

// Four 8 x 8 matrices of bf16, transposed: matrix m's rows are the 16 bytes that lanes 8 m .. 8 m + 7 point at;
// r[m] holds the elements (row 2 (lane % 4), 2 (lane % 4) + 1; column lane / 4).
__device__ __forceinline__ void ldmatrix4_trans(uint32_t *r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 16 columns of 16 TMEM lanes: u[2 j + h] goes to lane 8 h + lane / 4, column 4 j + lane % 4.
__device__ __forceinline__ void tmem_st_16x16(uint32_t taddr, const uint32_t *u) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(u[0]), "r"(u[1]),
                 "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}
// 3-D tile, shared -> global (64 channels of 128 tokens of a head), in the issuing thread's bulk group.
__device__ __forceinline__ void tma_store_3d(const void *tmap, const void *src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(tmap),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
// The larger magnitude of two pairs of bf16, NaN if either is.
__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// OUTPUT: o and final states, from the states in front of the segments; else a segment's own state.
template <bool OUTPUT, Source SOURCE>
__global__ void __launch_bounds__(OUTPUT ? 896 : 640, 1)
    linear_chunk_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
                        const ChunkParams p) {
    constexpr uint32_t kStages = OUTPUT ? 2 : 3;
    extern __shared__ __align__(1024) uint8_t sm[];
    Shared &sh = *reinterpret_cast<Shared *>(sm + kSmShared);
    volatile int &dead = sh.dead;
    const LinearChunkArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) {
            mbar_init(&sh.k_full[i], 1), mbar_init(&sh.v_full[i], 1), mbar_init(&sh.k_empty[i], OUTPUT ? 9 : 16);
            mbar_init(&sh.v_empty[i], OUTPUT ? 2 : 1), mbar_init(&sh.v_ready[i], OUTPUT ? 8 : 16);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.q_full[i], 1), mbar_init(&sh.q_empty[i], 16), mbar_init(&sh.gates_full[i], 1), mbar_init(&sh.gates_empty[i], OUTPUT ? 24 : 16);
            mbar_init(&sh.kt_full[i], OUTPUT ? 4 : 16), mbar_init(&sh.kt_empty[i], 1);
        }
        mbar_init(&sh.x_full, 1), mbar_init(&sh.qs_full, 1), mbar_init(&sh.pv_ready, 16);
        mbar_init(&sh.o_full, 1), mbar_init(&sh.o_empty, 16), mbar_init(&sh.d_full, 1), mbar_init(&sh.d_empty, 16);
        fence_mbar_init();
        dead = 0;
    }
    if (wid == 1) tmem_alloc(&sh.tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    // Behind the join only the states in front of the segments are awaited (by the warps that read them, and
    // write what it reads): the join itself began when all before it was done.
    if (!OUTPUT || !p.joined || wid >= 12) griddep_wait();
    griddep_launch_dependents();

    // a bounded wait; once one has given up, none waits any more
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!mbar_try_wait(bar, parity) && !dead && !mbar_wait(bar, parity)) dead = 1;
        __syncwarp();
    };
    // one arrival a warp
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    auto gave_up = [&] { return __any_sync(0xffffffffu, dead); };
    // f(segment and head, chunks, terms) for each of this CTA's, in the same order by every warp
    auto for_items = [&](auto f) {
        for_segments<OUTPUT, SOURCE>(p, blockIdx.x, gridDim.x, [&](const Item &s) {
            // a segment whose states serve o alone does without the third term
            f(s, s.w & kNoSlot ? 0 : (s.y + kTok - 1) / kTok, OUTPUT && (s.w & (kCut | kEnds)) == kCut ? 2 : 3);
        });
    };

    if (wid == 0) {
        // ---- TMA
        uint32_t c = 0;
        // With outputs, a chunk's o is left in the place of its Q, whose products are done, and leaves from there
        // before the next Q comes (16-byte stores of a row a thread took 2400 clocks a chunk; in the place of V, which
        // is wanted earlier, 131072 tokens of 8 heads take 343 instead of 325 us).  The last two chunks: first
        // token, head; -1: rows fewer than the tile's, which the other warps have stored.
        int token0 = -1, token1 = -1, head0 = 0, head1 = 0;
        auto store = [&](uint32_t n) {  // o of chunk n
            const uint32_t st = n % kStages;
            wait(&sh.q_empty[st], (n / kStages) & 1);
            const int token = n & 1 ? token1 : token0, head = n & 1 ? head1 : head0;
            if (token >= 0 && !gave_up() && elect_one()) {
                tma_store_3d(&map_o, sm + kSmQ + st * kTile, 0, head, token);
                tma_store_3d(&map_o, sm + kSmQ + st * kTile + kHalf, 64, head, token);
                bulk_commit();
                bulk_wait_read();
            }
            __syncwarp();
        };
        for_items([&](const Item &s, int chunks, int terms) {
            const int h = head_of(s), hk = (uint32_t)h / (uint32_t)a.group;
            for (int i = 0; i < chunks && !gave_up(); ++i, ++c) {
                const uint32_t st = c % kStages, before = ((c / kStages) & 1) ^ 1;
                const int row = s.x + i * kTok;
                auto load = [&](uint32_t at, const CUtensorMap *map, int head, uint64_t *bar) {
                    tma_load_3d(sm + at, map, 0, head, row, bar);
                    tma_load_3d(sm + at + kHalf, map, 64, head, row, bar);
                };
                wait(&sh.k_empty[st], before);
                if (elect_one()) {
                    mbar_arrive_expect_tx(&sh.k_full[st], kTile);
                    load(tile_k(st), &map_k, hk, &sh.k_full[st]);
                }
                wait(&sh.v_empty[st], before);
                if (elect_one()) {
                    mbar_arrive_expect_tx(&sh.v_full[st], kTile);
                    load(tile_v(st), &map_v, h, &sh.v_full[st]);
                }
                if (OUTPUT) {
                    if (c >= kStages) store(c - kStages);
                    const int token = s.y - i * kTok >= kTok ? row : -1;
                    if (c & 1) token1 = token, head1 = h;
                    else token0 = token, head0 = h;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&sh.q_full[st], kTile);
                        load(kSmQ + st * kTile, &map_q, hk, &sh.q_full[st]);
                    }
                }
                __syncwarp();
            }
        });
        if (OUTPUT) {
            for (uint32_t n = c > kStages ? c - kStages : 0; n < c; ++n) store(n);
            if (elect_one()) bulk_wait_all();
            __syncwarp();
        }
    } else if (wid == 1 && OUTPUT) {
        // ---- MMA of X and O
        uint32_t c = 0;
        const uint32_t q0 = smem_u32(sm + kSmQ), k0 = smem_u32(sm), s0 = smem_u32(sm + kSmS);
        const uint32_t v_lo = (smem_u32(sm) >> 4) | ((kHalf >> 4) << 16);
        for_items([&](const Item &s, int chunks, int terms) {
            for (int i = 0; i < chunks && !gave_up(); ++i, ++c) {
                const uint32_t st = c & 1, full = (c >> 1) & 1;
                wait(&sh.k_full[st], full);
                wait(&sh.q_full[st], full);
                if (c > 0) wait(&sh.o_full, (c - 1) & 1);  // P of the chunk before is read
                tc_fence_after();
                if (elect_one()) {
                    mma_tile<kTok, kTok, kHeadDim, kTok, kTok>(tmem, q0 + st * kTile, k0 + tile_k(st), false);
                    mma_commit(&sh.k_empty[st]);
                    mma_commit(&sh.x_full);
                }
                __syncwarp();
                wait(&sh.o_empty, c & 1);  // O is taken, and the copy of S is there
                tc_fence_after();
                if (elect_one()) {
                    mma_tile<kTok, kTok, kHeadDim, kTok, kTok, false, true>(tmem + kTmO, q0 + st * kTile, s0, false);
                    mma_commit(&sh.qs_full);
                }
                __syncwarp();
                wait(&sh.pv_ready, c & 1);  // (behind v_ready)
                tc_fence_after();
                if (elect_one()) {
                    constexpr uint32_t idesc = idesc_bf16(kTok, kTok) | (1u << 16);
                    const uint64_t v_at = ((uint64_t)kDescHi << 32) | (uint64_t)(v_lo + (tile_v(st) >> 4));
#pragma unroll
                    for (int j = 0; j < kTok / 16; ++j) mma_bf16_ts(tmem + kTmO, tmem + 16 * j, v_at + 128 * j, idesc, 1);
                    if (i == 0 && (s.w & kBegins)) {  // the second terms, of the tokens that are there
                        const int steps = (min(kTok, s.y) + 15) / 16;
#pragma unroll 1
                        for (int j = 0; j < steps; ++j) mma_bf16_ts(tmem + kTmO, tmem + 16 * j + 8, v_at + 128 * j, idesc, 1);
                    }
                    mma_commit(&sh.v_empty[st]);
                    mma_commit(&sh.o_full);
                }
                __syncwarp();
            }
        });
    } else if (wid == 2) {
        // ---- MMA of D
        // Kt comes in quarters through two buffers, or (without outputs) in whole chunks, likewise
        uint32_t c = 0, kt = 0;
        const uint32_t v_lo = (smem_u32(sm) >> 4) | ((kHalf >> 4) << 16);
        constexpr int kParts = OUTPUT ? 4 : 1;
        for_items([&](const Item &s, int chunks, int terms) {
            for (int i = 0; i < chunks && !gave_up(); ++i, ++c) {
                const uint32_t st = c % kStages;
                const int steps = (min(kTok, s.y - i * kTok) + 15) / 16;
                wait(&sh.v_ready[st], (c / kStages) & 1);
                if (c > 0) wait(&sh.d_empty, (c - 1) & 1);
#pragma unroll 1
                for (int b = 0; b < kParts; ++b, ++kt) {
                    wait(&sh.kt_full[kt & 1], (kt >> 1) & 1);
                    tc_fence_after();
                    if (elect_one()) {
                        constexpr uint32_t idesc = idesc_bf16(kTok, kTok) | (1u << 16);
                        constexpr int kSteps = 8 / kParts;
                        const uint32_t k_at = tmem + (OUTPUT ? kTmK : 0) + (kt & 1) * (kTmBuf * (4 / kParts));
                        const uint32_t v_at = v_lo + (tile_v(st) >> 4) + 256 * b;
#pragma unroll 1
                        for (int j = 0; j < kSteps && kSteps * b + j < steps; ++j)
#pragma unroll 1
                            for (int t = 0; t < terms; ++t)
                                mma_bf16_ts(tmem + kTmD, k_at + (j >> 1) * kTmBuf + t * kTmTerm + 8 * (j & 1),
                                            ((uint64_t)kDescHi << 32) | (uint64_t)(v_at + 128 * j), idesc, b + t + j > 0);
                        mma_commit(&sh.kt_empty[kt & 1]);
                        if (b == kParts - 1) {
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
        for_items([&](const Item &s, int chunks, int terms) {
            for (int i = 0; i < chunks && !gave_up(); ++i, ++c) {
                const uint32_t st = c & 1;
                float g[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int t = i * kTok + 32 * b + lane;
                    g[b] = t < s.y ? a.g[(int64_t)(s.x + t) * a.g_stride + head_of(s)] * kLog2e : 0.0f;
                }
                float lower[4], upper[4];
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
                    lower[b] = up;
                    upper[b] = lane < 31 ? exp2f(down) : 1.0f;
                }
                wait(&sh.gates_empty[st], ((c >> 1) & 1) ^ 1);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    sh.lower[st][32 * b + lane] = lower[b];
                    sh.upper[st][32 * b + lane] = upper[b];
                    if (lane == 31) sh.block[st][b] = lower[b];
                }
                if (lane == 31) {
                    sh.early[c & 3] = i == 0 && (s.w & kBegins);
                    const float whole = lower[0] + lower[1] + lower[2] + lower[3];
                    sh.whole[c & 3] = whole, sh.decay[c & 3] = decay_of_log2(whole);
                }
                arrive(&sh.gates_full[st]);
            }
        });
    } else if (wid >= 4) {
        constexpr int kGroups = OUTPUT ? 2 : 4;  // of four warps that look through V and make Kt
        constexpr int kWidth = kHeadDim / kGroups;
        const bool maker = !OUTPUT || wid < 12;
        const int g = (wid >> 2) - 1, u = OUTPUT ? g - 2 : g, w = wid & 3, row = 32 * w + lane;
        const uint32_t lanes = (uint32_t)(w * 32) << 16;
        // Kt: this lane's address of a matrix row (matrix 2 j + h: tokens 8 j .., channels 8 h .. of 16)
        const int token = 8 * (lane >> 4) + (lane & 7), channel = 32 * w + 8 * ((lane >> 3) & 1);
        const uint32_t k_at = smem_u32(sm) + (channel >> 6) * kHalf + token * 128;
        const uint32_t unit = (channel & 63) >> 3, turn = token & 7;
        uint32_t kt = 0;

        // V: kWidth channels of this thread's row; rows past the sequence's end become zeros, as those of K
        auto check = [&](uint32_t c, int rows) {
            const uint32_t st = c % kStages, full = (c / kStages) & 1;
            wait(&sh.k_full[st], full);
            wait(&sh.v_full[st], full);
            uint8_t *v = sm + tile_v(st) + (g * kWidth >> 6) * kHalf + row * 128;
            const int first16 = (g * kWidth & 63) >> 3;
            if (__builtin_expect(rows < kTok, 0)) {
                if (row >= rows)
                    for (int j = 0; j < kWidth / 8; ++j) {
                        const int at = ((first16 + j) ^ (row & 7)) << 4;
                        *(uint4 *)(v + at) = *(uint4 *)(v - kTile + at) = make_uint4(0, 0, 0, 0);
                    }
                __syncwarp();
                named_bar_sync(5, 128 * kGroups);
            }
            uint32_t most = 0;
#pragma unroll
            for (int j = 0; j < kWidth / 8; ++j) {
                const uint4 x = *(const uint4 *)(v + (((first16 + j) ^ (row & 7)) << 4));
                most = abs_max2(abs_max2(abs_max2(abs_max2(most, x.x), x.y), x.z), x.w);
            }
            if (row == 0) sh.any_odd[g][c & 3] = 0;
            if (__builtin_expect(!named_bar_and(1 + g, 128, exponent_of_ones(make_uint4(most, 0, 0, 0)) == 0), 0)) {
                // a channel's first such row, and zeros in the place of all of them
                if (row < kWidth) {
                    int first = kTok;
                    for (int j = rows - 1; j >= 0; --j) {
                        const int ch = 8 * first16 + row;
                        uint16_t *x = (uint16_t *)(v + (j - row) * 128 + (((ch >> 3) ^ (j & 7)) << 4) + (ch & 7) * 2);
                        if ((*x & 0x7f80) == 0x7f80) first = j, *x = 0;
                    }
                    sh.odd[c & 3][g * kWidth + row] = (uint8_t)first;
                }
                if (row == 0) sh.any_odd[g][c & 3] = 1;
                __syncwarp();
                named_bar_sync(1 + g, 128);
            }
            fence_async_smem();
            wait(&sh.gates_full[c & 1], (c >> 1) & 1);  // (so that who waits for v_ready has the decays, too)
            arrive(&sh.v_ready[st]);
        };
        // Kt: 32 tokens, block b, into the buffer at tk
        auto make_kt = [&](uint32_t c, int b, int terms, uint32_t tk, uint64_t *empty, uint32_t parity) {
            float behind = 0.0f;  // log2 decay of the blocks behind
            for (int j = b + 1; j < 4; ++j) behind += sh.block[c & 1][j];
            const float f = exp2f(behind);
            F2 weight[4];  // of tokens 8 j + 2 (lane % 4), and the one after
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = *(const float2 *)&sh.upper[c & 1][32 * b + 8 * j + 2 * (lane & 3)];
                weight[j] = f2(x.x * f, x.y * f);
            }
#pragma unroll
            for (int l = 0; l < 2; ++l) {  // 16 channels
                uint32_t raw[8], term[8];
                const uint32_t from = k_at + tile_k(c % kStages) + 32 * b * 128 + (((unit + 2 * l) ^ turn) << 4);
                ldmatrix4_trans(raw, from);
                ldmatrix4_trans(raw + 4, from + 16 * 128);
                F2 y[8];
#pragma unroll
                for (int m = 0; m < 8; ++m) {  // m = 2 j + h
                    y[m] = mul2(wide(raw[m]), weight[m >> 1]);
                    term[m] = narrow(y[m]);
                }
                if (l == 0) {
                    wait(empty, parity);
                    tc_fence_after();
                }
#pragma unroll
                for (int t = 0; t < 3; ++t) {
                    if (t == 2 && terms < 3) break;
                    tmem_st_16x16(tk + ((uint32_t)(16 * l) << 16) + t * kTmTerm, term);
                    if (t < 2) {
#pragma unroll
                        for (int m = 0; m < 8; ++m) {
                            y[m] = fma2(wide(term[m]), f2(-1.0f, -1.0f), y[m]);
                            term[m] = narrow(y[m]);
                        }
                    }
                }
            }
            tmem_st_wait();
            tc_fence_before();
        };
        if (maker && OUTPUT) {
            // ---- check of V, Kt
            uint32_t c = 0;
            for_items([&](const Item &s, int chunks, int terms) {
                for (int i = 0; i < chunks; ++i, ++c) {  // (not left early: these warps meet at barriers)
                    check(c, min(kTok, s.y - i * kTok));
#pragma unroll 1
                    for (int e = 0; e < 2; ++e, ++kt) {
                        if (32 * (g + 2 * e) < s.y - i * kTok) {
                            make_kt(c, g + 2 * e, terms, tmem + kTmK + g * kTmBuf + lanes, &sh.kt_empty[g], (kt & 1) ^ 1);
                        } else {  // no token: the quarter's products are left out, too
                            wait(&sh.kt_empty[g], (kt & 1) ^ 1);
                        }
                        arrive(&sh.kt_full[g]);
                    }
                    arrive(&sh.k_empty[c % kStages]);
                    arrive(&sh.gates_empty[c & 1]);
                }
            });
        } else if (!OUTPUT) {
            // ---- check of V, Kt, the state (of the chunk before): a thread stands for a key channel of it
            uint32_t c = 0;
            const uint32_t td = tmem + kTmD + 32 * u + lanes;
            for_items([&](const Item &s, int chunks, int terms) {
                F2 S[16];  // value channels 32 u + 2 e, and the one after
#pragma unroll
                for (int e = 0; e < 16; ++e) S[e] = 0;
                float log_decay = 0.0f;
                auto update = [&](uint32_t n) {  // by chunk n
                    wait(&sh.d_full, n & 1);
                    tc_fence_after();
                    const float2 decay = sh.decay[n & 3];
                    log_decay += sh.whole[n & 3];
                    float x[32];
                    tmem_ld32(td, x);
                    tmem_ld_wait_for(x);
                    tc_fence_before();
                    arrive(&sh.d_empty);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        S[e] = fma2(f2(decay.x, decay.x), S[e], fma2(f2(decay.y, decay.y), S[e], f2(x[2 * e], x[2 * e + 1])));
                    if (__builtin_expect(sh.any_odd[u][n & 3], 0)) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const uint8_t *from = &sh.odd[n & 3][32 * u + 2 * e];
                            float lo, hi;
                            unf2(S[e], lo, hi);
                            S[e] = f2(from[0] < kTok ? NAN : lo, from[1] < kTok ? NAN : hi);
                        }
                    }
                };
                for (int i = 0; i < chunks; ++i, ++c) {
                    const uint32_t st = c & 1;
                    check(c, min(kTok, s.y - i * kTok));
                    make_kt(c, g, terms, tmem + st * (4 * kTmBuf) + g * kTmBuf + lanes, &sh.kt_empty[st], ((c >> 1) & 1) ^ 1);
                    arrive(&sh.kt_full[st]);
                    arrive(&sh.k_empty[c % kStages]);
                    if (i > 0) update(c - 1);
                    arrive(&sh.gates_empty[st]);
                }
                if (chunks > 0) update(c - 1);
                const int64_t at = entry_of(p, s);
                float *out = p.states + at * kState + (int64_t)(32 * u) * kHeadDim + row;
#pragma unroll
                for (int e = 0; e < 16; ++e) unf2(S[e], out[2 * e * kHeadDim], out[(2 * e + 1) * kHeadDim]);
                if (u == 0 && row == 0) p.decay[at] = decay_of_log2(log_decay);
            });
        } else {
            // ---- P, the state and the outputs: a thread stands for a row of P, a token of o and a key channel of the state
            uint32_t c = 0;
            const uint32_t to = tmem + kTmO + 32 * u + lanes, td = tmem + kTmD + 32 * u + lanes;
            // chunk c - 1's outputs: a row of fewer than 128 is stored at o, the others are left for the copying warp
            auto take_outputs = [&](auto last, __nv_bfloat16 *o, int rows) {
                const uint32_t n = c - 1;
                wait(&sh.o_full, n & 1);
                tc_fence_after();
                uint32_t y[4][4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float x[16];
                    tmem_ld16(to + 16 * k, x);
                    tmem_ld_wait_for(x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[2 * k + (j >> 2)][j & 3] = pack2(x[2 * j], x[2 * j + 1]);
                }
                tc_fence_before();
                if (!last) arrive(&sh.o_empty);
                if (__builtin_expect(sh.any_odd[u >> 1][n & 3], 0)) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (sh.odd[n & 3][32 * u + j] <= row) y[j >> 3][(j >> 1) & 3] |= j & 1 ? 0x7fff0000u : 0x7fffu;
                }
                if (!last || rows == kTok) {  // into the place of Q
                    uint8_t *q = sm + kSmQ + (n & 1) * kTile + (u >> 1) * kHalf + row * 128;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *(uint4 *)(q + (((4 * (u & 1) + j) ^ (row & 7)) << 4)) = make_uint4(y[j][0], y[j][1], y[j][2], y[j][3]);
                    fence_async_smem();
                } else if (row < rows) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) ((uint4 *)o)[j] = make_uint4(y[j][0], y[j][1], y[j][2], y[j][3]);
                }
                arrive(&sh.q_empty[n & 1]);
            };
            for_items([&](const Item &s, int chunks, int) {
                const int64_t place = (int64_t)(32 * u) * kHeadDim + row;  // of this thread's part of a state
                if (s.w & kNoSlot) {
                    for (int t = row; t < s.y; t += kTok) {
                        uint32_t *to_o = (uint32_t *)((__nv_bfloat16 *)a.o + ((int64_t)(s.x + t) * a.H + head_of(s)) * kHeadDim + 32 * u);
                        for (int j = 0; j < 16; ++j) to_o[j] = 0x7fc07fc0u;
                    }
                    return;
                }
                F2 S[16];  // value channels 32 u + 2 e, and the one after
                const float *init = state_before(p, s);
                if (init) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) S[e] = f2(init[place + 2 * e * kHeadDim], init[place + (2 * e + 1) * kHeadDim]);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) S[e] = 0;
                }
                auto publish = [&] {  // the copy of S that the next chunk's O is taken from
                    uint8_t *to_s = sm + kSmS + (u >> 1) * kHalf + row * 128;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *(uint4 *)(to_s + (((4 * (u & 1) + j) ^ (row & 7)) << 4)) =
                            make_uint4(narrow(S[4 * j]), narrow(S[4 * j + 1]), narrow(S[4 * j + 2]), narrow(S[4 * j + 3]));
                    fence_async_smem();
                };
                if (chunks > 0) {
                    publish();
                    arrive(&sh.o_empty);
                }
                for (int i = 0; i < chunks; ++i, ++c) {
                    const uint32_t st = c & 1, full = (c >> 1) & 1;
                    if (i > 0) take_outputs(std::false_type(), nullptr, kTok);
                    wait(&sh.v_ready[st], full);
                    const bool odd = sh.any_odd[u >> 1][c & 3];
                    const float own = sh.lower[st][row];
                    float upto = own, before = own;  // before: log2 decay from the end of block u to this row
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const float x = sh.block[st][b];
                        if (b < w) upto += x;
                        if (b < w && b > u) before += x;
                    }
                    // P: columns 32 u ..  e^{G_i - G_j} as a factor of the row and one of the column, with the end of block u
                    // between them; on the diagonal block, whose rows lie before that end, only while the row's stays finite.
                    const float tail = u == w ? own - sh.block[st][w] : before;
                    const float f = exp2f(tail) * a.scale;
                    wait(&sh.x_full, c & 1);
                    tc_fence_after();
                    const bool exact = u == w && __any_sync(0xffffffffu, !(tail < 80.0f));
                    auto make_p = [&](auto two) {
                        constexpr int terms = two ? 2 : 1;
#pragma unroll 1
                        for (int e = 0; e < 2; ++e) {
                            const int j0 = 32 * u + 16 * e, seen = row - j0;  // seen: the last column that this row sees
                            uint32_t y[8 * terms];  // the columns' leading terms, and what these leave
                            auto split = [&](int j, F2 z) {
                                y[j] = narrow(z);
                                if (terms == 2) y[8 + j] = narrow(fma2(wide(y[j]), f2(-1.0f, -1.0f), z));
                            };
                            if (u <= w) {
                                float x[16];
                                tmem_ld16(tmem + lanes + j0, x);
                                tmem_ld_wait_for(x);
                                if (__builtin_expect(exact, 0)) {
#pragma unroll
                                    for (int j = 0; j < 8; ++j) {
                                        const float2 z = *(const float2 *)&sh.lower[st][j0 + 2 * j];
                                        split(j, f2(x[2 * j] * (a.scale * exp2f(own - z.x)), x[2 * j + 1] * (a.scale * exp2f(own - z.y))));
                                    }
                                } else {
#pragma unroll
                                    for (int j = 0; j < 16; j += 4) {
                                        const float4 z = *(const float4 *)&sh.upper[st][j0 + j];
                                        split(j / 2, mul2(f2(x[j], x[j + 1]), mul2(f2(z.x, z.y), f2(f, f))));
                                        split(j / 2 + 1, mul2(f2(x[j + 2], x[j + 3]), mul2(f2(z.z, z.w), f2(f, f))));
                                    }
                                }
                                if (u == w)
#pragma unroll
                                    for (int j = 0; j < 8 * terms; ++j) y[j] = seen > 2 * (j & 7) ? y[j] : seen == 2 * (j & 7) ? y[j] & 0xffffu : 0u;
                            } else {
#pragma unroll
                                for (int j = 0; j < 8 * terms; ++j) y[j] = 0;
                            }
                            if constexpr (terms == 2) tmem_st16(tmem + lanes + j0, y);
                            else tmem_st8(tmem + lanes + j0, y);  // over scores of the block that are read
                        }
                    };
                    if (__builtin_expect(sh.early[c & 3], 0)) make_p(std::true_type());
                    else make_p(std::false_type());
                    arrive(&sh.gates_empty[st]);
                    // the state, while Q . S is computed
                    wait(&sh.d_full, c & 1);
                    tc_fence_after();
                    const float2 decay = sh.decay[c & 3];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float x[16];
                        tmem_ld16(td + 16 * k, x);
                        tmem_ld_wait_for(x);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            F2 &y = S[8 * k + j];
                            y = fma2(f2(decay.x, decay.x), y, fma2(f2(decay.y, decay.y), y, f2(x[2 * j], x[2 * j + 1])));
                        }
                    }
                    tc_fence_before();
                    if (__builtin_expect(odd, 0)) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const uint8_t *from = &sh.odd[c & 3][32 * u + 2 * e];
                            float lo, hi;
                            unf2(S[e], lo, hi);
                            S[e] = f2(from[0] < kTok ? NAN : lo, from[1] < kTok ? NAN : hi);
                        }
                    }
                    // (`odd` is written again four chunks on: behind P . V of the chunk after the next, so behind this and
                    // this chunk's outputs)
                    arrive(&sh.d_empty);
                    // O so far, Q . S, times the row's decay
                    const float to_row = exp2f(upto) * a.scale;
                    wait(&sh.qs_full, c & 1);
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float x[16];
                        tmem_ld16(to + 16 * k, x);
                        tmem_ld_wait_for(x);
                        uint32_t z[16];
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            float lo, hi;
                            unf2(mul2(f2(x[j], x[j + 1]), f2(to_row, to_row)), lo, hi);
                            z[j] = __float_as_uint(lo), z[j + 1] = __float_as_uint(hi);
                        }
                        tmem_st16(to + 16 * k, z);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    arrive(&sh.pv_ready);
                    if (i + 1 < chunks) publish();
                }
                if (float *out = state_after(p, s)) {
                    out += place;
#pragma unroll
                    for (int e = 0; e < 16; ++e) unf2(S[e], out[2 * e * kHeadDim], out[(2 * e + 1) * kHeadDim]);
                }
                if (chunks > 0) {
                    const int first = (chunks - 1) * kTok;
                    take_outputs(std::true_type(), (__nv_bfloat16 *)a.o + ((int64_t)(s.x + first + row) * a.H + head_of(s)) * kHeadDim + 32 * u, s.y - first);
                }
            });
        }
    }
    tc_fence_before();
    __syncthreads();
    if (dead) {  // a wait gave up: copies still in flight land, then all that this CTA had to write becomes NaN
        const long long t0 = clock64();
        while (clock64() - t0 < 100000000LL) __nanosleep(1000);
        for_items([&](const Item &s, int, int) {
            const int64_t at = entry_of(p, s);
            float *state = OUTPUT ? nullptr : p.states + at * kState;
            if (OUTPUT) {
                for (int64_t j = tid; j < (int64_t)s.y * kHeadDim; j += blockDim.x)
                    ((__nv_bfloat16 *)a.o)[((s.x + j / kHeadDim) * a.H + head_of(s)) * kHeadDim + j % kHeadDim] = __float2bfloat16_rn(NAN);
                if (!(s.w & kNoSlot)) state = state_after(p, s);
            }
            if (state)
                for (int j = tid; j < kState; j += blockDim.x) state[j] = NAN;
            if (!OUTPUT && tid == 0) p.decay[at] = make_float2(NAN, 0.0f);
        });
    }
    if (wid == 1) tmem_dealloc(tmem, 512);
}

// Tokens of a segment: so many that the segments of all heads are about as many as SMs.  A cut costs two launches
// and some 10 us, as much as three chunks: no segment has fewer than two of them, or, where
// there are several sequences, four.  (5 sequences of 17 to 200 tokens, 8 heads: 22.8 us of the device cut by the chunk, 15.7 whole.)
inline Cut cut_of(int64_t total_tokens, int n_seqs, int H) {
    const int64_t chunks = (total_tokens + kTok - 1) / kTok, each = std::max<int64_t>(1, sm_count() / H);
    return {kTok * std::max<int64_t>(n_seqs == 1 ? 2 : 4, (chunks + each - 1) / each), sm_count(), 3 * kTok};
}

}  // namespace

size_t linear_chunk_tc_workspace_bytes(int64_t total_tokens, int n_seqs, int H) {
    return segments_workspace_bytes(total_tokens, n_seqs, H, cut_of(total_tokens, n_seqs, H));
}

cudaError_t launch_linear_chunk_tc(const LinearChunkArgs &a, cudaStream_t stream) {
    const int64_t T = a.total_tokens, rows = std::max<int64_t>(T, 1);
    const int hk = a.H / a.group;
    CUtensorMap map_q, map_k, map_v, map_o;
    // (without a token there is no copy, and maybe no pointer)
    const void *none = a.final_state ? (const void *)a.final_state : a.initial_state;
    if (T == 0 && !none) return cudaSuccess;
    if (!encode_heads64(&map_q, T ? a.q : none, kHeadDim, hk, rows, a.q_stride, kTok) ||
        !encode_heads64(&map_k, T ? a.k : none, kHeadDim, hk, rows, a.k_stride, kTok) ||
        !encode_heads64(&map_v, T ? a.v : none, kHeadDim, a.H, rows, a.v_stride, kTok) ||
        !encode_heads64(&map_o, T ? a.o : none, kHeadDim, a.H, rows, (int64_t)a.H * kHeadDim, kTok))
        return cudaErrorUnknown;
    const ChunkParams p = plan_segments(a, cut_of(T, a.n_seqs, a.H));
    const Source source = source_of(p);
    auto launch = [&](auto kernel, int threads, int64_t items) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
        return e != cudaSuccess ? e
                                : launch_dependent(kernel, dim3((unsigned)std::min<int64_t>(items, sm_count())), dim3(threads),
                                                   kSmemBytes, stream, map_q, map_k, map_v, map_o, p);
    };
    cudaError_t e = launch_segment_lists(p, stream);
    if (e == cudaSuccess && p.entries > 0) {
        e = launch(source == kOne ? linear_chunk_kernel<false, kOne> : linear_chunk_kernel<false, kListed>, 640, (int64_t)p.entries * a.H);
        if (e == cudaSuccess) e = launch_segment_join(p, stream);
    }
    if (e == cudaSuccess)
        e = launch(source == kOne     ? linear_chunk_kernel<true, kOne>
                   : source == kWhole ? linear_chunk_kernel<true, kWhole>
                                      : linear_chunk_kernel<true, kListed>,
                   896, ((int64_t)p.entries + a.n_seqs) * a.H);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kda
