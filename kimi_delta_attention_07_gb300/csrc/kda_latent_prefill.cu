// Expanded latent attention over packed sequences: per (query i, head h) with
// keys k_j = [kv[j,h,:128] ; k_rope[j]] and values v_j = kv[j,h,128:],
//   x_j = scale * q . k_j over visible j,  o = sum_j softmax(x)_j v_j.
//
// 2 (192 + 128) operations a visible (query, key) pair and head: bound by the
// tensor cores.  A CTA takes 256 queries of a head, as two tiles of 128, and runs
// over the keys in tiles of 128:
//   X_t [128 x 128] = Q_t [128 x 192] . K^T    operands in shared memory
//   O_t [128 x 128] += P_t [128 x 128] . V     P from TMEM, over X_t's columns
// X_0, X_1, O_0, O_1 fill the 512 TMEM columns.  With two tiles the tensor core works on
// one while the softmax of the other runs: the order is
//   P_0 V(i), X_0(i+1), P_1 V(i), X_1(i+1), ...
// 768 + 512 clocks a tile and step at the tensor core's 4096 products a clock.
//
// Softmax: a thread owns a query row (TMEM lane), so maximum, sum and rescaling
// need no exchange.  The reference that p is taken against is raised (and the
// row of O rescaled) only where the row's maximum passes it by 2^8; p, its sum
// and O share it, so that the quotient is unchanged.
//
// K and V tiles come as blocks of 64 columns (16 KB) through a ring of eight,
// K(i) three, V(i) two, released block by block.  The positional key's block is
// read for every head from the one shared copy.
//
// Masked places: keys that a row does not see get p = 0, and 0 times a value has
// to be 0 whatever the value is.  In the tiles where some key is not seen by
// some row, two warps look through V before it is used: rows past the
// sequence's end become 0, and so do values that are not finite; the epilogue
// then adds those to the rows that see them.
//
// CTAs ask for work with cluster launch control: the grid has a CTA per 256
// queries and head, heaviest first within a sequence, and a running CTA takes
// over the next unlaunched one, so that its loads overlap the last epilogue.
//
// Warps: 0..3 and 4..7 softmax and epilogue of the two tiles, 8 TMA and
// scheduling, 9 MMA, 10 and 11 the value blocks' check.
#include <algorithm>

#include "kda_attn.cuh"

namespace kda {

using namespace tc;

namespace {

constexpr int kTile = 128;           // queries per tile, keys per step
constexpr int kItem = 2 * kTile;     // queries per CTA
constexpr int kThreads = 384;
constexpr int kRing = 8;             // 16 KB blocks
constexpr uint32_t kBlock = kTile * 128;
constexpr float kRaise = 8.0f;       // log2 by which a score may pass its row's reference

// shared memory (from a 1024-byte boundary)
constexpr uint32_t kSmQ = 0;                          // [2 tiles][3 blocks]
constexpr uint32_t kSmRing = kSmQ + 2 * 3 * kBlock;   // kRing blocks
constexpr uint32_t kSmemBytes = kSmRing + kRing * kBlock + 1024;

constexpr uint32_t kTmemO = 256;  // X_t at 128 t, O_t at 256 + 128 t

struct Item {
    int n, h, q0, lq, off;  // sequence, head, first query in it, its queries, lk - lq
    int lk, steps0, steps1; // keys, steps of each tile
    int64_t qa, ka;         // the sequence's first query and key
    int masked;             // first step with a key that some row does not see
    int valid;              // 0: no further item
    __device__ __forceinline__ int steps(int t) const { return t ? steps1 : steps0; }
    __device__ __forceinline__ int most() const { return max(steps0, steps1); }
};

struct PrefillParams {
    LatentPrefillArgs a;
};

__device__ __forceinline__ int blocks_of(const LatentPrefillArgs &a, int n) {
    const int qa = a.cu_q[n], qb = a.cu_q[n + 1], ka = a.cu_k[n], kb = a.cu_k[n + 1];
    const bool ok = qa >= 0 && qb >= qa && qb <= a.total_q && ka >= 0 && kb >= ka && kb <= a.total_k;
    return ok ? (qb - qa + kItem - 1) / kItem : 0;
}

__device__ __forceinline__ uint32_t not_finite(uint32_t two_bf16) {
    return ((two_bf16 & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
           ((two_bf16 & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

// POSITIVE: scale > 0, so that the largest product is the largest score
template <bool POSITIVE>
__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_kv,
                          const __grid_constant__ CUtensorMap map_r, const PrefillParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    __shared__ uint64_t full[kRing], empty[kRing], q_full[2], q_empty[2], x_full[2], p_full[2], o_full[2], o_empty[2],
        unchecked[2][2], item_full[2], item_empty[2], next_full;
    __shared__ __align__(16) uint4 next_answer;
    __shared__ Item items[2];
    __shared__ int piece[kThreads];  // blocks of the sequences before each thread's
    __shared__ int warp_total[kThreads / 32];
    __shared__ volatile int dead, odd[2];
    __shared__ uint32_t tmem_base;

    const LatentPrefillArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1), mbar_init(&q_empty[i], 1);
            mbar_init(&x_full[i], 1), mbar_init(&p_full[i], 128);
            mbar_init(&o_full[i], 1), mbar_init(&o_empty[i], 128);
            mbar_init(&unchecked[0][i], 1), mbar_init(&unchecked[1][i], 1);
            mbar_init(&item_full[i], 1), mbar_init(&item_empty[i], 11);
        }
        mbar_init(&next_full, 1);
        fence_mbar_init();
        dead = 0;
    }
    if (wid == 9) tmem_alloc(&tmem_base, 512);
    // the blocks of 256 queries of the sequences before each thread's piece
    const int per = (a.n_seqs + kThreads - 1) / kThreads;
    {
        const int n0 = min(tid * per, a.n_seqs), n1 = min(n0 + per, a.n_seqs);
        int mine = 0;
        for (int n = n0; n < n1; ++n) mine += blocks_of(a, n);
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        if (lane == 31) warp_total[wid] = upto;
        __syncthreads();
        for (int w = 0; w < wid; ++w) upto += warp_total[w];
        piece[tid] = upto - mine;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    // a bounded wait; once one has given up, none waits any more
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!dead && !mbar_wait(bar, parity)) dead = 1;
    };
    // the it-th item of this CTA, as the scheduling thread published it
    auto item_of = [&](int it) -> const Item & {
        wait(&item_full[it & 1], (it >> 1) & 1);
        return items[it & 1];
    };
    auto item_done = [&](int it) { mbar_arrive(&item_empty[it & 1]); };

    if (wid == 8) {
        // ---- scheduling and TMA
        if (elect_one()) {
            int it = 0, qn[2] = {0, 0};  // items published; queries' tiles loaded
            uint32_t c = 0, checks = 0;  // blocks loaded; steps whose values are checked
            int cta = blockIdx.x;
            for (int asked = 0; cta >= 0; ++asked) {
                mbar_arrive_expect_tx(&next_full, 16);
                next_cta_request(&next_answer, &next_full);
                const int rank = cta / a.H;
                // the piece that holds block `rank`, then the sequence in it
                int lo = 0, hi = kThreads;
                while (lo + 1 < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (piece[mid] <= rank) lo = mid; else hi = mid;
                }
                int n = lo * per, before = piece[lo], blocks = 0;
                for (; n < min((lo + 1) * per, a.n_seqs); ++n) {
                    blocks = blocks_of(a, n);
                    if (rank < before + blocks) break;
                    before += blocks;
                    blocks = 0;
                }
                if (blocks > 0) {
                    wait(&item_empty[it & 1], ((it >> 1) & 1) ^ 1);
                    Item &s = items[it & 1];
                    s.n = n;
                    s.h = cta - rank * a.H;
                    s.qa = a.cu_q[n];
                    s.ka = a.cu_k[n];
                    s.lq = a.cu_q[n + 1] - a.cu_q[n];
                    s.lk = a.cu_k[n + 1] - a.cu_k[n];
                    s.off = s.lk - s.lq;
                    s.q0 = (blocks - 1 - (rank - before)) * kItem;
                    int first = s.lk;  // keys that every row of the item sees
                    for (int t = 0; t < 2; ++t) {
                        const int r0 = s.q0 + t * kTile, r1 = min(r0 + kTile, s.lq);  // rows [r0, r1)
                        const int seen = r1 <= r0 ? 0 : a.causal ? min(s.lk, r1 + s.off) : s.lk;
                        (t ? s.steps1 : s.steps0) = seen > 0 ? (seen + kTile - 1) / kTile : 0;
                        if (r1 > r0 && a.causal) first = min(first, max(r0 + 1 + s.off, 0));
                    }
                    s.masked = first / kTile;
                    s.valid = 1;
                    odd[it & 1] = 0;
                    const Item cur = s;
                    mbar_arrive(&item_full[it & 1]);
                    ++it;
                    for (int t = 0; t < 2; ++t) {
                        if (cur.steps(t) == 0) continue;
                        wait(&q_empty[t], (qn[t] & 1) ^ 1);
                        ++qn[t];
                        mbar_arrive_expect_tx(&q_full[t], 3 * kBlock);
                        for (int b = 0; b < 3; ++b)
                            tma_load_3d(sm + kSmQ + (t * 3 + b) * kBlock, &map_q, b * 64, cur.h,
                                        (int)cur.qa + cur.q0 + t * kTile, &q_full[t]);
                    }
                    const int steps = cur.most();
                    for (int i = 0; i < steps && !dead; ++i) {
                        const int row = (int)cur.ka + i * kTile;
                        for (int b = 0; b < 5; ++b, ++c) {
                            const uint32_t slot = c % kRing;
                            wait(&empty[slot], ((c / kRing) & 1) ^ 1);
                            // values to be checked land on the checking warp's barrier; it signals `full`
                            uint64_t *bar = b >= 3 && i >= cur.masked ? &unchecked[b - 3][checks & 1] : &full[slot];
                            mbar_arrive_expect_tx(bar, kBlock);
                            uint8_t *dst = sm + kSmRing + slot * kBlock;
                            if (b == 2) tma_load_2d(dst, &map_r, 0, row, bar);
                            else tma_load_3d(dst, &map_kv, (b < 2 ? b : b - 1) * 64, cur.h, row, bar);
                        }
                        if (i >= cur.masked) ++checks;
                    }
                }
                wait(&next_full, asked & 1);
                cta = dead ? -1 : next_cta_answer(&next_answer);
                fence_async_smem();
            }
            wait(&item_empty[it & 1], ((it >> 1) & 1) ^ 1);
            items[it & 1].valid = 0;
            mbar_arrive(&item_full[it & 1]);
        }
        __syncwarp();
    } else if (wid == 9) {
        // ---- MMA, issued by one thread
        if (elect_one()) {
            const uint32_t q_s = smem_u32(sm + kSmQ), ring = smem_u32(sm + kSmRing);
            constexpr uint32_t idesc_x = idesc_bf16(kTile, kTile);
            constexpr uint32_t idesc_o = idesc_bf16(kTile, 64) | (1u << 16);
            uint32_t c = 0;  // ring blocks before this step
            int qn[2] = {0, 0}, pn[2] = {0, 0}, on[2] = {0, 0};
            for (int it = 0;; ++it) {
                const Item s = item_of(it);
                if (dead || !s.valid) break;
                const int steps = s.most();
                // X_t(i); its K blocks are released by the last tile that reads them
                auto first_product = [&](int t, uint32_t ck, bool release) {
#pragma unroll
                    for (int b = 0; b < 3; ++b) {
                        const uint32_t slot = (ck + b) % kRing;
                        wait(&full[slot], ((ck + b) / kRing) & 1);
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16(tmem + t * kTile,
                                     ((uint64_t)kDescHi << 32) | operand_lo<false, kTile>(q_s + (t * 3 + b) * kBlock, k),
                                     ((uint64_t)kDescHi << 32) | operand_lo<false, kTile>(ring + slot * kBlock, k),
                                     idesc_x, b + k > 0);
                        if (release) mma_commit(&empty[slot]);
                    }
                    mma_commit(&x_full[t]);
                };
                for (int t = 0; t < 2; ++t)
                    if (s.steps(t) > 0) {
                        wait(&q_full[t], qn[t] & 1);
                        ++qn[t];
                        first_product(t, c, t == 1 || s.steps1 == 0);
                        if (s.steps(t) == 1) mma_commit(&q_empty[t]);
                    }
                for (int i = 0; i < steps && !dead; ++i, c += 5) {
#pragma unroll 1
                    for (int t = 0; t < 2; ++t) {
                        if (i >= s.steps(t)) continue;
                        wait(&p_full[t], pn[t] & 1);
                        ++pn[t];
                        if (i == 0) {
                            if (on[t] > 0) wait(&o_empty[t], (on[t] - 1) & 1);
                            ++on[t];
                        }
                        const bool last_v = t == 1 || i >= s.steps1;
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const uint32_t cv = c + 3 + b, slot = cv % kRing;
                            wait(&full[slot], (cv / kRing) & 1);
                            tc_fence_after();
#pragma unroll
                            for (int k = 0; k < kTile / 16; ++k)
                                mma_bf16_ts(tmem + kTmemO + t * kTile + b * 64, tmem + t * kTile + k * 8,
                                            ((uint64_t)kDescHi << 32) | operand_lo<true, kTile>(ring + slot * kBlock, k),
                                            idesc_o, i > 0 || k > 0);
                            if (last_v) mma_commit(&empty[slot]);
                        }
                        if (i + 1 == s.steps(t)) mma_commit(&o_full[t]);
                        if (i + 1 < s.steps(t)) {
                            first_product(t, c + 5, t == 1 || i + 1 >= s.steps1);
                            if (i + 2 == s.steps(t)) mma_commit(&q_empty[t]);
                        }
                    }
                }
                item_done(it);
            }
        }
        __syncwarp();
    } else if (wid >= 10) {
        // ---- the check of V's block g in steps with masked places, between its copy and `full`
        const int g = wid - 10;
        uint32_t c = 0;
        int checks = 0;
        for (int it = 0;; ++it) {
            const Item s = item_of(it);
            if (__any_sync(0xffffffffu, dead || !s.valid)) break;
            const int steps = s.most();
            for (int i = 0; i < steps; ++i, c += 5) {
                if (i < s.masked) continue;
                const uint32_t slot = (c + 3 + g) % kRing;
                wait(&unchecked[g][checks & 1], (checks >> 1) & 1);
                const int rows = min(s.lk - i * kTile, kTile);  // keys of the sequence in this tile
                uint8_t *blk = sm + kSmRing + slot * kBlock;
                bool found = false;
#pragma unroll 8
                for (int j = 0; j < kTile * 8 / 32; ++j) {
                    const int row = j * 4 + (lane >> 3);
                    uint4 *v = (uint4 *)(blk + row * 128 + (lane & 7) * 16);
                    if (row >= rows) {
                        *v = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    const uint4 u = *v;
                    const uint4 m = make_uint4(not_finite(u.x), not_finite(u.y), not_finite(u.z), not_finite(u.w));
                    if (m.x | m.y | m.z | m.w) {
                        found = true;
                        *v = make_uint4(u.x & ~m.x, u.y & ~m.y, u.z & ~m.z, u.w & ~m.w);
                    }
                }
                if (found) odd[it & 1] = 1;
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[slot]);
                ++checks;
            }
            __syncwarp();
            if (lane == 0) item_done(it);
        }
    } else {
        // ---- softmax of tile t: a thread owns a query row
        const int t = wid >> 2, quad = wid & 3;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t tx = tmem + t * kTile + lanes, to = tmem + kTmemO + t * kTile + lanes;
        const float scale2 = a.scale == 0.0f ? 1.0f : fabsf(a.scale) * kLog2e;
        int xn = 0, on = 0;
        for (int it = 0;; ++it) {
            const Item s = item_of(it);
            if (__any_sync(0xffffffffu, dead || !s.valid)) break;
            const int row = s.q0 + t * kTile + quad * 32 + lane;
            const bool real = row < s.lq;
            const int limit = !real ? 0 : a.causal ? min(s.lk, row + 1 + s.off) : s.lk;  // keys below it are seen
            float m = -INFINITY, l = 0.0f;  // m in units of x / |scale|
            const int steps = s.steps(t);
            bool gave_up = false;
            for (int i = 0; i < steps; ++i, ++xn) {
                wait(&x_full[t], xn & 1);
                if (__any_sync(0xffffffffu, dead)) {
                    gave_up = true;
                    break;
                }
                tc_fence_after();
                // scores 32 k .. 32 k + 31 of the row, requested and then prepared
                const int left = limit - i * kTile;
                const bool hide = __any_sync(0xffffffffu, left < kTile);
                auto prepare = [&](int k, float (&x)[32]) {
                    if (!POSITIVE) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[j] = a.scale < 0.0f ? -x[j] : 0.0f;
                    }
                    if (hide) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[j] = 32 * k + j < left ? x[j] : -INFINITY;
                    }
                };
                float x0[32], x1[32], top = -INFINITY;
                auto largest = [&](int k, float (&x)[32]) {
                    prepare(k, x);
#pragma unroll
                    for (int j = 0; j < 32; ++j) top = fmaxf(top, x[j]);
                };
                tmem_ld32(tx, x0);
                tmem_ld_wait32(x0);
                tmem_ld32(tx + 32, x1);
                largest(0, x0);
                tmem_ld_wait32(x1);
                tmem_ld32(tx + 64, x0);
                largest(1, x1);
                tmem_ld_wait32(x0);
                tmem_ld32(tx + 96, x1);
                largest(2, x0);
                tmem_ld_wait32(x1);
                tmem_ld32(tx, x0);
                largest(3, x1);
                tmem_ld_wait32(x0);
                tmem_ld32(tx + 32, x1);
                const bool raise = (top - m) * scale2 > kRaise;
                if (__any_sync(0xffffffffu, raise)) {
                    const float f = raise ? exp2_sfu((m - top) * scale2) : 1.0f;
                    if (raise) m = top;
                    l *= f;
                    if (i > 0) {  // X_t(i) was issued after P_t V(i-1): O_t is complete
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            float o[16];
                            tmem_ld16(to + 16 * k, o);
                            tmem_ld_wait();
                            uint32_t u[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(o[j] * f);
                            tmem_st16(to + 16 * k, u);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.0f : m * scale2;
                // P over the columns of scores that have been read: p_k takes 16 k .. 16 k + 15
                auto weigh = [&](int k, float (&x)[32]) {
                    prepare(k, x);
                    uint32_t u[16];
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float e0 = exp2_sfu(fmaf(x[2 * j], scale2, -ref));
                        const float e1 = exp2_sfu(fmaf(x[2 * j + 1], scale2, -ref));
                        sum += e0 + e1;
                        u[j] = pack2(e0, e1);
                    }
                    l += sum;
                    tmem_st16(tx + 16 * k, u);
                };
                weigh(0, x0);
                tmem_ld_wait32(x1);
                tmem_ld32(tx + 64, x0);
                weigh(1, x1);
                tmem_ld_wait32(x0);
                tmem_ld32(tx + 96, x1);
                weigh(2, x0);
                tmem_ld_wait32(x1);
                weigh(3, x1);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&p_full[t]);
            }
            const int64_t out = ((s.qa + row) * a.H + s.h);
            const float inv = gave_up ? NAN : l == 0.0f ? 1.0f : 1.0f / l;
            if (steps > 0 && !gave_up) {
                wait(&o_full[t], on & 1);
                ++on;
                tc_fence_after();
            }
            const bool add = odd[it & 1] != 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float o[32];
                if (steps > 0) {
                    tmem_ld32(to + 32 * k, o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0.0f;
                }
                if (__any_sync(0xffffffffu, add)) {
                    // values that were taken out of V because they are not finite
                    for (int key = s.masked * kTile; key < limit; ++key) {
                        const __nv_bfloat16 *v = a.kv + (s.ka + key) * a.kv_stride + (int64_t)s.h * kKvRow + kNope + 32 * k;
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float w = __bfloat162float(v[j]);
                            if (!(fabsf(w) < INFINITY)) o[j] += w;
                        }
                    }
                    __syncwarp();
                }
                if (real) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 u = make_uint4(pack2(o[8 * j] * inv, o[8 * j + 1] * inv),
                                                   pack2(o[8 * j + 2] * inv, o[8 * j + 3] * inv),
                                                   pack2(o[8 * j + 4] * inv, o[8 * j + 5] * inv),
                                                   pack2(o[8 * j + 6] * inv, o[8 * j + 7] * inv));
                        *(uint4 *)(a.o + out * kHeadDim + 32 * k + 8 * j) = u;
                    }
                }
            }
            if (real && a.lse)
                a.lse[out] = gave_up ? NAN : l == 0.0f ? -INFINITY : (m * scale2 + log2_sfu(l)) * kLn2;
            if (steps > 0) {
                tc_fence_before();
                mbar_arrive(&o_empty[t]);
            }
            __syncwarp();
            if (lane == 0) item_done(it);
            if (gave_up) break;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (dead) {  // let copies still in flight land before the CTA's memory is given up
        const long long t0 = clock64();
        while (clock64() - t0 < 100000000LL) __nanosleep(1000);
    }
    if (wid == 9) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, cudaStream_t stream) {
    CUtensorMap map_q, map_kv, map_r;
    if (!encode_heads64(&map_q, a.q, kQk, a.H, a.total_q, a.q_stride, kTile)) return cudaErrorUnknown;
    if (a.total_k > 0) {
        if (!encode_heads64(&map_kv, a.kv, kKvRow, a.H, a.total_k, a.kv_stride, kTile) ||
            !encode_rows64(&map_r, a.k_rope, kRope, a.total_k, a.rope_stride, kTile))
            return cudaErrorUnknown;
    } else {
        map_kv = map_r = map_q;  // no key: not used
    }
    auto kernel = a.scale > 0.0f ? latent_prefill_kernel<true> : latent_prefill_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    // every sequence adds at most one incomplete block
    const int64_t blocks = a.total_q / kItem + std::min<int64_t>(a.n_seqs, a.total_q);
    if (blocks * a.H > INT32_MAX) return cudaErrorInvalidValue;
    kernel<<<dim3((unsigned)(blocks * a.H)), kThreads, kSmemBytes, stream>>>(map_q, map_kv, map_r, PrefillParams{a});
    return cudaGetLastError();
}

}  // namespace kda
