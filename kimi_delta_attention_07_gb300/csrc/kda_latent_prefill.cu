// Expanded latent attention over packed sequences: per (query i, head h) with
// keys k_j = [kv[j,h,:128] ; k_rope[j]] and values v_j = kv[j,h,128:],
//   x_j = scale * q . k_j over visible j,  o = sum_j softmax(x)_j v_j.
//
// 2 (192 + 128) operations a visible (query, key) pair and head: bound by the
// tensor cores.  A CTA takes 256 queries of a head, as two tiles of 128, and runs
// over the keys in tiles of 128:
//   X_t [128 x 128] = Q_t [128 x 192] . K^T    operands in shared memory
//   O_t [128 x 128] += P_t [128 x 128] . V     P from TMEM, over X_t's columns
// X_0, X_1, O_0, O_1 fill the 512 TMEM columns.  With two tiles the tensor core
// works on one while the softmax of the other runs: one thread issues
//   P_0 V(i), X_0(i+1), P_1 V(i), X_1(i+1), ...
// (its MMAs execute in that order, so that X_t(i+1) overwrites P_t(i) after it was
// read), 768 + 512 clocks a tile and step at the tensor core's 4096 products a clock.
//
// What bounded a step was the chain X_t(i), softmax, P_t V(i), X_t(i+1) of a tile
// (4650 clocks with one thread a row, against the 2560 that the tensor core needs
// for both tiles) and the issuing thread's own instructions.  So two threads own a
// query row (TMEM lane), 64 keys of a step each; they exchange their maxima in a
// step and their sums at the end, and hand P over in two parts, the first of which
// is multiplied while the second is computed.  A step takes about 3200 clocks: 1580
// TFLOP/s on 8192 queries and keys without a mask, where shared memory, which
// X_t's operands alone read at its full 128 bytes a clock, leaves little room.
//
// The reference that p is taken against is raised (and the row of O rescaled) only
// where the row's maximum passes it by 2^8; p, its sum and O share it, so that the
// quotient is unchanged.
//
// K and V tiles come as blocks of 64 columns (16 KB) through a ring of eight, K(i)
// three, V(i) two; the positional key's block is read for every head from the one
// shared copy.
//
// Masked places: keys that a row does not see get p = 0, and 0 times a value has
// to be 0 whatever the value is.  In the tiles where some key is not seen by
// some row, two warps look through V before it is used: rows past the
// sequence's end become 0, and so do values that are not finite; they are added to
// the outputs of the rows that see them.
//
// Few queries behind many keys (a chunk of a prompt behind its cached part) would leave
// most SMs idle: the keys of a block of queries are then split into parts of whole
// steps, each an item whose (O, max, sum) goes to the workspace, and a second,
// dependent kernel joins them in order.
//
// CTAs ask for work with cluster launch control: the grid has a CTA per 256
// queries and head, heaviest first within a sequence, and a running CTA takes
// over the next unlaunched one, so that its loads overlap the last epilogue.
// 4096 queries and keys of 32 heads: 117 us a call in a graph of calls, 1470 TFLOP/s of the visible pairs.
//
// Warps: 0..7 and 8..15 softmax and epilogue of the two tiles, 16 TMA and
// scheduling, 17 MMA, 18 and 19 the value blocks' check.
#include <algorithm>
#include <type_traits>

#include "kda_attn.cuh"

namespace kda {

using namespace tc;

namespace {

constexpr int kTile = 128;           // queries per tile, keys per step
constexpr int kItem = 2 * kTile;     // queries per CTA
constexpr int kThreads = 640;
constexpr int kRing = 8;             // 16 KB blocks
constexpr uint32_t kBlock = kTile * 128;
constexpr int kSplitSteps = KDA_LATENT_PREFILL_SPLIT_KEYS / kTile;  // items of fewer are not split
constexpr int kMinSteps = 2;         // of a part, where an item's keys are split
constexpr float kRaise = 8.0f;       // log2 by which a score may pass its row's reference

// shared memory (from a 1024-byte boundary)
constexpr uint32_t kSmQ = 0;                          // [2 tiles][3 blocks]
constexpr uint32_t kSmRing = kSmQ + 2 * 3 * kBlock;   // kRing blocks
constexpr uint32_t kSmShared = kSmRing + kRing * kBlock;
constexpr int kPieces = 128;  // of the sequences, for finding the one that a block belongs to

constexpr uint32_t kTmemO = 256;  // X_t at 128 t, O_t at 256 + 128 t

struct Item {
    int h, q0, lq, off;     // head, first query (-128: tile 1 begins the sequence), its queries, lk - lq
    int lk, steps0, steps1; // keys, steps of each tile
    int qa, ka;             // the sequence's first query and key
    int masked;             // first step with a key that some row does not see
    int valid;              // 0: no further item
    __device__ __forceinline__ int steps(int t) const { return t ? steps1 : steps0; }
    __device__ __forceinline__ int most() const { return max(steps0, steps1); }
};

struct SplitItem : Item {
    int part;  // of an item whose keys are split: its place in the workspace; else -1
};

template <typename ITEM>
struct Shared {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], q_full[2], q_empty[2], x_full[2], p_full[2][2], o_full[2], o_empty[2],
        unchecked[2][2], item_full[2], item_empty[2], next_full;
    uint4 next_answer;
    ITEM items[3];            // two handed out in turn; [2]: claimed, not handed out yet
    float half[2][2][kTile];  // what the two threads of a row exchange
    int piece[kPieces];       // blocks of 256 queries of the sequences before each piece
    int warp_total[kPieces / 32];
    volatile int dead, odd[2];
    uint32_t tmem_base;
};
constexpr uint32_t kSmemBytes = kSmShared + sizeof(Shared<SplitItem>);
static_assert(kSmemBytes <= 232448, "shared memory");

struct Stat {  // of a row's part: reference (log2), sum
    float m, l;
};
struct Join {  // an item whose keys are split: first token, rows, parts (0: nothing to join)
    int32_t q, rows, parts, pad;
};
struct Part {
    float o[kItem][kHeadDim];  // not divided by the sum
};

struct PrefillParams {
    LatentPrefillArgs a;
};
struct SplitParams : PrefillParams {
    int splits, blocks;  // most parts of an item; blocks of queries, of which there are at most so many
    Part *parts;  // [CTA of the grid]
    Stat *stats;  // [CTA of the grid][kItem]
    Join *joins;  // [block of queries][H]
};

__device__ __forceinline__ int blocks_of(const LatentPrefillArgs &a, int n) {
    const int qa = a.cu_q[n], qb = a.cu_q[n + 1], ka = a.cu_k[n], kb = a.cu_k[n + 1];
    const bool ok = qa >= 0 && qb >= qa && qb <= a.total_q && ka >= 0 && kb >= ka && kb <= a.total_k;
    return ok ? (qb - qa + kItem - 1) / kItem : 0;
}

// Whether a key's 128 + 64 values are all finite.
__device__ __forceinline__ bool finite_key(const __nv_bfloat16 *nope, const __nv_bfloat16 *rope) {
    uint32_t ones = 0;
#pragma unroll 1
    for (int j = 0; j < kQk / 8; ++j)
        ones |= exponent_of_ones(*(const uint4 *)(j < kNope / 8 ? nope + 8 * j : rope + 8 * j - kNope));
    return ones == 0;
}

// POSITIVE: scale > 0, so that the largest product is the largest score.  SPLIT: the keys of an item
// may be split (types of its own, because the other kernel's registers are so short that a
// member more in its item takes it from 123 to 139 us).
template <bool POSITIVE, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_kv,
                          const __grid_constant__ CUtensorMap map_r,
                          const std::conditional_t<SPLIT, SplitParams, PrefillParams> p) {
    using ITEM = std::conditional_t<SPLIT, SplitItem, Item>;
    // all shared memory is dynamic, so that it begins on a 1024-byte boundary
    extern __shared__ __align__(1024) uint8_t sm[];
    auto &sh = *reinterpret_cast<Shared<ITEM> *>(sm + kSmShared);
    auto &k_full = sh.k_full, &k_empty = sh.k_empty, &v_full = sh.v_full, &v_empty = sh.v_empty;
    auto &q_full = sh.q_full, &q_empty = sh.q_empty, &x_full = sh.x_full, &o_full = sh.o_full, &o_empty = sh.o_empty,
         &item_full = sh.item_full, &item_empty = sh.item_empty;
    auto &p_full = sh.p_full, &unchecked = sh.unchecked;
    volatile int &dead = sh.dead;
    volatile int *odd = sh.odd;

    const LatentPrefillArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 1), mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 2), mbar_init(&v_empty[i], 1);  // a copy and a second arrival, or two checks
            mbar_init(&q_full[i], 1), mbar_init(&q_empty[i], 1);
            mbar_init(&x_full[i], 1), mbar_init(&p_full[i][0], 256), mbar_init(&p_full[i][1], 256);
            mbar_init(&o_full[i], 1), mbar_init(&o_empty[i], 256);
            mbar_init(&unchecked[0][i], 1), mbar_init(&unchecked[1][i], 1);
            mbar_init(&item_full[i], 1), mbar_init(&item_empty[i], 19);
        }
        mbar_init(&sh.next_full, 1);
        fence_mbar_init();
        dead = 0;
        for (int i = 0; i < 3; ++i) sh.items[i].valid = 0;
    }
    if (wid == 17) tmem_alloc(&sh.tmem_base, 512);
    griddep_wait();
    if (!SPLIT) griddep_launch_dependents();  // (a join's CTAs would take registers that ours need)
    // the blocks of 256 queries of the sequences before each thread's piece
    const int per = (a.n_seqs + kPieces - 1) / kPieces;
    int upto = 0, own = 0;
    if (tid < kPieces) {
        const int n0 = min(tid * per, a.n_seqs), n1 = min(n0 + per, a.n_seqs);
        for (int n = n0; n < n1; ++n) own += blocks_of(a, n);
        upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        if (lane == 31) sh.warp_total[wid] = upto;
    }
    __syncthreads();
    if (tid < kPieces) {
        for (int w = 0; w < wid; ++w) upto += sh.warp_total[w];
        sh.piece[tid] = upto - own;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    // a bounded wait; once one has given up, none waits any more
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return;
        if (!dead && !mbar_wait(bar, parity)) dead = 1;
    };
    // the it-th item of this CTA, as the scheduling thread published it
    auto item_of = [&](int it) -> const ITEM & {
        wait(&item_full[it & 1], (it >> 1) & 1);
        return sh.items[it & 1];
    };
    auto item_done = [&](int it) { mbar_arrive(&item_empty[it & 1]); };

    if (wid == 16) {
        // ---- scheduling and TMA
        if (elect_one()) {
            int it = 0, qn[2] = {0, 0};  // items published; queries' tiles loaded
            uint32_t step = 0, checks = 0, asked = 0;  // steps loaded; those whose values are checked
            // the item of a CTA of the grid; false if there is none (the grid is an upper bound)
            auto item_of_cta = [&](int cta, ITEM &s) {
                int rank = cta / a.H, split = 0;
                s.h = cta - rank * a.H;
                Join *join = nullptr;
                if constexpr (SPLIT) {
                    // (blocks inside parts, so that the blocks of a head read the same keys at the same time)
                    split = rank / p.blocks, rank -= split * p.blocks;
                    if (split == 0) join = p.joins + rank * a.H + s.h;
                }
                // the piece that holds block `rank`, then the sequence in it
                int lo = 0, hi = kPieces;
                while (lo + 1 < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (sh.piece[mid] <= rank) lo = mid; else hi = mid;
                }
                int n = lo * per, before = sh.piece[lo], blocks = 0;
                for (; n < min((lo + 1) * per, a.n_seqs); ++n) {
                    blocks = blocks_of(a, n);
                    if ((unsigned)(rank - before) < (unsigned)blocks) break;
                    before += blocks;
                    blocks = 0;
                }
                if (blocks == 0) {
                    if (join) join->parts = 0;
                    return false;
                }
                s.qa = a.cu_q[n];
                s.ka = a.cu_k[n];
                s.lq = a.cu_q[n + 1] - s.qa;
                s.lk = a.cu_k[n + 1] - s.ka;
                s.off = s.lk - s.lq;
                s.q0 = (blocks - 1 - (rank - before)) * kItem;
                int first = s.lk;  // keys that every row of the item sees
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int r0 = s.q0 + t * kTile, r1 = min(r0 + kTile, s.lq);  // rows [r0, r1)
                    const int seen = r1 <= r0 ? 0 : a.causal ? min(s.lk, r1 + s.off) : s.lk;
                    (t ? s.steps1 : s.steps0) = seen > 0 ? (seen + kTile - 1) / kTile : 0;
                    if (r1 > r0 && a.causal) first = min(first, max(r0 + 1 + s.off, 0));
                }
                s.masked = first / kTile;
                s.valid = 1;
                // short sequences take the tiles in turn, so that one's epilogue runs beside the next one's scores
                // (32 of 128 queries behind 1024 keys, 32 heads: 124 instead of 137 us)
                if (!SPLIT && s.lq <= kTile && (it & 1)) s.q0 = -kTile, s.steps1 = s.steps0, s.steps0 = 0;
                if constexpr (SPLIT) {
                    // parts of equal length, each a sequence of its own whose keys begin at its first step
                    const int most = s.most(), parts = most < kSplitSteps ? 1 : min(p.splits, (most + kMinSteps - 1) / kMinSteps);
                    if (join) *join = {s.qa + s.q0, min(s.lq - s.q0, kItem), parts > 1 ? parts : 0, 0};
                    if (split >= parts) return false;
                    const int base = most / parts, rem = most - base * parts;
                    const int k0 = split * base + min(split, rem), len = base + (split < rem);
                    s.ka += k0 * kTile, s.lk -= k0 * kTile, s.off -= k0 * kTile;
                    s.steps0 = min(max(s.steps0 - k0, 0), len), s.steps1 = min(max(s.steps1 - k0, 0), len);
                    s.masked = max(s.masked - k0, 0);
                    s.part = parts > 1 ? cta : -1;
                }
                return true;
            };
            auto ask = [&] {
                mbar_arrive_expect_tx(&sh.next_full, 16);
                next_cta_request(&sh.next_answer, &sh.next_full);
            };
            // the next item that the answers name; false once there is none
            auto next_item = [&](ITEM &s) {
                for (;;) {
                    // (also when another wait has given up: a CTA that was handed over is this one's to answer for)
                    if (!mbar_wait(&sh.next_full, asked++ & 1)) {
                        dead = 1;
                        return false;
                    }
                    const int cta = next_cta_answer(&sh.next_answer);
                    fence_async_smem();
                    if (cta < 0) return false;
                    if (item_of_cta(cta, s)) return true;
                    ask();
                }
            };
            ITEM cur, next;
            bool more = item_of_cta(blockIdx.x, cur);
            if (!more) {
                ask();
                more = next_item(cur);
            }
            while (more) {
                wait(&item_empty[it & 1], ((it >> 1) & 1) ^ 1);
                if (dead) {  // the item two before may still be in hand
                    sh.items[2] = cur;
                    break;
                }
                sh.items[it & 1] = cur;
                odd[it & 1] = 0;
                mbar_arrive(&item_full[it & 1]);
                ++it;
                auto queries = [&](int t) {
                    if (cur.steps(t) == 0) return;
                    wait(&q_empty[t], (qn[t]++ & 1) ^ 1);
                    mbar_arrive_expect_tx(&q_full[t], 3 * kBlock);
                    for (int b = 0; b < 3; ++b)
                        tma_load_3d(sm + kSmQ + (t * 3 + b) * kBlock, &map_q, b * 64, cur.h,
                                    cur.qa + cur.q0 + t * kTile, &q_full[t]);
                };
                queries(0);
                const int steps = cur.most();
                for (int i = 0; i < steps && !dead; ++i, ++step) {
                    // The next item is asked for with the last step's loads, so that no CTA holds one that another
                    // could begin (with the first step's, 2048 tokens of 32 heads take 50 instead of 41 us).
                    if (i == steps - 1) ask();
                    // ring blocks 5 step ..: K three, V two; block c takes the place of block c - 8, which
                    // for K(step) are K(step - 2)'s last and V(step - 2)'s, for V(step) K(step - 1)'s first two
                    const int row = cur.ka + i * kTile;
                    const uint32_t par = step & 1, before = ((step >> 1) & 1) ^ 1, c = 5 * step;
                    auto block = [&](uint32_t b) { return sm + kSmRing + ((c + b) % kRing) * kBlock; };
                    wait(&k_empty[par], before);
                    mbar_arrive_expect_tx(&k_full[par], 3 * kBlock);
                    tma_load_3d(block(0), &map_kv, 0, cur.h, row, &k_full[par]);
                    wait(&v_empty[par], before);
                    tma_load_3d(block(1), &map_kv, 64, cur.h, row, &k_full[par]);
                    tma_load_2d(block(2), &map_r, 0, row, &k_full[par]);
                    if (i == 0) queries(1);
                    if (step > 0) wait(&k_empty[par ^ 1], ((step - 1) >> 1) & 1);
                    if (i >= cur.masked) {  // to the checking warps, which signal v_full
                        for (int g = 0; g < 2; ++g) {
                            mbar_arrive_expect_tx(&unchecked[g][checks & 1], kBlock);
                            tma_load_3d(block(3 + g), &map_kv, kNope + 64 * g, cur.h, row, &unchecked[g][checks & 1]);
                        }
                        ++checks;
                    } else {
                        mbar_arrive_expect_tx(&v_full[par], 2 * kBlock);
                        tma_load_3d(block(3), &map_kv, kNope, cur.h, row, &v_full[par]);
                        tma_load_3d(block(4), &map_kv, kNope + 64, cur.h, row, &v_full[par]);
                        mbar_arrive(&v_full[par]);
                    }
                    if (i == steps - 1) {
                        // its queries go from DRAM into L2 while this one's last steps run
                        more = next_item(next);
                        if (more) sh.items[2] = next;
                        if (more)
                            for (int b = 0; b < 6; ++b)
                                if (next.steps(b / 3) > 0)
                                    tma_prefetch_3d(&map_q, (b % 3) * 64, next.h, next.qa + next.q0 + (b / 3) * kTile);
                    }
                }
                if (steps == 0) {
                    ask();
                    more = next_item(next);
                    if (more) sh.items[2] = next;
                }
                if (dead) break;
                cur = next;
            }
            wait(&item_empty[it & 1], ((it >> 1) & 1) ^ 1);
            if (!dead) sh.items[it & 1].valid = 0;
            mbar_arrive(&item_full[it & 1]);
        }
        __syncwarp();
    } else if (wid == 17) {
        // ---- MMA, issued by one thread.  It shares its scheduler with four softmax warps, so that
        // every instruction between two MMAs costs some twenty clocks: one wait for a whole K
        // or V tile, ahead of the wait for P, and nothing recomputed.
        if (elect_one()) {
            const uint32_t q_lo = (smem_u32(sm + kSmQ) >> 4) | (1u << 16), k_lo = (smem_u32(sm + kSmRing) >> 4) | (1u << 16),
                           v_lo = (smem_u32(sm + kSmRing) >> 4) | ((uint32_t)((kTile * 128) >> 4) << 16);
            constexpr uint32_t kStep = kBlock >> 4;  // a block, in descriptor units
            constexpr uint64_t hi = (uint64_t)kDescHi << 32;
            constexpr uint32_t idesc_x = idesc_bf16(kTile, kTile);
            constexpr uint32_t idesc_o = idesc_bf16(kTile, 64) | (1u << 16);
            uint32_t step = 0, pn0 = 0, pn1 = 0;  // steps and P tiles so far
            int qn[2] = {0, 0}, on[2] = {0, 0};
            // X_t of step n: K's ring blocks are 5 n ..
            auto scores = [&](auto t, uint32_t n) {
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < 3; ++b) {
                    const uint32_t k = k_lo + ((5 * n + b) % kRing) * kStep;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_bf16(tmem + t * kTile, hi | (q_lo + (t * 3 + b) * kStep + 2 * j), hi | (k + 2 * j), idesc_x,
                                 b + j > 0);
                }
                mma_commit(&x_full[t]);
            };
            // O_t += P_t V(step); P comes in two parts: keys 0..31 and 64..95, then the others
            auto values = [&](auto t, uint32_t pn, bool first) {
                const uint32_t v0 = v_lo + ((5 * step + 3) % kRing) * kStep, v1 = v_lo + ((5 * step + 4) % kRing) * kStep;
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    wait(&p_full[t][part], pn & 1);
                    tc_fence_after();
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int k = (j >> 1) * 4 + part * 2 + (j & 1);
                            mma_bf16_ts(tmem + kTmemO + t * kTile + b * 64, tmem + t * kTile + k * 8,
                                        hi | ((b ? v1 : v0) + 128 * k), idesc_o, !first || part + j > 0);
                        }
                }
            };
            const std::integral_constant<int, 0> t0;
            const std::integral_constant<int, 1> t1;
            for (int it = 0;; ++it) {
                const Item s = item_of(it);
                if (dead || !s.valid) break;
                const int s0 = s.steps0, s1 = s.steps1, steps = s.most();
                if (s0 > 0) wait(&q_full[0], qn[0]++ & 1);
                if (s1 > 0) wait(&q_full[1], qn[1]++ & 1);
                if (steps > 0) {
                    wait(&k_full[step & 1], (step >> 1) & 1);
                    if (s0 > 0) scores(t0, step);
                    if (s1 > 0) scores(t1, step);
                    mma_commit(&k_empty[step & 1]);
                    if (s0 == 1) mma_commit(&q_empty[0]);
                    if (s1 == 1) mma_commit(&q_empty[1]);
                    if (s0 > 0 && on[0]++ > 0) wait(&o_empty[0], on[0] & 1);
                    if (s1 > 0 && on[1]++ > 0) wait(&o_empty[1], on[1] & 1);
                }
                for (int i = 0; i < steps && !dead; ++i, ++step) {
                    const uint32_t next = step + 1;
                    wait(&v_full[step & 1], (step >> 1) & 1);
                    if (i < s0) {
                        values(t0, pn0++, i == 0);
                        if (i + 1 < steps) wait(&k_full[next & 1], (next >> 1) & 1);
                        if (i + 1 < s0) scores(t0, next);
                        else mma_commit(&o_full[0]);
                        if (i + 2 == s0) mma_commit(&q_empty[0]);
                    }
                    if (i < s1) {
                        values(t1, pn1++, i == 0);
                        mma_commit(&v_empty[step & 1]);
                        if (i + 1 < s1 && i >= s0) wait(&k_full[next & 1], (next >> 1) & 1);
                        if (i + 1 < s1) scores(t1, next);
                        else mma_commit(&o_full[1]);
                        if (i + 2 == s1) mma_commit(&q_empty[1]);
                    } else {
                        mma_commit(&v_empty[step & 1]);
                    }
                    if (i + 1 < steps) mma_commit(&k_empty[next & 1]);
                }
                item_done(it);
            }
        }
        __syncwarp();
    } else if (wid >= 18) {
        // ---- the check of V's block g in steps with masked places, between its copy and v_full
        const int g = wid - 18;
        uint32_t step = 0;
        int checks = 0;
        for (int it = 0;; ++it) {
            const Item s = item_of(it);
            if (__any_sync(0xffffffffu, dead || !s.valid)) break;
            const int steps = s.most();
            for (int i = 0; i < steps; ++i, ++step) {
                if (i < s.masked) continue;
                const uint32_t slot = (5 * step + 3 + g) % kRing;
                wait(&unchecked[g][checks & 1], (checks >> 1) & 1);
                const int rows = min(s.lk - i * kTile, kTile);  // keys of the sequence in this tile
                uint4 *v = (uint4 *)(sm + kSmRing + slot * kBlock) + lane;  // rows lane / 8 + 4 j
                for (int j = (rows - (lane >> 3) + 3) >> 2; j < kTile / 4; ++j) v[32 * j] = make_uint4(0, 0, 0, 0);
                uint32_t ones = 0;
#pragma unroll 8
                for (int j = 0; j < kTile / 4; ++j) ones |= exponent_of_ones(v[32 * j]);
                if (ones) {
                    odd[it & 1] = 1;
                    for (int j = 0; j < kTile / 4; ++j) v[32 * j] = finite_or_zero(v[32 * j]);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_full[step & 1]);
                ++checks;
            }
            __syncwarp();
            if (lane == 0) item_done(it);
        }
    } else {
        // ---- softmax of tile t: two threads own a query row, 64 keys of a step each
        const int t = wid >> 3, half = (wid >> 2) & 1, quad = wid & 3;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t tx = tmem + t * kTile + lanes, to = tmem + kTmemO + t * kTile + half * 64 + lanes;
        const float scale2 = a.scale == 0.0f ? 1.0f : fabsf(a.scale) * kLog2e;
        float *mine = &sh.half[t][half][quad * 32 + lane], *other = &sh.half[t][half ^ 1][quad * 32 + lane];
        int xn = 0, on = 0;
        for (int it = 0;; ++it) {
            std::conditional_t<SPLIT, const ITEM &, const ITEM> s = item_of(it);
            bool split = false;
            if constexpr (SPLIT) split = s.part >= 0;
            if (!named_bar_and(1 + t, 256, !dead && s.valid)) break;
            const int row = s.q0 + t * kTile + quad * 32 + lane;
            const bool real = (unsigned)row < (unsigned)s.lq;
            const int limit = !real ? 0 : a.causal ? min(s.lk, row + 1 + s.off) : s.lk;  // keys below it are seen
            float m = -INFINITY, l = 0.0f;  // m in units of x / |scale|
            const int steps = s.steps(t);
            bool gave_up = false;  // the same in both halves: decided by their votes
            for (int i = 0; i < steps; ++i, ++xn) {
                wait(&x_full[t], xn & 1);
                const bool given = dead;
                tc_fence_after();
                float x[2][32], top = -INFINITY;
                tmem_ld32(tx + 64 * half, x[0]);
                tmem_ld32(tx + 64 * half + 32, x[1]);
                tmem_ld_wait_for(x[0]);
                tmem_ld_wait_for(x[1]);
                const int left = limit - i * kTile - 64 * half;
                if (!POSITIVE) {
#pragma unroll
                    for (int j = 0; j < 64; ++j) x[j >> 5][j & 31] = x[j >> 5][j & 31] * (a.scale < 0.0f ? -1.0f : 0.0f);
                }
                if (__any_sync(0xffffffffu, left < 64)) {
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        if (j >= left) x[j >> 5][j & 31] = -INFINITY;
                }
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                    top = max3(max3(top, x[0][j], x[0][j + 1]), x[1][j], x[1][j + 1]);
                *mine = top;
                if (!named_bar_and(1 + t, 256, !given)) {
                    gave_up = true;
                    break;
                }
                top = fmaxf(top, *other);
                const bool raise = (top - m) * scale2 > kRaise;
                if (__any_sync(0xffffffffu, raise)) {
                    const float f = raise ? exp2_sfu((m - top) * scale2) : 1.0f;
                    if (raise) m = top;
                    l *= f;
                    if (i > 0) {  // X_t(i) was issued after P_t V(i-1): O_t is complete
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            float o[8];
                            tmem_ld8(to + 8 * k, o);
                            tmem_ld_wait_for(o);
                            uint32_t u[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(o[j] * f);
                            tmem_st8(to + 8 * k, u);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.0f : m * scale2;
                // P over columns of scores that both halves have read: key j of the step in column j / 2
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    uint32_t u[16];
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float e0 = exp2_sfu(fmaf(x[part][2 * j], scale2, -ref));
                        const float e1 = exp2_sfu(fmaf(x[part][2 * j + 1], scale2, -ref));
                        sum += e0 + e1;
                        u[j] = pack2(e0, e1);
                    }
                    l += sum;
                    tmem_st16(tx + 32 * half + 16 * part, u);
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(&p_full[t][part]);
                }
            }
            const int64_t out = (int64_t)(s.qa + row) * a.H + s.h;
            if (steps > 0 && !gave_up) {
                wait(&o_full[t], on & 1);
                ++on;
                tc_fence_after();
                *mine = l;
                gave_up = !named_bar_and(1 + t, 256, !dead);
                l += *other;
            }
            const float inv = gave_up ? NAN : l == 0.0f ? 1.0f : 1.0f / l;
            uint32_t w[8][4];  // the thread's 64 values of its row, eight units of 16 bytes
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float o[32];
                if (steps > 0) {
                    tmem_ld32(to + 32 * k, o);
                    tmem_ld_wait_for(o);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0.0f;
                }
                if constexpr (SPLIT) {
                    if (split && real) {
                        const int place = t * kTile + quad * 32 + lane;
                        float4 *dst = (float4 *)(p.parts[s.part].o[place] + 64 * half + 32 * k);
#pragma unroll
                        for (int j = 0; j < 8; ++j) dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                        if (half == 0 && k == 0)
                            p.stats[(int64_t)s.part * kItem + place] = {gave_up ? NAN : m * scale2, gave_up ? NAN : l};
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) w[4 * k + (j >> 2)][j & 3] = pack2(o[2 * j] * inv, o[2 * j + 1] * inv);
            }
            if (steps > 0) {
                tc_fence_before();
                mbar_arrive(&o_empty[t]);
            }
            // Eight lanes exchange their units, so that a store writes whole 128-byte lines of four rows
            // (as against 16 bytes of 32 rows: 128.3 instead of 126.0 us for 4096 tokens, 32 heads).
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                const bool up = lane & o;
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (!(u & o))
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[u][j] : w[u | o][j], o);
                            if (up) w[u][j] = got; else w[u | o][j] = got;
                        }
            }
            if (!split) {
                const int first = s.q0 + t * kTile + quad * 32 + (lane & ~7);
                __nv_bfloat16 *dst = a.o + ((int64_t)(s.qa + first) * a.H + s.h) * kHeadDim + 64 * half + 8 * (lane & 7);
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if ((unsigned)(first + r) < (unsigned)s.lq)
                        *(uint4 *)(dst + (int64_t)r * a.H * kHeadDim) = make_uint4(w[r][0], w[r][1], w[r][2], w[r][3]);
            }
            if (real && a.lse && half == 0 && !split)
                a.lse[out] = gave_up ? NAN : l == 0.0f ? -INFINITY : (m * scale2 + log2_sfu(l)) * kLn2;
            if (__any_sync(0xffffffffu, odd[it & 1])) {
                // Values that were taken out of V because they are not finite, for the rows that see them.  A key that is
                // not finite either has a score of -inf (p = 0, and 0 times the value is NaN) or makes the row NaN.
                __syncwarp();  // (other lanes have written the row)
                const int end = !real ? 0 : SPLIT ? min(limit, steps * kTile) : limit;
#pragma unroll 1
                for (int key = s.masked * kTile; key < end; ++key) {
                    const __nv_bfloat16 *v = a.kv + (int64_t)(s.ka + key) * a.kv_stride + (int64_t)s.h * kKvRow;
                    const bool by_zero = !finite_key(v, a.k_rope + (int64_t)(s.ka + key) * a.rope_stride);
#pragma unroll 1
                    for (int j = 64 * half; j < 64 * half + 64; ++j) {
                        const float u = __bfloat162float(v[kNope + j]);
                        if (fabsf(u) < INFINITY) continue;
                        if constexpr (SPLIT) {
                            if (split) {
                                p.parts[s.part].o[t * kTile + quad * 32 + lane][j] += by_zero ? NAN : u;
                                continue;
                            }
                        }
                        __nv_bfloat16 *dst = a.o + out * kHeadDim + j;
                        *dst = __float2bfloat16_rn(__bfloat162float(*dst) + (by_zero ? NAN : u));
                    }
                }
            }
            __syncwarp();
            if (lane == 0) item_done(it);
            if (gave_up) break;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (dead) {
        // A wait gave up: what this CTA had in hand becomes NaN, and copies still in flight land before
        // its memory is given up.
        for (int i = 0; i < 3; ++i) {
            const ITEM &s = sh.items[i];
            if (!s.valid) continue;
            const int first = max(s.q0, 0), rows = min(s.lq - first, kItem);
            for (int j = tid; j < rows * kHeadDim; j += kThreads) {
                const int64_t out = (int64_t)(s.qa + first + j / kHeadDim) * a.H + s.h;
                a.o[out * kHeadDim + j % kHeadDim] = __float2bfloat16_rn(NAN);
                if (a.lse && j % kHeadDim == 0) a.lse[out] = NAN;
                if constexpr (SPLIT)
                    if (s.part >= 0 && j % kHeadDim == 0) p.stats[(int64_t)s.part * kItem + j / kHeadDim] = {NAN, NAN};
            }
        }
        const long long t0 = clock64();
        while (clock64() - t0 < 100000000LL) __nanosleep(1000);
    }
    if (wid == 17) tmem_dealloc(tmem, 512);
}

// Joins the parts of an item whose keys were split, in their order: a warp per query row, four channels a lane.
constexpr int kJoinThreads = 256, kJoinRows = kJoinThreads / 32, kMaxSplits = 160;
__global__ void __launch_bounds__(kJoinThreads) latent_prefill_join_kernel(const SplitParams p) {
    __shared__ float weights[kJoinRows][kMaxSplits];
    griddep_wait();
    griddep_launch_dependents();
    const LatentPrefillArgs &a = p.a;
    const Join j = p.joins[blockIdx.y];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, row = blockIdx.x * kJoinRows + wid;
    const int rank = blockIdx.y / a.H, h = blockIdx.y - rank * a.H;
    if (row >= j.rows || j.parts <= 0) return;
    // (the record of an item that no CTA could take is whatever the workspace held)
    if (j.rows > kItem || j.parts > p.splits || j.q < 0 || j.q >= a.total_q - row) return;
    const int first = rank * a.H + h, step = p.blocks * a.H;  // places of the item's parts
    auto slot = [&](int i) { return (int64_t)(first + i * step); };
    // a part that saw nothing has no reference, and its sum is 0; NaN (which fmaxf skips) has a weight of NaN
    float top = -INFINITY, l = 0.0f;
    for (int i = lane; i < j.parts; i += 32) top = fmaxf(top, p.stats[slot(i) * kItem + row].m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    for (int i = lane; i < j.parts; i += 32) {
        const Stat s = p.stats[slot(i) * kItem + row];
        const float w = s.m == -INFINITY ? 0.0f : exp2_sfu(s.m - top);
        weights[wid][i] = w;
        l += w * s.l;
    }
    l = warp_sum(l);
    __syncwarp();
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float *src = p.parts[first].o[row] + 4 * lane;
#pragma unroll 8
    for (int i = 0; i < j.parts; ++i, src += (int64_t)step * kItem * kHeadDim) {
        const float4 u = *(const float4 *)src;
        const float w = weights[wid][i];
        o.x += w * u.x, o.y += w * u.y, o.z += w * u.z, o.w += w * u.w;
    }
    const float inv = l == 0.0f ? 1.0f : 1.0f / l;
    const int64_t out = (int64_t)(j.q + row) * a.H + h;
    *(uint2 *)(a.o + out * kHeadDim + 4 * lane) = make_uint2(pack2(o.x * inv, o.y * inv), pack2(o.z * inv, o.w * inv));
    if (a.lse && lane == 0) a.lse[out] = l == 0.0f ? -INFINITY : (top + log2_sfu(l)) * kLn2;
}

// Blocks of queries at most: a sequence's last one may hold a single query.
inline int64_t block_bound(int n_seqs, int64_t total_q) {
    return (total_q + (kItem - 1) * std::min<int64_t>(n_seqs, total_q)) / kItem;
}

// Parts that an item's keys are split into at most, from what the host knows: the waves of parts times
// their steps, to which a part's start and outputs add about three and the join five.  8 heads, 64
// queries and 2112 keys: 36 us whole, 15 us split; 16 heads, 512 queries behind 32768 keys: 421 and
// 131 us; 1 head, 512 behind 65536: 820 and 41 us.  1024 queries and keys of 8 heads, which the
// rule leaves whole: 20.8 and 21.9 us.  The host has no lengths, so that a long sequence among short
// ones is left whole: 16 queries behind 131072 keys, 8 heads, 112 us alone and 1780 us beside 15 sequences
// of 256 keys.
inline int splits_for(int n_seqs, int64_t total_q, int64_t total_k, int H) {
    const int64_t items = block_bound(n_seqs, total_q) * H, steps = (total_k / n_seqs + kTile - 1) / kTile;
    const int sms = sm_count();
    // (below SPLIT_KEYS no caller has a workspace, whatever the costs say)
    if (items == 0 || items > 2 * sms || steps < kSplitSteps || total_k < KDA_LATENT_PREFILL_SPLIT_KEYS) return 1;
    const int64_t most = std::min<int64_t>({4 * sms / items, (steps + kMinSteps - 1) / kMinSteps, kMaxSplits});
    int best = 1;
    double least = 0.85 * ((items + sms - 1) / sms) * (steps + 3.0);
    for (int n = 2; n <= most; ++n) {
        const double cost = (double)((items * n + sms - 1) / sms) * ((double)steps / n + 3.0) + 5.0;
        if (cost < least) best = n, least = cost;
    }
    return best;
}

struct Layout {
    size_t joins, stats, parts, total;
};
inline Layout layout(int64_t items, int splits) {
    Layout l;
    l.joins = 0;
    l.stats = align_up((size_t)items * sizeof(Join), 256);
    l.parts = l.stats + align_up((size_t)items * splits * kItem * sizeof(Stat), 256);
    l.total = l.parts + (size_t)items * splits * sizeof(Part);
    return l;
}

}  // namespace

int64_t latent_prefill_items(int n_seqs, int64_t total_q, int H) { return block_bound(n_seqs, total_q) * H; }

size_t latent_prefill_workspace_bytes(int n_seqs, int64_t total_q, int64_t total_k, int H) {
    const int splits = splits_for(n_seqs, total_q, total_k, H);
    return splits == 1 ? 0 : layout(block_bound(n_seqs, total_q) * H, splits).total;
}

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
    const int64_t items = latent_prefill_items(a.n_seqs, a.total_q, a.H);
    const int splits = splits_for(a.n_seqs, a.total_q, a.total_k, a.H);
    auto launch = [&](auto kernel, const auto &p) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
        return e != cudaSuccess ? e
                                : launch_dependent(kernel, dim3((unsigned)(items * splits)), dim3(kThreads), kSmemBytes, stream,
                                                   map_q, map_kv, map_r, p);
    };
    cudaError_t e;
    if (splits == 1) {
        const PrefillParams p{a};
        e = a.scale > 0.0f ? launch(latent_prefill_kernel<true, false>, p) : launch(latent_prefill_kernel<false, false>, p);
    } else {
        const Layout l = layout(items, splits);
        uint8_t *ws = (uint8_t *)a.workspace;
        const SplitParams p{{a}, splits, (int)(items / a.H), (Part *)(ws + l.parts), (Stat *)(ws + l.stats), (Join *)(ws + l.joins)};
        e = a.scale > 0.0f ? launch(latent_prefill_kernel<true, true>, p) : launch(latent_prefill_kernel<false, true>, p);
        if (e == cudaSuccess)
            e = launch_dependent(latent_prefill_join_kernel, dim3(kItem / kJoinRows, (unsigned)items), dim3(kJoinThreads), 0,
                                 stream, p);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kda
