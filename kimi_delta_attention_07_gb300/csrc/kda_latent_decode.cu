// Absorbed latent attention over the paged cache: per query row (request n,
// new token s, head h), with cached rows c_p of 576 values (latent 512, key 64),
//   x_p = scale * q . c_p,   o = sum_p softmax(x)_p c_p[:512].
//
// All heads of a request read the same rows, so the kernel is bound by
// streaming the cache once (1152 bytes a token) as long as the products, 2 * 1088
// operations a token and query row, keep up: 32 rows want 60 operations a byte,
// which takes the tensor cores.
//
// Orientation: tokens are the M axis of both products' first operand,
//   X^T [128 tokens x 32 rows]   = C [128 x 576] . Q^T         (per tile)
//   O^T [512 x 32 rows]         += C[:, :512]^T . P^T [128 x 32]
// so that the few query rows are the N axis (32, where M would be padded to 128)
// and one shared-memory tile of the cache, as TMA laid it down, serves as the
// K-major operand of the first product and as the MN-major operand of the
// second.  A softmax thread owns one token (TMEM lane) and holds its 32 rows'
// scores in registers; p goes through shared memory as the MN-major B operand.
//
// Running maximum: rows keep a reference that is only raised (and O^T in TMEM
// rescaled) when some score passes it by 2^8, which is decided by one vote a
// tile; p is then at most 2^8, and p, its sum and O share the reference, so
// that the quotient is unchanged.  Sums are fp32 per thread, joined at the end.
//
// Work split: the tiles of all requests, in order, are cut evenly into one
// range per CTA (a persistent CTA per SM; rows beyond 32 take further CTAs over
// the same tiles).  A request inside one range is finished there; one that
// crosses ranges leaves (O, max, sum) parts in the workspace, which a second,
// dependent kernel joins in range order.
//
// Warps: 0..3 softmax and epilogue, 4 TMA, 5 MMA.
#include <algorithm>

#include "kda_attn.cuh"

namespace kda {

using namespace tc;

namespace {

constexpr int kTile = 128;   // tokens per tile
constexpr int kRows = 32;    // query rows per CTA
constexpr int kPairs = 5;    // ring slots of two 64-column blocks (four per tile)
constexpr int kThreads = 192;
constexpr uint32_t kBlock = kTile * 128;  // one 64-column block of a tile
constexpr float kRaise = 8.0f;            // log2 by which a score may pass its row's reference

// shared memory (from a 1024-byte boundary)
constexpr uint32_t kSmQ = 0;                               // [9][32 rows][128 B]
constexpr uint32_t kSmP = kSmQ + 9 * kRows * 128;          // [128 tokens][64 B]
constexpr uint32_t kSmRope = kSmP + kTile * 64;            // one block
constexpr uint32_t kSmPair = kSmRope + kBlock;             // kPairs x two blocks
constexpr uint32_t kSmEnd = kSmPair + kPairs * 2 * kBlock;
constexpr uint32_t kSmemBytes = kSmEnd + 1024;             // + alignment of the base

constexpr uint32_t kTmemCols = 256;  // O^T: 4 x 32, X^T: 32
constexpr uint32_t kTmemX = 128;

struct Part {  // of a request that crosses ranges
    float o[kRows][kLatent];
    float m[kRows], l[kRows];
};
struct Join {  // written by the second range of a crossing request
    int32_t n, first, last, pad;  // ranges first..last hold its parts; n < 0: none
};

struct Grid {
    int row_blocks, ranges;
};
inline Grid decode_grid(int S, int H) {
    Grid g;
    g.row_blocks = (S * H + kRows - 1) / kRows;
    g.ranges = std::max(1, sm_count() / g.row_blocks);
    return g;
}

struct DecodeParams {
    LatentDecodeArgs a;
    int row_blocks, ranges;
    Part *parts;  // [range][row block][2]: begun before the range / begun in it
    Join *joins;  // [range]
};

__device__ __forceinline__ int tiles_of(const LatentDecodeArgs &a, int len) {
    // an empty request (or one that cannot be read) still has a tile: its outputs are written
    const bool ok = len >= 0 && (int64_t)len <= ((int64_t)a.max_pages << a.page_shift);
    return ok && len > 0 ? (int)(((int64_t)len + kTile - 1) / kTile) : 1;
}

// One request's share of a range.
struct Segment {
    int n, len, tile0, tiles, total;  // tiles [tile0, tile0 + tiles) of the request's `total`
    bool ok;
    __device__ __forceinline__ bool whole() const { return tiles == total; }
};

// Walks the range's requests; every role keeps its own.
struct Walk {
    const LatentDecodeArgs &a;
    int n, off;
    int64_t left;
    __device__ __forceinline__ bool next(Segment &s) {
        if (left <= 0) return false;
        s.n = n;
        s.len = a.seq_lens[n];
        s.ok = s.len >= 0 && (int64_t)s.len <= ((int64_t)a.max_pages << a.page_shift);
        s.total = tiles_of(a, s.len);
        if (!s.ok) s.len = 0;
        s.tile0 = off;
        s.tiles = (int)min((int64_t)(s.total - off), left);
        left -= s.tiles;
        ++n;
        off = 0;
        return true;
    }
};

__global__ void __launch_bounds__(kThreads, 1)
    latent_decode_kernel(const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_c, const DecodeParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    __shared__ uint64_t full_pair[kPairs], empty_pair[kPairs], full_rope, full_q, x_full, p_full, o_full, o_empty;
    __shared__ uint32_t tmem_base;
    __shared__ int64_t piece[kThreads], total_tiles;
    __shared__ int start_n, start_off;
    __shared__ float sh_m[4][kRows], sh_l[4][kRows];
    __shared__ volatile int dead;

    const LatentDecodeArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int rb = blockIdx.x % p.row_blocks, range = blockIdx.x / p.row_blocks;

    if (tid == 0) {
        for (int i = 0; i < kPairs; ++i) mbar_init(&full_pair[i], 1), mbar_init(&empty_pair[i], 1);
        mbar_init(&full_rope, 1);
        mbar_init(&full_q, 1);
        mbar_init(&x_full, 1);
        mbar_init(&p_full, 128);
        mbar_init(&o_full, 1);
        mbar_init(&o_empty, 128);
        fence_mbar_init();
        dead = 0;
    }
    if (wid == 5) tmem_alloc(&tmem_base, kTmemCols);
    griddep_wait();
    griddep_launch_dependents();

    // this range's first request: sums over contiguous pieces of the requests,
    // then a walk inside the piece where the range begins
    {
        const int per = (a.n_seqs + kThreads - 1) / kThreads;
        const int n0 = min(tid * per, a.n_seqs), n1 = min(n0 + per, a.n_seqs);
        int64_t mine = 0;
        for (int n = n0; n < n1; ++n) mine += tiles_of(a, a.seq_lens[n]);
        piece[tid] = mine;
        __syncthreads();
        int64_t before = 0, total = 0;
        for (int i = 0; i < kThreads; ++i) {
            if (i < tid) before += piece[i];
            total += piece[i];
        }
        if (tid == 0) total_tiles = total;
        const int64_t ranges = min((int64_t)p.ranges, total);  // none is empty
        const int64_t begin = range < ranges ? total * range / ranges : total;
        if (range >= ranges && rb == 0 && tid == 0) p.joins[range] = {-1, 0, 0, 0};
        if (begin >= before && begin < before + mine) {
            int n = n0;
            for (;; ++n) {
                const int t = tiles_of(a, a.seq_lens[n]);
                if (begin < before + t) break;
                before += t;
            }
            start_n = n;
            start_off = (int)(begin - before);
            // the range that follows a request's first one names the parts to join
            Join j = {-1, 0, 0, 0};
            if (start_off > 0) {
                const int64_t t0 = before, t1 = before + tiles_of(a, a.seq_lens[n]) - 1;
                // the range that holds tile t: the last r with total * r / ranges <= t
                const int first = (int)(((t0 + 1) * ranges + total - 1) / total) - 1;
                const int last = (int)(((t1 + 1) * ranges + total - 1) / total) - 1;
                if (first == range - 1) j = {n, first, last, 0};
            }
            if (rb == 0) p.joins[range] = j;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int64_t ranges = min((int64_t)p.ranges, total_tiles);
    Walk walk{a, start_n, start_off,
              range < ranges ? total_tiles * (range + 1) / ranges - total_tiles * range / ranges : 0};
    // a bounded wait; once one has given up, none waits any more
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!dead && !mbar_wait(bar, parity)) dead = 1;
    };
    const uint32_t tmem = tmem_base;
    Segment s;

    if (wid == 4) {
        // ---- TMA: Q per request, then per tile pair 0, the key block, pairs 1..3
        const int box = min(1 << a.page_shift, kTile);
        const int per_tile = kTile / box;  // pages of a tile
        const int beyond = (int)(a.n_pages << a.page_shift);  // a row outside: reads zeros
        int pair = 0, phase = 0, rope_phase = 0;
        bool first_tile = true;
        while (!dead && walk.next(s)) {
            const int32_t *table = a.block_table + (int64_t)s.n * a.max_pages;
            auto row_of = [&](int tile) {  // this lane's page of the tile, as a cache row
                const int64_t pos = (int64_t)tile * kTile + lane * box;
                if (lane >= per_tile || pos >= s.len) return beyond;
                const int id = table[pos >> a.page_shift];
                if (id < 0 || id >= a.n_pages) return beyond;
                return (id << a.page_shift) + (int)(pos & ((1 << a.page_shift) - 1));
            };
            int next_row = row_of(s.tile0);
            for (int i = 0; i < s.tiles && !dead; ++i) {
                const int tile = s.tile0 + i, row = next_row;
                if (i + 1 < s.tiles) next_row = row_of(tile + 1);
                const int held = min(per_tile, (s.len - tile * kTile + box - 1) / box);  // pages with tokens
                const int boxes = max(held, 0);
                auto load_pair = [&](int k) {
                    wait(&empty_pair[pair], phase ^ 1);
                    if (lane == 0) mbar_arrive_expect_tx(&full_pair[pair], boxes * 2 * box * 128);
                    __syncwarp();
                    const int half = lane & 1, j = lane >> 1;
                    const int r = __shfl_sync(0xffffffffu, row, j);
                    if (j < boxes)
                        tma_load_2d(sm + kSmPair + pair * 2 * kBlock + half * kBlock + j * box * 128, &map_c,
                                    (2 * k + half) * 64, r, &full_pair[pair]);
                    if (++pair == kPairs) pair = 0, phase ^= 1;
                };
                load_pair(0);
                // the first product of the tile before has read the key block and, where
                // the request changes, its queries
                if (!first_tile) wait(&x_full, rope_phase), rope_phase ^= 1;
                first_tile = false;
                if (i == 0) {
                    if (lane == 0) mbar_arrive_expect_tx(&full_q, 9 * kRows * 128);
                    __syncwarp();
                    if (lane < 9)
                        tma_load_2d(sm + kSmQ + lane * kRows * 128, &map_q, lane * 64,
                                    s.n * (a.S * a.H) + rb * kRows, &full_q);
                }
                if (lane == 0) mbar_arrive_expect_tx(&full_rope, boxes * box * 128);
                __syncwarp();
                if (lane < boxes)
                    tma_load_2d(sm + kSmRope + lane * box * 128, &map_c, kLatent, row, &full_rope);
                for (int k = 1; k < 4; ++k) load_pair(k);
            }
        }
    } else if (wid == 5) {
        // ---- MMA, issued by one thread, in order: X(i), then P.C(i)
        if (lane == 0) {
            int pair = 0, phase = 0, tile_phase = 0, seg_phase = 0;
            bool first_segment = true;
            const uint32_t q0 = smem_u32(sm + kSmQ), pair0 = smem_u32(sm + kSmPair);
            while (!dead && walk.next(s)) {
                wait(&full_q, seg_phase);
                for (int i = 0; i < s.tiles && !dead; ++i) {
                    int pr = pair, ph = phase;
                    for (int k = 0; k < 4; ++k) {
                        wait(&full_pair[pr], ph);
                        tc_fence_after();
                        for (int half = 0; half < 2; ++half)
                            mma_tile<128, kRows, 64, kTile, kRows>(
                                tmem + kTmemX, pair0 + pr * 2 * kBlock + half * kBlock,
                                q0 + (2 * k + half) * kRows * 128, k + half > 0);
                        if (++pr == kPairs) pr = 0, ph ^= 1;
                        if (k == 0) {
                            wait(&full_rope, tile_phase);
                            tc_fence_after();
                            mma_tile<128, kRows, 64, kTile, kRows>(tmem + kTmemX, smem_u32(sm + kSmRope),
                                                                   q0 + 8 * kRows * 128, true);
                        }
                    }
                    mma_commit(&x_full);
                    wait(&p_full, tile_phase);
                    if (i == 0 && !first_segment) wait(&o_empty, seg_phase ^ 1);
                    tc_fence_after();
                    for (int k = 0; k < 4; ++k) {
                        mma_tile_n32<128, kTile, kTile, true>(tmem + k * 32, pair0 + pair * 2 * kBlock,
                                                              smem_u32(sm + kSmP), i > 0);
                        mma_commit(&empty_pair[pair]);
                        if (++pair == kPairs) pair = 0, phase ^= 1;
                    }
                    tile_phase ^= 1;
                }
                mma_commit(&o_full);
                seg_phase ^= 1;
                first_segment = false;
            }
        }
        __syncwarp();
    } else {
        // ---- softmax: thread = token of the tile, registers = the 32 query rows
        const Walk again = walk;
        const uint32_t lanes = (uint32_t)(wid * 32) << 16;
        const float scale2 = a.scale * kLog2e;
        const int rows = min(kRows, a.S * a.H - rb * kRows);
        int pair = 0, tile_phase = 0, seg_phase = 0;
        bool gave_up = false;  // the same in all four warps: decided by their votes
        while (!gave_up && walk.next(s)) {
            float m[kRows], l[kRows];
#pragma unroll
            for (int c = 0; c < kRows; ++c) m[c] = -INFINITY, l[c] = 0.0f;
            bool bad = !s.ok;
            for (int i = 0; i < s.tiles; ++i) {
                const int64_t pos = (int64_t)(s.tile0 + i) * kTile + tid;
                if (pos < s.len) {
                    const int id = a.block_table[(int64_t)s.n * a.max_pages + (pos >> a.page_shift)];
                    bad |= id < 0 || id >= a.n_pages;
                }
                wait(&x_full, tile_phase);
                tc_fence_after();
                float x[kRows];
                tmem_ld32(tmem + kTmemX + lanes, x);
                tmem_ld_wait();
                const int64_t tile_end = (int64_t)(s.tile0 + i + 1) * kTile;
                if (tile_end > s.len - a.S + 1) {
                    // row r (new token r / H) sees positions below len - S + 1 + r / H
#pragma unroll
                    for (int c = 0; c < kRows; ++c) {
                        const int64_t limit = s.len - a.S + 1 + (rb * kRows + c) / a.H;
                        x[c] = pos < limit ? x[c] * scale2 : -INFINITY;
                    }
                    if (pos >= s.len) {
                        // no token: its row in shared memory may hold anything, and 0 times that has to be 0
                        int pr = pair;
                        for (int k = 0; k < 4; ++k) {
                            for (int half = 0; half < 2; ++half) {
                                uint4 *r = (uint4 *)(sm + kSmPair + pr * 2 * kBlock + half * kBlock + tid * 128);
#pragma unroll
                                for (int j = 0; j < 8; ++j) r[j] = make_uint4(0, 0, 0, 0);
                            }
                            if (++pr == kPairs) pr = 0;
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < kRows; ++c) x[c] *= scale2;
                }
                pair = (pair + 4) % kPairs;
                float over = -INFINITY;  // fmaxf skips the NaN of -inf - -inf
#pragma unroll
                for (int c = 0; c < kRows; ++c) over = fmaxf(over, x[c] - m[c]);
                const bool lost = dead;
                if (!named_bar_and(1, 128, !(over > kRaise) && !lost)) {
                    if (!named_bar_and(1, 128, !lost)) {
                        gave_up = true;
                        break;
                    }
                    float t[kRows];
#pragma unroll
                    for (int c = 0; c < kRows; ++c) t[c] = x[c];
                    sh_m[wid][lane] = reduce_columns(t, [](float u, float v) { return fmaxf(u, v); });
                    named_bar_sync(1, 128);
                    float f[kRows];
#pragma unroll
                    for (int c = 0; c < kRows; ++c) {
                        const float top = fmaxf(fmaxf(fmaxf(sh_m[0][c], sh_m[1][c]), fmaxf(sh_m[2][c], sh_m[3][c])), m[c]);
                        f[c] = top == -INFINITY ? 1.0f : exp2_sfu(m[c] - top);
                        m[c] = top;
                        l[c] *= f[c];
                    }
                    if (i > 0) {  // the second product of the tile before is done: X(i) was issued after it
                        for (int k = 0; k < 4; ++k) {
                            float o[kRows];
                            tmem_ld32(tmem + k * 32 + lanes, o);
                            tmem_ld_wait();
                            uint32_t u[kRows];
#pragma unroll
                            for (int c = 0; c < kRows; ++c) u[c] = __float_as_uint(o[c] * f[c]);
                            tmem_st32(tmem + k * 32 + lanes, u);
                        }
                        tmem_st_wait();
                    }
                    named_bar_sync(1, 128);  // sh_m is read before it is written again
                }
#pragma unroll
                for (int c = 0; c < kRows; ++c) {
                    x[c] = exp2_sfu(x[c] - (m[c] == -INFINITY ? 0.0f : m[c]));
                    l[c] += x[c];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 v = make_uint4(pack2(x[8 * j], x[8 * j + 1]), pack2(x[8 * j + 2], x[8 * j + 3]),
                                               pack2(x[8 * j + 4], x[8 * j + 5]), pack2(x[8 * j + 6], x[8 * j + 7]));
                    *(uint4 *)(sm + kSmP + sw64_off(tid, 8 * j)) = v;
                }
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(&p_full);
                tile_phase ^= 1;
            }
            if (gave_up) break;
            // ---- the request's part of this range is done
            sh_l[wid][lane] = reduce_columns(l, [](float u, float v) { return u + v; });
            const bool fine = named_bar_and(1, 128, !bad);
            wait(&o_full, seg_phase);
            seg_phase ^= 1;
            tc_fence_after();
            const int64_t row0 = (int64_t)s.n * a.S * a.H + rb * kRows;
            Part *part = p.parts + ((int64_t)range * p.row_blocks + rb) * 2 + (s.tile0 == 0 ? 1 : 0);
            float lt[kRows];
#pragma unroll
            for (int c = 0; c < kRows; ++c) {
                lt[c] = sh_l[0][c] + sh_l[1][c] + sh_l[2][c] + sh_l[3][c];
                if (!fine) lt[c] = NAN;
            }
            if (tid < rows) {
                float mt = 0.0f, ls = 0.0f;
#pragma unroll
                for (int c = 0; c < kRows; ++c)
                    if (c == tid) mt = m[c], ls = lt[c];
                if (!s.whole()) part->m[tid] = mt, part->l[tid] = ls;
                else if (a.lse) a.lse[row0 + tid] = mt == -INFINITY && ls == 0.0f ? -INFINITY : (mt + log2_sfu(ls)) * kLn2;
            }
#pragma unroll
            for (int c = 0; c < kRows; ++c) lt[c] = lt[c] == 0.0f ? 1.0f : 1.0f / lt[c];
            for (int k = 0; k < 4; ++k) {
                float o[kRows];
                tmem_ld32(tmem + k * 32 + lanes, o);
                tmem_ld_wait();
                const int d = k * 128 + tid;
                if (s.whole()) {
#pragma unroll
                    for (int c = 0; c < kRows; ++c)
                        if (c < rows) a.o[(row0 + c) * kLatent + d] = __float2bfloat16_rn(o[c] * lt[c]);
                } else {
#pragma unroll
                    for (int c = 0; c < kRows; ++c)
                        if (c < rows) part->o[c][d] = o[c];
                }
            }
            tc_fence_before();
            mbar_arrive(&o_empty);
            named_bar_sync(1, 128);  // sh_l is read before the next request writes it
        }
        if (!named_bar_and(1, 128, !dead)) {
            // a wait gave up: the range's outputs are NaN
            Walk w = again;
            while (w.next(s)) {
                const int64_t row0 = (int64_t)s.n * a.S * a.H + rb * kRows;
                Part *part = p.parts + ((int64_t)range * p.row_blocks + rb) * 2 + (s.tile0 == 0 ? 1 : 0);
                for (int c = 0; c < rows; ++c) {
                    if (!s.whole()) {
                        if (tid == 0) part->m[c] = NAN, part->l[c] = NAN;
                        continue;
                    }
                    for (int d = tid; d < kLatent; d += 128) a.o[(row0 + c) * kLatent + d] = __float2bfloat16_rn(NAN);
                    if (a.lse && tid == 0) a.lse[row0 + c] = NAN;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (dead) {  // let copies still in flight land before the CTA's memory is given up
        const long long t0 = clock64();
        while (clock64() - t0 < 100000000LL) __nanosleep(1000);
    }
    if (wid == 5) tmem_dealloc(tmem, kTmemCols);
}

// Joins the parts of a request that crosses ranges, in range order; a thread
// owns four values of a row.
constexpr int kJoinRows = 4;
__global__ void __launch_bounds__(128) latent_decode_join_kernel(const DecodeParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const LatentDecodeArgs &a = p.a;
    const int range = blockIdx.x / p.row_blocks, rb = blockIdx.x % p.row_blocks;
    const Join j = p.joins[range];
    if (j.n < 0) return;
    for (int c = blockIdx.y * kJoinRows; c < (int)(blockIdx.y + 1) * kJoinRows; ++c) {
        const int row = rb * kRows + c;
        if (row >= a.S * a.H) return;
        auto part = [&](int r) { return p.parts + ((int64_t)r * p.row_blocks + rb) * 2 + (r == j.first ? 1 : 0); };
        float top = -INFINITY;
        bool nan = false;
        for (int r = j.first; r <= j.last; ++r) {
            const float m = part(r)->m[c], l = part(r)->l[c];
            nan |= !(l == l) || !(m == m);
            top = fmaxf(top, m);
        }
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float l = 0.0f;
        for (int r = j.first; r <= j.last; ++r) {
            const float m = part(r)->m[c];
            const float w = m == -INFINITY ? 0.0f : exp2_sfu(m - top);
            const float4 v = *(const float4 *)&part(r)->o[c][4 * threadIdx.x];
            if (m != -INFINITY) {
                l += w * part(r)->l[c];
                o.x += w * v.x, o.y += w * v.y, o.z += w * v.z, o.w += w * v.w;
            }
        }
        const float inv = nan ? NAN : l == 0.0f ? 1.0f : 1.0f / l;
        const int64_t out = (int64_t)j.n * a.S * a.H + row;
        uint2 u;
        u.x = pack2(o.x * inv, o.y * inv);
        u.y = pack2(o.z * inv, o.w * inv);
        *(uint2 *)(a.o + out * kLatent + 4 * threadIdx.x) = u;
        if (a.lse && threadIdx.x == 0)
            a.lse[out] = nan ? NAN : top == -INFINITY ? -INFINITY : (top + log2_sfu(l)) * kLn2;
    }
}

inline size_t joins_bytes(const Grid &g) { return align_up((size_t)g.ranges * sizeof(Join), 256); }

}  // namespace

size_t latent_decode_workspace_bytes(int n_seqs, int S, int H) {
    const Grid g = decode_grid(S, H);
    return joins_bytes(g) + (size_t)g.ranges * g.row_blocks * 2 * sizeof(Part);
}

cudaError_t launch_latent_decode(const LatentDecodeArgs &a, cudaStream_t stream) {
    const Grid g = decode_grid(a.S, a.H);
    DecodeParams p{a, g.row_blocks, g.ranges, nullptr, (Join *)a.workspace};
    p.parts = (Part *)((uint8_t *)a.workspace + joins_bytes(g));
    CUtensorMap map_q, map_c;
    const int box = std::min(1 << a.page_shift, kTile);
    if (!encode_rows64(&map_q, a.q, kLatentRow, (int64_t)a.n_seqs * a.S * a.H, kLatentRow, kRows) ||
        !encode_rows64(&map_c, a.cache, kLatentRow, a.n_pages << a.page_shift, kLatentRow, box))
        return cudaErrorUnknown;
    cudaError_t e = cudaFuncSetAttribute(latent_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    e = launch_dependent(latent_decode_kernel, dim3(g.ranges * g.row_blocks), dim3(kThreads), kSmemBytes,
                         stream, map_q, map_c, p);
    if (e != cudaSuccess) return e;
    e = launch_dependent(latent_decode_join_kernel, dim3(g.ranges * g.row_blocks, kRows / kJoinRows), dim3(128),
                         0, stream, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kda
