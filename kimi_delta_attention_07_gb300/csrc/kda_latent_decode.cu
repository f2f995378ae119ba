// Absorbed latent attention over the paged cache: per query row (request n,
// new token s, head h), with cached rows c_p of 576 values (latent 512, key 64),
//   x_p = scale * q . c_p,   o = sum_p softmax(x)_p c_p[:512].
//
// All heads of a request read the same rows, so the kernel is bound by
// streaming the cache once (1152 bytes a token) as long as the products, 2 * 1088
// operations a token and query row, keep up: 32 rows want 60 operations a byte,
// which takes the tensor cores.
//
// Orientation: tokens are the M axis of the first product and the cache is the
// first operand of both,
//   X^T [64 (48 used) tokens x 32 rows] = C [64 x 576] . Q^T      (per tile)
//   O^T [512 x 32 rows]                += C[:, :512]^T . P^T [48 x 32]
// so that the few query rows are the N axis (as M they would be padded to 64 or
// 128) and one shared-memory tile of the cache, as TMA laid it down, serves as
// the K-major operand of the first product and as the MN-major operand of the
// second.  The scores of a tile lie in 16 TMEM lanes a warp and are read as
// accumulator fragments, 16 a thread; p goes through shared memory as the
// MN-major B operand.
//
// Loads: DRAM wants whole rows.  Loading the cache by blocks of 64 columns (a
// GEMM's K-blocks) reached 3.8 to 5.7 TB/s in a load-only kernel, whole rows of
// 16 tokens in one copy 6.8 TB/s once 72 KB an SM are in flight.  So a copy is
// 16 tokens (they are in one page, whatever its size), laid down by a 4-D map as
// [2 groups of 8 tokens][9 blocks][8 rows][128 B]: a swizzle atom per (group,
// block), 9216 bytes between groups, which both operand descriptors can step.
//
// Tiles of 48 tokens: a tile stays in shared memory until its second product is
// done, which is about 1.2 us after it has arrived (at 44 bytes a ns); three
// tiles of 48 keep more in flight (90 KB) than two of 64 (68 KB).  The first
// product's M is 64: its last 16 rows are whatever follows in the ring.  256
// requests of 512 to 4096 tokens, 32 heads (697 MB): 123 us, 5.7 TB/s; with the
// products cut to a ninth and a quarter, so that little but the loads is left, 118 us.  With 64
// query rows a CTA the queries leave room for 128 tokens, as two tiles of 64 (no
// row of the first product is wasted; four tiles of 32 are 8 to 15 % slower); p
// then takes the place of the tile's positional block, which the first product
// has read.  2 requests of 231k tokens in all, 64 rows: 65 us, 40 of them at 6.7
// TB/s between the first tile's arrival and the last one's.
//
// Running maximum: a row keeps a reference that is only raised (and its column of
// O^T in TMEM rescaled) when one of its scores passes it by 2^8; whether any row's
// did is decided by one vote a tile.  p is then at most 2^8, and p, its sum and O
// share the reference, so that the quotient is unchanged.  Sums are fp32 per thread, joined at the end.
//
// Work split: the tiles of all requests, in order, are cut evenly into one
// range per CTA (a persistent CTA per SM; query rows beyond 32, or 64 where much
// is read, take further CTAs over the same tiles).  A request inside one range is
// finished there; one that crosses ranges leaves (O, max, sum) parts in the
// workspace, which a second, dependent kernel joins in range order.
//
// Warps: 0 TMA, 1 first products, 2 second products (one warp that polled for both
// took 135 us where two take 129), 3 the join's records, 4..7 softmax (16 tokens of the tile each: the
// last one has none of 48), rescaling and epilogue.
#include <algorithm>

#include "kda_attn.cuh"
#include "kda_latent_split.cuh"

namespace kda {

using namespace tc;

namespace {

constexpr int kCopy = 16;   // tokens per copy
constexpr int kThreads = 256;
constexpr uint32_t kGroup = 9 * 1024;        // 8 tokens
constexpr uint32_t kCopyBytes = 2 * kGroup;
constexpr float kRaise = 8.0f;  // log2 by which a score may pass its row's reference

// What depends on the query rows per CTA, 32 or 64.
template <int ROWS>
struct Cfg {
    static constexpr int kCopies = ROWS == 32 ? 3 : 4;  // copies in a tile
    static constexpr int kTile = kCopies * kCopy;
    static constexpr int kSlots = ROWS == 32 ? 3 : 2;  // tiles in the ring
    static constexpr bool kOwnP = ROWS == 32;  // two P of their own, else P over the tile's positional block
    // shared memory (from a 1024-byte boundary); the ring comes first, so that the
    // 16 rows which a first product of 48 tokens reads past its tile are inside
    static constexpr uint32_t kTileBytes = kCopies * kCopyBytes;
    static constexpr uint32_t kPBytes = 64 * ROWS * 2;              // [64 tokens][ROWS]
    static constexpr uint32_t kSmQ = kSlots * kTileBytes;           // [9][ROWS][128 B]
    static constexpr uint32_t kSmP = kSmQ + 9 * ROWS * 128;         // two P
    static constexpr uint32_t kSmemBytes = kSmP + (kOwnP ? 2 * kPBytes : 0) + 1024;  // + alignment of the base
    static_assert(9 * ROWS * 128 >= 2 * kGroup, "rows past the last tile");
    static constexpr uint32_t kTmemX = 4 * ROWS;  // O^T: 4 x ROWS columns, then X^T: 2 x ROWS
    static constexpr uint32_t kTmemCols = 8 * ROWS;
};

// Operand descriptors of a tile (128-byte swizzle, 8-token groups kGroup apart):
// K-major for block b (64 columns) and step k of 16 columns; MN-major for
// columns 128 b.. and step k of 16 tokens, 64-column blocks 1024 bytes apart.
constexpr uint32_t kTileDescHi = (kGroup >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t tile_desc_k(uint32_t tile, int b, int k) {
    return ((uint64_t)kTileDescHi << 32) | (((tile & 0x3FFFFu) >> 4) + b * 64 + k * 2) | (1u << 16);
}
__device__ __forceinline__ uint64_t tile_desc_mn(uint32_t tile, int b, int k) {
    return ((uint64_t)kTileDescHi << 32) | (((tile & 0x3FFFFu) >> 4) + b * 128 + k * (kCopyBytes >> 4)) | (64u << 16);
}

// P as B operand, MN-major, and the place of a token's row in it: an own buffer of rows of 64 bytes
// (64-byte swizzle), or the last block of the tile, which the second product does not read.
__device__ __forceinline__ uint64_t own_p_desc(uint32_t p, int k) {
    return ((uint64_t)kDescHiSw64 << 32) | (((p & 0x3FFFFu) >> 4) + k * (16 * 64 >> 4));
}
__device__ __forceinline__ uint64_t tile_p_desc(uint32_t tile, int k) {
    return ((uint64_t)kTileDescHi << 32) | (((tile & 0x3FFFFu) >> 4) + 8 * 64 + k * (kCopyBytes >> 4)) | (64u << 16);
}
__device__ __forceinline__ uint32_t tile_p_off(int token, int row) {
    return (token >> 3) * kGroup + 8 * 1024 + sw128_off(token & 7, row, 64);
}

template <int ROWS>
struct Part {  // of a request that crosses ranges
    float o[ROWS][kLatent];
};
struct Stat {  // and its rows' reference and sum
    float m, l;
};
struct Grid {
    int row_blocks, ranges;
};
inline Grid decode_grid(int S, int H, int rows) {
    Grid g;
    g.row_blocks = (S * H + rows - 1) / rows;
    g.ranges = std::max(1, sm_count() / g.row_blocks);
    return g;
}

struct DecodeParams {
    LatentDecodeArgs a;
    int row_blocks, ranges;
    void *parts;  // Part [range][row block][2]: begun before the range / begun in it
    Stat *stats;  // [row][2][range]: what a joining warp reads lies together
    Join *joins;  // [ranges]
};

template <int kRows>
__global__ void __launch_bounds__(kThreads, 1)
    latent_decode_kernel(const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_c, const DecodeParams p) {
    using C = Cfg<kRows>;
    constexpr int kSlots = C::kSlots, kCopies = C::kCopies, kTile = C::kTile;
    constexpr int kCols = kRows / 4;  // score columns of a softmax thread
    constexpr uint32_t kSmTile = 0, kSmQ = C::kSmQ, kSmP = C::kSmP, kTmemX = C::kTmemX, kTileBytes = C::kTileBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    __shared__ uint64_t full[kSlots], empty[kSlots][kCopies], full_q, empty_q, x_full[2], p_full[2], pv_done[2], o_empty;
    __shared__ uint32_t tmem_base;
    __shared__ int piece[kThreads / 32], start_n, start_off, start_len;
    __shared__ float sh_col[4][kRows], sh_row[kRows];
    __shared__ __align__(16) float sh_inv[kRows];
    __shared__ volatile int dead, lost, odd;

    const LatentDecodeArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int rb = blockIdx.x % p.row_blocks, range = blockIdx.x / p.row_blocks;

    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&full[i], 1);
            for (int j = 0; j < kCopies; ++j) mbar_init(&empty[i][j], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&x_full[i], 1), mbar_init(&p_full[i], 128), mbar_init(&pv_done[i], 1);
        }
        mbar_init(&full_q, 1), mbar_init(&empty_q, 1), mbar_init(&o_empty, 128);
        fence_mbar_init();
        dead = lost = odd = 0;
    }
    if (wid == 1) tmem_alloc(&tmem_base, C::kTmemCols);
    // (the join is not let in early: its CTAs would settle on the SMs that finish
    // first and run there one after the other)
    griddep_wait();

    // this range's first request: sums over contiguous pieces of the requests,
    // then a walk inside the piece where the range begins
    const int per = (a.n_seqs + kThreads - 1) / kThreads;
    const int n0 = min(tid * per, a.n_seqs), n1 = min(n0 + per, a.n_seqs);
    int mine = 0, last_len = 0;
    for (int n = n0; n < n1; ++n) {
        last_len = a.seq_lens[n];
        mine += tiles_of<kTile>(a, last_len);
    }
    int before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
    }
    if (lane == 31) piece[wid] = before;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    before -= mine;
    int total = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i < wid) before += piece[i];
        total += piece[i];
    }
    const int ranges = min(p.ranges, total);  // none is empty
    const Cut cut(total, ranges);
    const int range_begin = cut.begin(min(range, ranges)), range_end = cut.begin(min(range + 1, ranges));
    if (range_begin >= before && range_begin < before + mine) {
        int n = n0, len = last_len;
        for (; n + 1 < n1; ++n) {
            len = a.seq_lens[n];
            const int t = tiles_of<kTile>(a, len);
            if (range_begin < before + t) break;
            before += t;
            len = last_len;
        }
        start_n = n;
        start_len = len;
        start_off = range_begin - before;
    }
    __syncthreads();
    Walk<kTile> walk{a, start_n, start_off, range_end - range_begin, start_len, false};
    // a bounded wait; once one has given up, none waits any more
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!dead && !mbar_wait(bar, parity)) dead = 1;
    };
    const uint32_t tmem = tmem_base;
    Segment s;

    if (wid == 0) {
        // ---- TMA: the queries of a request, then its tiles
        int slot = 0, phase = 0, seg = 0;
        for (; !dead && walk.next(s); ++seg) {
            const int32_t *table = a.block_table + (int64_t)s.n * a.max_pages;
            // lane j's copy of a tile: the cache row it begins at, negative where there is nothing to copy
            auto row_of = [&](int tile) {
                const int64_t pos = (int64_t)tile * kTile + lane * kCopy;
                if (lane >= kCopies || pos >= s.len) return -1;
                const int id = table[pos >> a.page_shift];
                if (id < 0 || id >= a.n_pages) return -1;
                return (id << a.page_shift) + (int)(pos & ((1 << a.page_shift) - 1));
            };
            int next_row = row_of(s.tile0);
            auto queries = [&] {
                // the queries of the request before have been read by its last first product
                wait(&empty_q, (seg & 1) ^ 1);
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full_q, 9 * kRows * 128);
                    tma_load_3d(sm + kSmQ, &map_q, 0, s.n * (a.S * a.H) + rb * kRows, 0, &full_q);
                }
                __syncwarp();
            };
            if (seg == 0) queries();  // while the table entries come
            for (int i = 0; i < s.tiles && !dead; ++i) {
                const int row = next_row;
                if (i + 1 < s.tiles) next_row = row_of(s.tile0 + i + 1);
                const int copies = __popc(__ballot_sync(0xffffffffu, row >= 0));
                for (int j = 0; j < kCopies; ++j) {
                    wait(&empty[slot][j], phase ^ 1);
                    if (j == 0 && lane == 0) mbar_arrive_expect_tx(&full[slot], copies * kCopyBytes);
                    __syncwarp();
                    if (lane == j && row >= 0)
                        tma_load_4d(sm + kSmTile + slot * kTileBytes + j * kCopyBytes, &map_c, 0, 0, 0, row >> 3,
                                    &full[slot]);
                }
                if (i == 0 && seg > 0) queries();
                if (++slot == kSlots) slot = 0, phase ^= 1;
            }
        }
    } else if (wid == 1) {
        // ---- first products, one tile ahead of the softmax (two accumulators)
        if (elect_one()) {
            const uint32_t q0 = smem_u32(sm + kSmQ), tile_0 = smem_u32(sm + kSmTile);
            constexpr uint32_t idesc = idesc_bf16(64, kRows);
            int t = 0, slot = 0, phase = 0;
            for (int seg = 0; !dead && walk.next(s); ++seg) {
                wait(&full_q, seg & 1);
                for (int i = 0; i < s.tiles && !dead; ++i, ++t) {
                    wait(&full[slot], phase);
                    // its accumulator was read by the softmax of two tiles ago
                    if (t >= 2) wait(&p_full[t & 1], ((t >> 1) & 1) ^ 1);
                    tc_fence_after();
                    const uint32_t d = tmem + kTmemX + (t & 1) * kRows, tile = tile_0 + slot * kTileBytes;
#pragma unroll
                    for (int b = 0; b < 9; ++b)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16(d, tile_desc_k(tile, b, k),
                                     ((uint64_t)kDescHi << 32) | operand_lo<false, kRows>(q0 + b * kRows * 128, k),
                                     idesc, b + k > 0);
                    mma_commit(&x_full[t & 1]);
                    if (++slot == kSlots) slot = 0, phase ^= 1;
                }
                mma_commit(&empty_q);
            }
        }
        __syncwarp();
    } else if (wid == 2) {
        // ---- second products
        if (elect_one()) {
            const uint32_t tile_0 = smem_u32(sm + kSmTile), p0 = smem_u32(sm + kSmP);
            constexpr uint32_t idesc = idesc_bf16(128, kRows) | (1u << 15) | (1u << 16);
            int t = 0, slot = 0;
            for (int seg = 0; !dead && walk.next(s); ++seg) {
                for (int i = 0; i < s.tiles && !dead; ++i, ++t) {
                    wait(&p_full[t & 1], (t >> 1) & 1);
                    if (i == 0 && seg > 0) wait(&o_empty, (seg - 1) & 1);
                    tc_fence_after();
                    const uint32_t tile = tile_0 + slot * kTileBytes, pt = p0 + (t & 1) * C::kPBytes;
#pragma unroll
                    for (int k = 0; k < kCopies; ++k) {
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            mma_bf16(tmem + b * kRows, tile_desc_mn(tile, b, k),
                                     C::kOwnP ? own_p_desc(pt, k) : tile_p_desc(tile, k), idesc,
                                     i > 0 || k > 0);
                        mma_commit(&empty[slot][k]);
                    }
                    mma_commit(&pv_done[t & 1]);
                    if (++slot == kSlots) slot = 0;
                }
            }
        }
        __syncwarp();
    } else if (wid == 3) {
        // ---- the join's records, by the CTA that answers for the range.  They follow from the lengths alone: where
        // a wait gives up, the parts' NaN reach the joined rows, and other rows' parts are joined as ever.
        if (rb == 0 && lane == 0) write_joins(walk, cut, range_begin, range, a.n_seqs <= p.ranges, p.joins);
        __syncwarp();
    } else if (wid >= 4) {
        const int tid = threadIdx.x - 128, wid = tid >> 5;  // of the four softmax warps
        // ---- softmax: a thread holds scores of tokens 16 w + lane / 4 (+ 8) of the tile by
        // rows 8 j + 2 (lane % 4) + {0, 1}; warp 3 has no tokens (its scores are hidden)
        const Walk<kTile> again = walk;
        const uint32_t lanes = (uint32_t)(wid * 32) << 16;
        const float scale2 = a.scale * kLog2e;
        const int rows = min(kRows, a.S * a.H - rb * kRows);
        const int tok = 16 * wid + (lane >> 2), col = 2 * (lane & 3);
        // of the thread's rows: new token r / H sees positions below len - S + 1 + r / H; rows past the request's
        // (the next request's queries, whose scores nobody reads) see none of the last tiles
        int limit[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
            const int r = 8 * (c >> 1) + col + (c & 1);
            limit[c] = r < rows ? (rb * kRows + r) / a.H - a.S + 1 : INT32_MIN / 2;
        }
        int slot = 0, t = 0;
        bool gave_up = false;  // the same in all four warps: decided by their votes
        while (!gave_up && walk.next(s)) {
            float m[kCols], l[kCols];
#pragma unroll
            for (int c = 0; c < kCols; ++c) m[c] = -INFINITY, l[c] = 0.0f;
            bool bad = !s.ok;
            for (int i = 0; i < s.tiles; ++i, ++t) {
                const int64_t pos0 = (int64_t)(s.tile0 + i) * kTile;
                if (tid >= 96 && tid < 96 + kCopies && pos0 + (tid - 96) * kCopy < s.len) {
                    const int64_t page = (pos0 + (tid - 96) * kCopy) >> a.page_shift;
                    const int id = a.block_table[(int64_t)s.n * a.max_pages + page];
                    bad |= id < 0 || id >= a.n_pages;
                }
                wait(&x_full[t & 1], (t >> 1) & 1);
                tc_fence_after();
                float x[2 * kCols];
#pragma unroll
                for (int k = 0; k < kRows / 32; ++k)
                    tmem_ld_16x32(tmem + kTmemX + (t & 1) * kRows + 32 * k + lanes,
                                  *reinterpret_cast<float(*)[16]>(x + 16 * k));
#pragma unroll
                for (int k = 0; k < kRows / 32; ++k) tmem_ld_wait_for(*reinterpret_cast<float(*)[16]>(x + 16 * k));
#pragma unroll
                for (int j = 0; j < 2 * kCols; ++j) x[j] *= scale2;
                if (pos0 + kTile > s.len - a.S + 1 || wid >= kCopies) {
                    // the last tiles: what a row does not see, and rows of the tile that hold no token
#pragma unroll
                    for (int j = 0; j < 2 * kCols; ++j) {
                        const int64_t pos = pos0 + tok + ((j >> 1) & 1) * 8;
                        if (wid >= kCopies || pos >= (int64_t)s.len + limit[(j >> 2) * 2 + (j & 1)]) x[j] = -INFINITY;
                    }
                    if (tid < 2 * kTile && pos0 + (tid >> 1) >= s.len - a.S + 1) {
                        // A place that some row does not see gets p = 0 there, and 0 times its values has to be 0:
                        // rows without a token (shared memory may hold anything) become 0, and so do values of
                        // a new token that are not finite (given back in the end to the rows that see it).
                        const bool none = pos0 + (tid >> 1) >= s.len;
                        uint4 *r = (uint4 *)(sm + kSmTile + slot * kTileBytes + (tid >> 4) * kGroup +
                                             ((tid >> 1) & 7) * 128 + (tid & 1) * 4096);
                        // Each row goes through its places from another one on, so that eight rows are in different
                        // banks (1024 requests of 60 tokens: 50 instead of 55 us).
                        int turn = (tid >> 1) & 7;
                        asm volatile("" : "+r"(turn));  // its addresses are not kept in registers across the tiles
                        for (int b = 0; b < 4; ++b, r += 64) {
                            if (none) {
#pragma unroll
                                for (int j = 0; j < 8; ++j) r[j ^ turn] = make_uint4(0, 0, 0, 0);
                            } else {
                                uint32_t ones = 0;
#pragma unroll
                                for (int j = 0; j < 8; ++j) ones |= exponent_of_ones(r[j ^ turn]);
                                if (ones) odd = 1;
                                for (int j = 0; ones && j < 8; ++j) r[j] = finite_or_zero(r[j]);
                            }
                        }
                    }
                }
                uint8_t *const held = sm + kSmTile + slot * kTileBytes;
                if (++slot == kSlots) slot = 0;
                float over = -INFINITY;  // fmaxf skips the NaN of -inf - -inf
#pragma unroll
                for (int j = 0; j < 2 * kCols; ++j) over = fmaxf(over, x[j] - m[(j >> 2) * 2 + (j & 1)]);
                const bool given = dead;
                if (given) lost = 1;
                if (!named_bar_and(1, 128, !(over > kRaise) && !given)) {
                    if (lost) {  // written before the vote only
                        gave_up = true;
                        break;
                    }
                    // The rows that passed their reference take their maximum so far.  The others keep theirs, so that
                    // a row's rounding follows from its own scores, whatever the rows beside it hold.
#pragma unroll
                    for (int c = 0; c < kCols; ++c) {
                        const int j = (c >> 1) * 4 + (c & 1);
                        float top = fmaxf(x[j], x[j + 2]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        if (lane < 4) sh_col[wid][8 * (c >> 1) + col + (c & 1)] = top;
                    }
                    named_bar_sync(1, 128);
#pragma unroll
                    for (int c = 0; c < kCols; ++c) {
                        const int r = 8 * (c >> 1) + col + (c & 1);
                        const float top = fmaxf(fmaxf(fmaxf(sh_col[0][r], sh_col[1][r]), fmaxf(sh_col[2][r], sh_col[3][r])), m[c]);
                        const bool up = top - m[c] > kRaise;  // (not where both are -inf)
                        const float f = up ? exp2_sfu(m[c] - top) : 1.0f;
                        if (up) m[c] = top;
                        l[c] *= f;
                        if (wid == 0 && lane < 4) sh_row[r] = f;
                    }
                    if (i > 0) {
                        wait(&pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1);
                        tc_fence_after();
                        named_bar_sync(1, 128);
                        for (int k = 0; k < 4 * kRows / 32; ++k) {
                            float o[32];
                            tmem_ld32(tmem + k * 32 + lanes, o);
                            tmem_ld_wait_for(o);
                            uint32_t u[32];
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                u[c] = __float_as_uint(o[c] * sh_row[(32 * k) % kRows + c]);
                            tmem_st32(tmem + k * 32 + lanes, u);
                        }
                        tmem_st_wait();
                    }
                    named_bar_sync(1, 128);  // sh_col and sh_row are read before they are written again
                }
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    const int j = (c >> 1) * 4 + (c & 1);
                    const float ref = m[c] == -INFINITY ? 0.0f : m[c];
                    x[j] = exp2_sfu(x[j] - ref);
                    x[j + 2] = exp2_sfu(x[j + 2] - ref);
                    l[c] += x[j] + x[j + 2];
                }
                auto put = [&](int token, int row, uint32_t two) {
                    uint8_t *at = C::kOwnP ? sm + kSmP + (t & 1) * C::kPBytes + sw64_off(token, row) : held + tile_p_off(token, row);
                    *(uint32_t *)at = two;
                };
                // an own buffer's p was read by the second product of two tiles ago (a tile's positional
                // block by its first product)
                if (C::kOwnP && t >= 2) wait(&pv_done[t & 1], ((t >> 1) & 1) ^ 1);
#pragma unroll
                for (int j = 0; j < kRows / 8; ++j) {
                    put(tok, 8 * j + col, pack2(x[4 * j], x[4 * j + 1]));
                    put(tok + 8, 8 * j + col, pack2(x[4 * j + 2], x[4 * j + 3]));
                }
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(&p_full[t & 1]);
            }
            if (gave_up) break;
            // ---- the request's part of this range is done
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], o);
                if (lane < 4) {
                    const int r = 8 * (c >> 1) + col + (c & 1);
                    sh_col[wid][r] = l[c];
                    if (wid == 0) sh_row[r] = m[c];
                }
            }
            // (what follows the vote is done while the last second product runs)
            const bool fine = named_bar_and(1, 128, !bad);
            const int64_t row0 = (int64_t)s.n * a.S * a.H + rb * kRows;
            if (tid < rows) {
                float lt = (sh_col[0][tid] + sh_col[1][tid]) + (sh_col[2][tid] + sh_col[3][tid]);
                if (!fine) lt = NAN;
                const float mt = sh_row[tid];
                // what the row's sums are divided by; a row that saw nothing has zeros
                sh_inv[tid] = lt == 0.0f ? 1.0f : 1.0f / lt;
                if (!s.whole()) p.stats[(2 * (rb * kRows + tid) + (s.tile0 == 0 ? 1 : 0)) * p.ranges + range] = {mt, lt};
                else if (a.lse) a.lse[row0 + tid] = lt == 0.0f ? -INFINITY : (mt + log2_sfu(lt)) * kLn2;
            }
            Part<kRows> *part = (Part<kRows> *)p.parts + ((int64_t)range * p.row_blocks + rb) * 2 + (s.tile0 == 0 ? 1 : 0);
            wait(&pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1);
            tc_fence_after();
            named_bar_sync(1, 128);
            // O^T's columns are query rows, eight at a time: few instructions where rows are few (1024 requests of
            // 60 tokens, 8 rows: 38 us, 43 by sixteen and 48 by 32)
            for (int c0 = 0; c0 < rows; c0 += 8) {
                float o[4][8];
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld8(tmem + k * kRows + c0 + lanes, o[k]);
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld_wait_for(o[k]);
                if (s.whole()) {
                    __nv_bfloat16 *dst = a.o + (row0 + c0) * kLatent + tid;
                    float inv[8];
#pragma unroll
                    for (int c = 0; c < 8; c += 4) *(float4 *)(inv + c) = *(const float4 *)(sh_inv + c0 + c);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            if (c0 + c < rows) dst[c * kLatent + k * 128] = __float2bfloat16_rn(o[k][c] * inv[c]);
                } else {
                    float *dst = &part->o[c0][tid];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            if (c0 + c < rows) dst[c * kLatent + k * 128] = o[k][c];
                }
            }
            tc_fence_before();
            mbar_arrive(&o_empty);
            named_bar_sync(1, 128);  // sh_col and sh_row are read before the next request writes them
        }
        const bool alive = named_bar_and(1, 128, !dead);
        if (alive && odd) {
            // A value that is not finite is NaN in its channel for every row that sees its token: by that row's
            // scores where one is NaN or +inf, and by 0 times the value where it is -inf.  (The tiles have lost
            // it; a thread writes the channels that it wrote above.)
            Walk<kTile> w = again;
#pragma unroll 1
            while (w.next(s)) {
                const int64_t row0 = (int64_t)s.n * a.S * a.H + rb * kRows;
                Part<kRows> *part = (Part<kRows> *)p.parts + ((int64_t)range * p.row_blocks + rb) * 2 + (s.tile0 == 0 ? 1 : 0);
                const int64_t begin = max((int64_t)s.tile0 * kTile, (int64_t)s.len - a.S + 1);
                const int64_t end = min((int64_t)(s.tile0 + s.tiles) * kTile, (int64_t)s.len);
                for (int64_t pos = begin; pos < end; ++pos) {
                    const int id = a.block_table[(int64_t)s.n * a.max_pages + (pos >> a.page_shift)];
                    if (id < 0 || id >= a.n_pages) continue;  // (the whole request is NaN)
                    const __nv_bfloat16 *token =
                        a.cache + (((int64_t)id << a.page_shift) + (pos & ((1 << a.page_shift) - 1))) * kLatentRow;
                    const int first = max((int)(pos - s.len + a.S) * a.H - rb * kRows, 0);  // row that sees it
                    for (int d = tid; d < kLatent; d += 128) {
                        if (fabsf(__bfloat162float(token[d])) < INFINITY) continue;
                        for (int r = first; r < rows; ++r) {
                            if (s.whole()) a.o[(row0 + r) * kLatent + d] = __float2bfloat16_rn(NAN);
                            else part->o[r][d] = NAN;
                        }
                    }
                }
            }
        }
        if (!alive) {
            // a wait gave up: the range's outputs are NaN, and so are its parts
            Walk<kTile> w = again;
            while (w.next(s)) {
                const int64_t row0 = (int64_t)s.n * a.S * a.H + rb * kRows;
                for (int c = 0; c < rows; ++c) {
                    for (int d = tid; d < kLatent; d += 128) a.o[(row0 + c) * kLatent + d] = __float2bfloat16_rn(NAN);
                    if (a.lse && tid == 0) a.lse[row0 + c] = NAN;
                }
                if (!s.whole() && tid < rows)
                    p.stats[(2 * (rb * kRows + tid) + (s.tile0 == 0 ? 1 : 0)) * p.ranges + range] = {NAN, NAN};
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (dead) {  // let copies still in flight land before the CTA's memory is given up
        const long long t0 = clock64();
        while (clock64() - t0 < 100000000LL) __nanosleep(1000);
    }
    if (wid == 1) tmem_dealloc(tmem, C::kTmemCols);
}

// Joins the parts of a request that crosses ranges.  With many rows a warp takes
// a query row.  With few (MANY parts each, as a single long request leaves) a
// CTA takes a quarter of a row's 512 values, each of its eight warps every
// eighth part, and their sums are added in order.
constexpr int kJoinThreads = 256;
template <int kRows, bool MANY>
__global__ void __launch_bounds__(kJoinThreads) latent_decode_join_kernel(const DecodeParams p) {
    extern __shared__ float weights[];  // [8 warps][ranges]
    constexpr int kVec = MANY ? 1 : 4, kStep = MANY ? 8 : 1, kBatch = MANY ? 10 : 4;
    __shared__ float4 sums[kStep][32];
    griddep_wait();
    griddep_launch_dependents();
    const LatentDecodeArgs &a = p.a;
    const Join j = p.joins[blockIdx.x];
    if (j.n < 0) return;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int row = MANY ? blockIdx.y : blockIdx.y * 8 + wid, sub = MANY ? wid : 0;
    if (row >= a.S * a.H) return;
    const int d0 = (MANY ? blockIdx.z * 128 : 0) + 4 * lane;
    const int rb = row / kRows, c = row % kRows, parts = j.last - j.first + 1;
    auto part = [&](int i) {  // the first range began the request
        return (const Part<kRows> *)p.parts + ((int64_t)(j.first + i) * p.row_blocks + rb) * 2 + (i == 0 ? 1 : 0);
    };
    // values are requested in batches, the first one before the weights that it waits for
    float4 v[kBatch][kVec];
    auto request = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int k = 0; k < kVec; ++k)
                v[i][k] = i0 + i * kStep < parts ? *(const float4 *)&part(i0 + i * kStep)->o[c][128 * k + d0]
                                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    };
    request(sub);
    // the largest reference (fmaxf skips NaN, whose weight is NaN below); a part that saw nothing
    // has no reference, and its sum is 0, or NaN where the request cannot be read
    float top = -INFINITY, l = 0.0f;
    const Stat *stat = p.stats + (int64_t)2 * row * p.ranges + j.first;
    auto stat_of = [&](int i) { return stat[i == 0 ? p.ranges : i]; };
    float *weight = weights + wid * p.ranges;
    constexpr int kEach = 5;  // parts a lane keeps; beyond them (no GPU of 160 SMs) they are read again
    Stat mine[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        mine[i] = lane + 32 * i < parts ? stat_of(lane + 32 * i) : Stat{-INFINITY, 0.0f};
        top = fmaxf(top, mine[i].m);
    }
    for (int i = lane + 32 * kEach; i < parts; i += 32) top = fmaxf(top, stat_of(i).m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    auto weigh = [&](int i, const Stat &s) {
        const float w = s.m == -INFINITY ? 0.0f : exp2_sfu(s.m - top);
        weight[i] = w;
        l += w * s.l;
    };
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (lane + 32 * i < parts) weigh(lane + 32 * i, mine[i]);
    for (int i = lane + 32 * kEach; i < parts; i += 32) weigh(i, stat_of(i));
    l = warp_sum(l);
    __syncwarp();
    float4 o[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = sub; i0 < parts; i0 += kBatch * kStep) {
        if (i0 > sub) request(i0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const float w = weight[min(i0 + i * kStep, parts - 1)];
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                const float4 &u = v[i][k];
                if (i0 + i * kStep < parts) o[k].x += w * u.x, o[k].y += w * u.y, o[k].z += w * u.z, o[k].w += w * u.w;
            }
        }
    }
    if (MANY) {
        sums[sub][lane] = o[0];
        __syncthreads();
        if (wid) return;
#pragma unroll
        for (int i = 1; i < kStep; ++i) {
            const float4 u = sums[i][lane];
            o[0].x += u.x, o[0].y += u.y, o[0].z += u.z, o[0].w += u.w;
        }
    }
    const float inv = l == 0.0f ? 1.0f : 1.0f / l;
    const int64_t out = (int64_t)j.n * a.S * a.H + row;
#pragma unroll
    for (int k = 0; k < kVec; ++k)
        *(uint2 *)(a.o + out * kLatent + 128 * k + d0) =
            make_uint2(pack2(o[k].x * inv, o[k].y * inv), pack2(o[k].z * inv, o[k].w * inv));
    if (a.lse && lane == 0 && d0 == 0) a.lse[out] = l == 0.0f ? -INFINITY : (top + log2_sfu(l)) * kLn2;
}

// Rows of 576 as {64 columns, rows, 9 blocks}: a box is the K-major operand of `box_rows` rows.
inline bool encode_blocks(CUtensorMap *m, const void *base, int64_t rows, int box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {64, (cuuint64_t)rows, 9};
    const cuuint64_t strides[2] = {kLatentRow * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 9};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The cache as {64 columns, 8 rows, 9 blocks, groups of 8 rows}, a copy being two groups.
inline bool encode_cache(CUtensorMap *m, const void *base, int64_t rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {64, 8, 9, (cuuint64_t)rows / 8};
    const cuuint64_t strides[3] = {kLatentRow * 2, 128, 8 * kLatentRow * 2};
    const cuuint32_t box[4] = {64, 8, 9, 2};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline size_t joins_bytes(const Grid &g) { return align_up((size_t)g.ranges * sizeof(Join), 256); }
template <int ROWS>
size_t stats_bytes(const Grid &g) {
    return align_up((size_t)g.ranges * g.row_blocks * ROWS * 2 * sizeof(Stat), 256);
}
template <int ROWS>
size_t workspace_bytes(int S, int H) {
    const Grid g = decode_grid(S, H, ROWS);
    return joins_bytes(g) + stats_bytes<ROWS>(g) + (size_t)g.ranges * g.row_blocks * 2 * sizeof(Part<ROWS>);
}

template <int ROWS>
cudaError_t launch(const LatentDecodeArgs &a, cudaStream_t stream) {
    const Grid g = decode_grid(a.S, a.H, ROWS);
    DecodeParams p{a, g.row_blocks, g.ranges};
    uint8_t *ws = (uint8_t *)a.workspace;
    p.joins = (Join *)ws;
    p.stats = (Stat *)(ws + joins_bytes(g));
    p.parts = ws + joins_bytes(g) + stats_bytes<ROWS>(g);
    CUtensorMap map_q, map_c;
    if (!encode_blocks(&map_q, a.q, (int64_t)a.n_seqs * a.S * a.H, ROWS) ||
        !encode_cache(&map_c, a.cache, a.n_pages << a.page_shift))
        return cudaErrorUnknown;
    cudaError_t e = cudaFuncSetAttribute(latent_decode_kernel<ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Cfg<ROWS>::kSmemBytes);
    if (e != cudaSuccess) return e;
    e = launch_dependent(latent_decode_kernel<ROWS>, dim3(g.ranges * g.row_blocks), dim3(kThreads),
                         Cfg<ROWS>::kSmemBytes, stream, map_q, map_c, p);
    if (e != cudaSuccess) return e;
    const size_t weights = (size_t)8 * g.ranges * sizeof(float);
    const int joins = std::min(a.n_seqs, g.ranges), rows = a.S * a.H;
    if (joins * rows <= 128)
        e = launch_dependent(latent_decode_join_kernel<ROWS, true>, dim3(joins, rows, 4), dim3(kJoinThreads), weights,
                             stream, p);
    else
        e = launch_dependent(latent_decode_join_kernel<ROWS, false>, dim3(joins, (rows + 7) / 8), dim3(kJoinThreads),
                             weights, stream, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t latent_decode_workspace_bytes(int n_seqs, int S, int H) {
    return std::max(workspace_bytes<32>(S, H), workspace_bytes<64>(S, H));
}

cudaError_t launch_latent_decode(const LatentDecodeArgs &a, cudaStream_t stream) {
    // 64 query rows a CTA read the cache half as often, but take 3 us longer over a first tile, and their
    // ring holds 128 tokens against 144.  What counts is how often 32 rows a CTA would read the tokens that
    // the block table can hold: 128k tokens (4 requests, 128 rows each) 29.1 us with 32 rows and 30.2 us with
    // 64, 180k (7 requests, 64 rows) 34.8 and 37.3, 187k (183 requests, 128 rows) 47.6 and 46.2, 256k
    // (16 requests, 48 rows) 44.6 and 40.0, 640k (4 requests, 128 rows) 85.6 and 68.9.
    const int64_t read = (((int64_t)a.n_seqs * a.max_pages) << a.page_shift) * ((a.S * a.H + 31) / 32);
    return a.S * a.H > 32 && read > 184320 ? launch<64>(a, stream) : launch<32>(a, stream);
}

}  // namespace kda
