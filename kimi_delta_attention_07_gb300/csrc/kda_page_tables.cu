// Block tables and slot maps of one step, from request lengths on the device.
//
// With P = page_size, request n needs
//   need_n = ceil((ctx_n + new_n) / P) - ceil(ctx_n / P)
// pages, which are free_pages[e_n - need_n .. e_n), e the inclusive prefix sum
// of need; packed token t of request r (cu_r <= t < cu_{r+1}) has position
// p = ctx_r + t - cu_r and row table[r][p / P] * P + p % P.
//
// One launch: the prefix sums over N requests are a few KB, so every CTA takes
// them itself (in shared memory, one block scan over contiguous pieces) and
// no CTA waits for another.  A CTA then fills its share of the rows' new table
// entries (a warp per request) and of the tokens; the page of a token is read
// from the free list where it is new, so that no CTA reads what another one
// writes.  Bound by launch and scan latency: the slots and positions of 256
// requests with 1.1M new tokens (9 MB) take 8.5 us, those of 8 requests with one
// token each 3.4 us.
#include <algorithm>

#include "kda_hybrid.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kTokensPerThread = 4;

__device__ __forceinline__ int64_t warp_inclusive_scan(int64_t x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

struct Need {
    int64_t held, total;  // pages before and after this step
    int64_t added;        // packed tokens (new_lens, 0 if negative)
    bool fits;            // lengths and table row admit the request
};

__device__ __forceinline__ Need request_need(const PageTablesArgs &a, int64_t ctx, int64_t add) {
    const int64_t r = ((int64_t)1 << a.page_shift) - 1;
    Need d;
    d.added = add > 0 ? add : 0;
    d.held = (ctx + r) >> a.page_shift;
    d.total = (ctx + add + r) >> a.page_shift;
    d.fits = ctx >= 0 && add >= 0 && ctx + add <= INT32_MAX && d.total <= a.max_pages;
    return d;
}

__device__ __forceinline__ int32_t clamp32(int64_t x) {
    return (int32_t)(x < INT32_MAX ? x : INT32_MAX);
}

__global__ void __launch_bounds__(kThreads) page_tables_kernel(const PageTablesArgs a) {
    extern __shared__ int32_t sh[];
    int32_t *cu = sh;                  // [N + 1] offsets of the packed new tokens (until then: new_lens)
    int32_t *first = cu + a.n_seqs + 1;  // [N] place of the first new page in free_pages, -1: refused
    int32_t *ctx = first + a.n_seqs;     // [N] ctx_lens
    __shared__ int64_t part[2][kThreads / 32];
    __shared__ int32_t seen[2];  // {largest end of a request that fits, refused}
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;

    griddep_wait();
    griddep_launch_dependents();
    const int64_t begin = a.free_start ? max(a.free_start[0], 0) : 0;
    if (tid < 2) seen[tid] = tid == 0 ? clamp32(begin) : 0;
    // Long pieces come through shared memory, read coalesced; an odd length has no bank conflicts (16384
    // requests of one token: 31 us, 530 when each thread reads its piece from global memory).  Short ones
    // do without the barrier (256 requests, 1.1M tokens: 8.5 and 9.1 us).
    const int pieces = (a.n_seqs + kThreads - 1) / kThreads;
    const bool staged = pieces > 4;
    const int per = staged ? pieces | 1 : pieces;
    if (staged) {
        for (int n = tid; n < a.n_seqs; n += kThreads) ctx[n] = a.ctx_lens[n], cu[n] = a.new_lens[n];
        __syncthreads();
    }
    const int32_t *ctx_of = staged ? ctx : a.ctx_lens, *new_of = staged ? cu : a.new_lens;
    const int n0 = min(tid * per, a.n_seqs), n1 = min(n0 + per, a.n_seqs);
    int64_t pages = 0, tokens = 0;
    for (int n = n0; n < n1; ++n) {
        const Need d = request_need(a, ctx_of[n], new_of[n]);
        pages += d.fits ? d.total - d.held : 0;
        tokens += d.added;
    }
    int64_t ps = warp_inclusive_scan(pages, lane), ts = warp_inclusive_scan(tokens, lane);
    if (lane == 31) part[0][wid] = ps, part[1][wid] = ts;
    __syncthreads();
    for (int w = 0; w < wid; ++w) ps += part[0][w], ts += part[1][w];
    ps += begin - pages;
    ts -= tokens;
    const bool writer = blockIdx.x == 0;
    for (int n = n0; n < n1; ++n) {
        const int32_t held = ctx_of[n], added = new_of[n];
        const Need d = request_need(a, held, added);
        const int64_t need = d.fits ? d.total - d.held : 0;
        const bool fits = d.fits && (need == 0 || ps + need <= a.n_free);
        cu[n] = clamp32(ts);
        first[n] = fits ? clamp32(ps) : -1;
        ctx[n] = held;
        if (writer) {
            a.cu_seqlens[n] = clamp32(ts);
            a.seq_lens[n] = fits ? held + added : max(held, 0);
            if (fits) {
                if (need) atomicMax(&seen[0], (int32_t)(ps + need));
            } else {
                atomicAdd(&seen[1], 1);
            }
        }
        ps += need;
        ts += d.added;
    }
    if (tid == kThreads - 1) cu[a.n_seqs] = clamp32(ts);
    __syncthreads();
    if (writer && tid == 0) {
        a.cu_seqlens[a.n_seqs] = cu[a.n_seqs];
        a.status[0] = seen[0];
        a.status[1] = seen[1];
    }

    // new table entries: a warp per request
    for (int n = blockIdx.x * (kThreads / 32) + wid; n < a.n_seqs; n += gridDim.x * (kThreads / 32)) {
        if (first[n] < 0) continue;
        const Need d = request_need(a, ctx[n], a.new_lens[n]);
        int32_t *row = a.block_table + (int64_t)n * a.max_pages;
        for (int64_t j = d.held + lane; j < d.total; j += 32)
            row[j] = a.free_pages[first[n] + (j - d.held)];
    }

    // slots and positions: four consecutive packed tokens a thread, which mostly share a
    // request and a page, stored as one vector each
    const int32_t packed = cu[a.n_seqs], mask = (1 << a.page_shift) - 1;
    const int64_t step = (int64_t)gridDim.x * kThreads * kTokensPerThread;
    for (int64_t t0 = ((int64_t)blockIdx.x * kThreads + tid) * kTokensPerThread; t0 < a.max_tokens;
         t0 += step) {
        // the last request whose tokens begin at or before t0
        int r = 0, hi = a.n_seqs;
        while (r + 1 < hi) {
            const int mid = (r + hi) >> 1;
            if (cu[mid] <= t0) r = mid; else hi = mid;
        }
        int32_t slot[kTokensPerThread], pos[kTokensPerThread];
        int32_t page = -1, of = -1;  // page id of table entry `of` of request r
#pragma unroll
        for (int i = 0; i < kTokensPerThread; ++i) {
            slot[i] = pos[i] = -1;
            const int64_t t = t0 + i;
            if (t >= packed) continue;
            while (cu[r + 1] <= t) ++r, of = -1;
            if (first[r] < 0) continue;
            const int32_t p = ctx[r] + (int32_t)(t - cu[r]), j = p >> a.page_shift;
            if (j != of) {
                const int32_t held = (int32_t)(((int64_t)ctx[r] + mask) >> a.page_shift);
                page = j < held ? a.block_table[(int64_t)r * a.max_pages + j] : a.free_pages[first[r] + (j - held)];
                of = j;
            }
            if (page >= 0 && page < a.n_pages) slot[i] = (page << a.page_shift) + (p & mask), pos[i] = p;
        }
        if (a.vector_stores && t0 + kTokensPerThread <= a.max_tokens) {
            *reinterpret_cast<int4 *>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int i = 0; i < kTokensPerThread; ++i)
                if (t0 + i < a.max_tokens) a.slots[t0 + i] = slot[i], a.positions[t0 + i] = pos[i];
        }
    }
}

}  // namespace

cudaError_t launch_page_tables(const PageTablesArgs &a, cudaStream_t stream) {
    const size_t smem = (3 * (size_t)a.n_seqs + 1) * sizeof(int32_t);
    if (smem > 40 * 1024) {  // 48 KB, less what the kernel's static arrays take of them
        const cudaError_t e = cudaFuncSetAttribute(
            page_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const int64_t per_cta = kThreads * kTokensPerThread;
    const int64_t want = std::max<int64_t>((a.max_tokens + per_cta - 1) / per_cta,
                                           (a.n_seqs + kThreads / 32 - 1) / (kThreads / 32));
    const int resident = (int)std::min<size_t>(8, (200 * 1024) / std::max<size_t>(smem, 1));  // at least 1
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(want, sm_count() * resident));
    const cudaError_t e = launch_dependent(page_tables_kernel, dim3(grid), dim3(kThreads), smem, stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kda
