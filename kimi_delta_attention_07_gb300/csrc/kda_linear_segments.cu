// Segments of a chunked linear-attention forward: the lists of them, and the join of their states.
#include <algorithm>

#include "kda_linear_segments.cuh"

namespace kda {
namespace {

// The segments: a list of all for the outputs, sorted by length (into kBuckets classes), and one of those that have a
// successor.  Their order in a class is left to chance; what is computed does not depend on it.  (Sequences that
// overlap, as no well-formed offsets do, may be more than the lists hold; what is past their ends is left out.
// 65535 sequences of at most `entries` such segments each, some hundreds, are below 2^31.)
// Lanes whose sequences are of one class share an addition: on their own, 4096 sequences of one length took 283 us.
constexpr int kIndexThreads = 1024, kBuckets = 64;
__global__ void __launch_bounds__(kIndexThreads) segment_lists_kernel(const ChunkParams p) {
    __shared__ int place[kBuckets], inner, cuts;
    const LinearChunkArgs &a = p.a;
    __shared__ int longest, followed;
    __shared__ uint32_t sum;
    const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
    const int most = p.entries + a.n_seqs, most_inner = p.entries;
    for (int i = tid; i < kBuckets; i += threads) place[i] = 0;
    if (tid == 0) inner = cuts = longest = followed = sum = 0;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    // f(first token, tokens (-1: no sequence), slot), by whole warps, offsets and slots of four sequences a thread
    // requested together (once, if there are no more)
    constexpr int kAhead = 4;
    Span span[kAhead];
    int slots[kAhead], held = -1;
    auto for_sequences = [&](auto f) {
#pragma unroll 1
        for (int n0 = tid - lane; n0 < a.n_seqs; n0 += kAhead * threads) {
            if (n0 != held) {
                held = n0;
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int n = n0 + j * threads + lane;
                    span[j] = n < a.n_seqs ? span_of(a, n) : Span{0, -1};
                    slots[j] = n < a.n_seqs ? (int)slot_of(a, n) : 0;
                }
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (n0 + j * threads < a.n_seqs) f(span[j].first, span[j].len, slots[j]);
        }
    };
    // Cut, or not.  (16 sequences of 4000 tokens, 8 heads: 142 us uncut, 200 cut at the time, now 129; one of 60000 and 15 of 300: cut, 185.)
    int my_longest = 0, my_followed = 0;
    uint32_t my_sum = 0;
    for_sequences([&](int, int len, int) {
        if (len <= 0) return;
        my_longest = max(my_longest, len), my_sum += len;
        my_followed += (uint32_t)(len - 1) / (uint32_t)p.segment;
    });
    my_longest = __reduce_max_sync(0xffffffffu, my_longest), my_sum = __reduce_add_sync(0xffffffffu, my_sum);
    my_followed = __reduce_add_sync(0xffffffffu, my_followed);
    if (lane == 0) atomicMax(&longest, my_longest), atomicAdd(&sum, my_sum), atomicAdd(&followed, my_followed);
    __syncthreads();
    const int segment = p.entries > 0 && cut_pays(longest, sum, followed, p.segment, a.H / (float)p.parallel, p.fixed) ? p.segment : max(longest, 1);
    const float scale = (kBuckets - 1) / (float)segment;
    // the segments before a sequence's last one, the tokens of that, and its class
    auto full_of = [&](int len) { return len > 0 ? (int)((uint32_t)(len - 1) / (uint32_t)segment) : 0; };
    auto bucket_of = [&](int len, int rows) { return len < 0 ? -1 : max(0, kBuckets - 1 - (int)(rows * scale)); };
    for_sequences([&](int, int len, int) {
        const int full = full_of(len), bucket = bucket_of(len, len - full * segment);
        const uint32_t same = __match_any_sync(0xffffffffu, bucket);
        if (full > 0) atomicAdd(&place[0], full);
        if (bucket >= 0 && lane == __ffs(same) - 1) atomicAdd(&place[bucket], __popc(same));
    });
    __syncthreads();
    if (tid < 32) {
        const int x = place[2 * tid], own = x + place[2 * tid + 1];
        int upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (tid >= o) upto += y;
        }
        place[2 * tid] = upto - own;
        place[2 * tid + 1] = upto - own + x;
        if (tid == 31) p.counts[0] = min(upto, most);
    }
    __syncthreads();
    for_sequences([&](int first, int len, int at_slot) {
        const int full = full_of(len), rows = len - full * segment, bucket = bucket_of(len, rows), entry = (uint32_t)first / (uint32_t)segment;
        const uint32_t same = __match_any_sync(0xffffffffu, bucket);
        const int slot = at_slot < 0 ? kNoSlot : 0, cut = full > 0 ? kCut : 0;
        if (full > 0) {
            int at = atomicAdd(&place[0], full), in = slot ? most_inner : atomicAdd(&inner, full);
            const int c = slot ? most_inner : atomicAdd(&cuts, 1);
            if (c < most_inner) p.cuts[c] = make_int4(entry, full, at_slot, 0);
#pragma unroll 1
            for (int l = 0; l < full; ++l, ++at, ++in) {
                const Item s = make_int4(first + l * segment, segment, at_slot, (l == 0 ? kBegins : 0) | cut | slot | (entry + l) << kEntry);
                if (at < most) p.outputs[at] = s;
                if (in < most_inner) p.inner[in] = s;
            }
        }
        const int leader = __ffs(same) - 1;
        int at = bucket >= 0 && lane == leader ? atomicAdd(&place[bucket], __popc(same)) : 0;
        at = __shfl_sync(0xffffffffu, at, leader) + __popc(same & ((1u << lane) - 1));
        if (bucket >= 0 && at < most)
            p.outputs[at] = make_int4(first + full * segment, rows, at_slot, (full == 0 ? kBegins : 0) | kEnds | cut | slot | (entry + full) << kEntry);
    });
    __syncthreads();
    if (tid == 0) p.counts[1] = min(inner, most_inner), p.counts[2] = min(cuts, most_inner);
}

// The states in front of the segments of each sequence that is cut, in place of the segments' own: entry l gets
// that in front of segment l + 1.  A sequence's initial state is copied, because its last segment may
// overwrite it while the first one still reads.  A segment's decay is the sum of two floats: one head's 205 segments
// of 2^-20 a token, fp32, were off by 5.9e-6 with one.
// (131072 tokens of 8 heads, 18 segments: 6 us, from L2; eight segments requested ahead.)
constexpr int kJoinThreads = 256, kJoinParts = kState / (4 * kJoinThreads);
__global__ void __launch_bounds__(kJoinThreads) segment_join_kernel(const ChunkParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const LinearChunkArgs &a = p.a;
    const int h = blockIdx.y;
    Item only = make_int4(0, 0, 0, 0);
    if (a.n_seqs == 1) {
        const Span span = span_of(a, 0);
        const int64_t slot = slot_of(a, 0);
        if (span.len <= p.segment || slot < 0) return;
        only = make_int4(0, (span.len - 1) / p.segment, (int)slot, 0);
    }
    const int listed = a.n_seqs == 1 ? 1 : p.counts[2];
    for (int i = blockIdx.x; i < listed; i += gridDim.x) {
        const Item s = a.n_seqs == 1 ? only : p.cuts[i];
        const int count = s.y, entry = s.x;
        const int64_t at = 4 * ((int64_t)blockIdx.z * kJoinThreads + threadIdx.x);
        const int64_t step = (int64_t)a.H * kState, own = ((int64_t)entry * a.H + h) * kState + at;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (a.initial_state) {
            x = *(const float4 *)(a.initial_state + ((int64_t)s.z * a.H + h) * kState + at);
            *(float4 *)(p.first + own) = x;
        }
        float *state = p.states + own;
        const float2 *decay = p.decay + (int64_t)entry * a.H + h;
        constexpr int kAhead = 8;
        for (int l = 0; l < count; l += kAhead) {
            float4 y[kAhead];
            float2 d[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (l + j < count) y[j] = *(const float4 *)(state + (l + j) * step), d[j] = decay[(int64_t)(l + j) * a.H];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (l + j >= count) break;
                x.x = fmaf(d[j].x, x.x, fmaf(d[j].y, x.x, y[j].x)), x.y = fmaf(d[j].x, x.y, fmaf(d[j].y, x.y, y[j].y));
                x.z = fmaf(d[j].x, x.z, fmaf(d[j].y, x.z, y[j].z)), x.w = fmaf(d[j].x, x.w, fmaf(d[j].y, x.w, y[j].w));
                *(float4 *)(state + (l + j) * step) = x;
            }
        }
    }
}

// A segment's entry is floor(sequence's first token / segment) and its place in the sequence: distinct for those that have a
// successor, whatever the lengths.  None where no cut can pay: a single sequence is taken to have all tokens (one of H = 64 and
// 768 tokens 35 us cut, 26 uncut, of 4096 105 and 109; fp32, H = 16, 65 tokens 40 and 16, 256 43 and 55), several to be, at best,
// nearly one, with one segment to add up (7 of 17 to 200 tokens, 8 heads: 12 us, 18 with launches that find nothing to cut).
inline int64_t entries_of(int64_t total_tokens, int n_seqs, int H, const Cut &cut) {
    const int64_t entries = total_tokens > 0 ? (total_tokens - 1) / cut.segment : 0, followed = n_seqs == 1 ? entries : std::min<int64_t>(entries, 1);
    return cut_pays(total_tokens, total_tokens, followed, cut.segment, H / (float)cut.parallel, cut.fixed) ? entries : 0;
}
// Whether sequences that are not cut are listed for their order: more of them and heads than are worked on at the same time,
// and more tokens than a list's launch counts for.
inline bool order_pays(int64_t total_tokens, int n_seqs, int H, const Cut &cut) {
    return total_tokens > 640 && (int64_t)n_seqs * H > cut.parallel;
}

struct Layout {
    size_t outputs, inner, cuts, decay, states, total;
};
inline Layout layout(int64_t total_tokens, int n_seqs, int H, const Cut &cut) {
    const int64_t entries = entries_of(total_tokens, n_seqs, H, cut);
    const bool lists = n_seqs > 1 && (entries > 0 || order_pays(total_tokens, n_seqs, H, cut));
    Layout l;
    l.outputs = lists ? 256 : 0;
    l.inner = l.outputs + (lists ? align_up((size_t)(entries + n_seqs) * sizeof(Item), 256) : 0);
    l.cuts = l.inner + (lists ? align_up((size_t)entries * sizeof(Item), 256) : 0);
    l.decay = l.cuts + (lists ? align_up((size_t)entries * sizeof(Item), 256) : 0);
    l.states = l.decay + align_up((size_t)entries * H * sizeof(float2), 256);
    l.total = l.states + (size_t)entries * H * 2 * kState * sizeof(float);
    return l;
}

}  // namespace

size_t segments_workspace_bytes(int64_t total_tokens, int n_seqs, int H, const Cut &cut) {
    return layout(total_tokens, n_seqs, H, cut).total;
}

ChunkParams plan_segments(const LinearChunkArgs &a, const Cut &cut) {
    const Layout l = layout(a.total_tokens, a.n_seqs, a.H, cut);
    uint8_t *ws = (uint8_t *)a.workspace;
    ChunkParams p{a};
    p.segment = (int)cut.segment;
    p.entries = (int)entries_of(a.total_tokens, a.n_seqs, a.H, cut);
    p.listed = a.n_seqs > 1 && (p.entries > 0 || (a.cu_seqlens && order_pays(a.total_tokens, a.n_seqs, a.H, cut)));
    p.joined = p.entries > 0;
    p.parallel = cut.parallel;
    p.fixed = cut.fixed;
    p.counts = (int *)ws;
    p.outputs = (Item *)(ws + l.outputs);
    p.inner = (Item *)(ws + l.inner);
    p.cuts = (Item *)(ws + l.cuts);
    p.decay = (float2 *)(ws + l.decay);
    p.states = (float *)(ws + l.states);
    p.first = p.states + (int64_t)p.entries * a.H * kState;
    return p;
}

cudaError_t launch_segment_lists(const ChunkParams &p, cudaStream_t stream) {
    if (source_of(p) != kListed) return cudaSuccess;
    return launch_dependent(segment_lists_kernel, dim3(1), dim3(std::min(kIndexThreads, (p.a.n_seqs + 31) / 32 * 32)), 0, stream, p);
}

cudaError_t launch_segment_join(const ChunkParams &p, cudaStream_t stream) {
    // (no more CTAs than two for each place of an SM: most calls of several sequences have nothing to join)
    const int most = std::max(1, 16 * sm_count() / (p.a.H * kJoinParts));
    return launch_dependent(segment_join_kernel, dim3((unsigned)std::min({p.a.n_seqs, p.entries, most}), (unsigned)p.a.H, kJoinParts),
                            dim3(kJoinThreads), 0, stream, p);
}

}  // namespace kda
