// Sequences of a chunked linear-attention forward cut into segments, so that long sequences of few
// heads fill the GPU: a kernel takes every segment's own state from zero (all but each sequence's last),
// the join turns them into the states in front of the segments, and a kernel computes the outputs from those.
#pragma once

#include "kda_linear.cuh"

namespace kda {

constexpr int kState = kHeadDim * kHeadDim;

// A segment to work on, in four registers: what warps look at in every chunk must not be in local memory,
// for which the L1 cache has no room beside this shared memory.
enum : int { kBegins = 1 << 16, kEnds = 1 << 17, kCut = 1 << 18, kNoSlot = 1 << 19 };
constexpr int kEntry = 20;
// first token, tokens, slot of the states, flags: in the low 16 bits, once it is picked, the head, in the upper 12 its entry (some hundreds at most)
typedef int4 Item;
__device__ __forceinline__ int head_of(const Item &s) { return s.w & 0xffff; }

struct ChunkParams {
    LinearChunkArgs a;
    int segment;    // tokens; several sequences may be left uncut
    int entries;    // segments whose state the workspace holds, at most
    int parallel;   // segments and heads that are worked on at the same time
    int fixed;      // tokens of one that cost as much as the two launches of a cut
    bool listed;    // there are lists
    bool joined;    // the kernel follows the others: its inputs are there before it begins
    int *counts;    // length of each list
    Item *outputs;  // all segments, the longest first
    Item *inner;    // [entries]: those that others follow in their sequence
    Item *cuts;     // [entries]: the sequences that are cut: first entry, such segments, slot
    float *states;  // [entries][H][V][K]
    float *first;   // [entries][H][V][K]: copies of initial states (those that a later CTA may overwrite)
    float2 *decay;  // [entries][H], each the sum of two floats
};

// Whether a cut pays, by the time (in tokens of one segment and head) of the longest part, or of all (and a quarter of the longest for
// the uneven end) where that is more.  A segment's own state takes half the time of its outputs.  each: H / parallel; followed:
// segments with a successor.
__host__ __device__ inline bool cut_pays(int64_t longest, int64_t sum, int64_t followed, int64_t segment, float each, int fixed) {
    const float most = (float)longest, whole = (float)sum * each, part = (float)segment;
    const float uncut = fmaxf(most, whole + 0.25f * most);
    const float cut = fmaxf(part, whole + 0.25f * part) + fixed + 0.5f * fmaxf(part, (float)followed * part * each);
    return followed > 0 && cut < uncut;
}

// Where the segments are found: in the lists; a single sequence needs none, nor do sequences that cannot be cut (no
// entries), if they are few or short or of one length (5 of 17 to 200 tokens, 8 heads, take 12.2 us of the
// device, 15.7 with lists).  Others are listed for their order though there is nothing to cut: eight of 333 to
// 4001 tokens, 96 heads: 352 us; 414 in the order given, a rising one.  A kernel for each: with
// a choice in every warp's loop, 131072 tokens of 8 heads take 335 instead of 316 us.
enum Source { kListed, kOne, kWhole };
inline Source source_of(const ChunkParams &p) { return p.listed ? kListed : p.entries > 0 ? kOne : kWhole; }

// f(segment and head) for each of the `cta`-th of `ctas`, of all segments (OUTPUT) or of those that have a successor:
// back and forth over the list, so that who had one of the longest gets one of the shortest next.
template <bool OUTPUT, Source SOURCE, typename F>
__device__ __forceinline__ void for_segments(const ChunkParams &p, uint32_t cta, uint32_t ctas, F f) {
    const LinearChunkArgs &a = p.a;
    const Span only = SOURCE == kOne ? span_of(a, 0) : Span{0, -1};
    const int slot = SOURCE == kOne ? (int)slot_of(a, 0) : 0, full = only.len > 0 ? (uint32_t)(only.len - 1) / p.segment : 0;
    const int count = SOURCE == kWhole ? a.n_seqs : SOURCE == kListed ? p.counts[OUTPUT ? 0 : 1] : only.len < 0 ? 0 : OUTPUT ? full + 1 : slot < 0 ? 0 : full;
    const uint32_t items = (uint32_t)count * a.H;
    for (uint32_t k = 0;; ++k) {
        const uint32_t i = k * ctas + (k & 1 ? ctas - 1 - cta : cta);
        if (i >= items) break;
        const uint32_t n = i / (uint32_t)a.H;
        Item s;
        if constexpr (SOURCE == kListed) {
            s = (OUTPUT ? p.outputs : p.inner)[n];
        } else if constexpr (SOURCE == kOne) {
            s = make_int4(only.first + n * p.segment, min(p.segment, only.len - (int)n * p.segment), slot,
                          (n == 0 ? kBegins : 0) | (n == full ? kEnds : 0) | (full > 0 ? kCut : 0) | (slot < 0 ? kNoSlot : 0) | (n << kEntry));
        } else {
            const Span span = span_of(a, n);
            const int own = (int)slot_of(a, n);
            if (span.len < 0) continue;
            s = make_int4(span.first, span.len, own, kBegins | kEnds | (own < 0 ? kNoSlot : 0));
        }
        s.w |= i - n * a.H;
        f(s);
    }
}
// A segment's (and head's) place in states, first and decay.
__device__ __forceinline__ int64_t entry_of(const ChunkParams &p, const Item &s) {
    return (int64_t)((uint32_t)s.w >> kEntry) * p.a.H + head_of(s);
}
// The state in front of a segment: nullptr for zeros.
__device__ __forceinline__ const float *state_before(const ChunkParams &p, const Item &s) {
    const LinearChunkArgs &a = p.a;
    const int64_t at = entry_of(p, s);
    if (!(s.w & kBegins)) return p.states + (at - a.H) * kState;
    if (!a.initial_state) return nullptr;
    return s.w & kCut ? p.first + at * kState : a.initial_state + ((int64_t)s.z * a.H + head_of(s)) * kState;
}
// Where the state behind a segment goes: nullptr if nowhere.
__device__ __forceinline__ float *state_after(const ChunkParams &p, const Item &s) {
    const LinearChunkArgs &a = p.a;
    return (s.w & kEnds) && a.final_state ? a.final_state + ((int64_t)s.z * a.H + head_of(s)) * kState : nullptr;
}

// How a call's sequences are cut: tokens of a segment, and the terms of what a cut costs (ChunkParams).
struct Cut {
    int64_t segment;
    int parallel, fixed;
};
size_t segments_workspace_bytes(int64_t total_tokens, int n_seqs, int H, const Cut &cut);
ChunkParams plan_segments(const LinearChunkArgs &a, const Cut &cut);
cudaError_t launch_segment_lists(const ChunkParams &p, cudaStream_t stream);
cudaError_t launch_segment_join(const ChunkParams &p, cudaStream_t stream);

}  // namespace kda
