// How absorbed attention cuts its work: the tiles of all requests, in order, in
// even ranges, a range's share of each request, and which requests' parts a
// second kernel joins.  It follows from the lengths alone.  Host code too, so
// that it can be checked there.
#pragma once

#include "kda_hybrid.cuh"

namespace kda {

// Tiles [0, total) cut into `ranges` pieces that differ by at most one tile.
struct Cut {
    int base, rem;
    __host__ __device__ __forceinline__ Cut(int total, int ranges) : base(total / ranges), rem(total - base * ranges) {}
    __host__ __device__ __forceinline__ int begin(int range) const { return range * base + (range < rem ? range : rem); }
    __host__ __device__ __forceinline__ int range_of(int tile) const {
        const int longer = rem * (base + 1);
        return tile < longer ? tile / (base + 1) : rem + (tile - longer) / base;
    }
};

template <int TILE>
__host__ __device__ __forceinline__ int tiles_of(const LatentDecodeArgs &a, int len) {
    // an empty request (or one that cannot be read) still has a tile: its outputs are written
    const bool ok = len >= 0 && (int64_t)len <= ((int64_t)a.max_pages << a.page_shift);
    return ok && len > 0 ? (int)(((int64_t)len + TILE - 1) / TILE) : 1;
}

// One request's share of a range.
struct Segment {
    int n, len, tile0, tiles, total;  // tiles [tile0, tile0 + tiles) of the request's `total`
    bool ok;
    __host__ __device__ __forceinline__ bool whole() const { return tiles == total; }
};

// Walks the range's requests; every role keeps its own.
template <int TILE>
struct Walk {
    const LatentDecodeArgs &a;
    int n, off, left;
    int len;  // of request n if it is the first, which the setup has read
    bool begun;
    __host__ __device__ __forceinline__ bool next(Segment &s) {
        if (left <= 0) return false;
        s.n = n;
        s.len = begun ? a.seq_lens[n] : len;
        begun = true;
        s.ok = s.len >= 0 && (int64_t)s.len <= ((int64_t)a.max_pages << a.page_shift);
        s.total = tiles_of<TILE>(a, s.len);
        if (!s.ok) s.len = 0;
        s.tile0 = off;
        s.tiles = s.total - off < left ? s.total - off : left;
        left -= s.tiles;
        ++n;
        off = 0;
        return true;
    }
};

struct Join {  // ranges first..last hold request n's parts; n < 0: nothing to join
    int32_t n, first, last, pad;
};

// The records of the requests that begin in a range (its first tile is `at`): entry n where there are no more
// requests than ranges, else the range's own entry (at most one request leaves a range).
template <int TILE>
__host__ __device__ __forceinline__ void write_joins(Walk<TILE> walk, const Cut &cut, int at, int range, bool by_request,
                                                     Join *joins) {
    Join leaves = {-1, 0, 0, 0};
    Segment s;
    while (walk.next(s)) {
        if (s.tile0 == 0) {
            Join j = {-1, 0, 0, 0};
            if (!s.whole()) j = {s.n, range, cut.range_of(at + s.total - 1), 0};
            if (by_request) joins[s.n] = j;
            leaves = j;
        }
        at += s.tiles;
    }
    if (!by_request) joins[range] = leaves;
}

}  // namespace kda
