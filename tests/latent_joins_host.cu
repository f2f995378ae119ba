// Host check of how absorbed attention cuts its work (kda_latent_split.cuh): the records that the ranges write, for
// random lengths, against the tiles laid out one by one.  Row blocks other than the first write none, whatever happens
// in them.  Prints "ok" and the number of requests that cross a range.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "kda_latent_split.cuh"

using namespace kda;

template <int TILE>
static int check(std::mt19937 &rng, int n, int ranges_most, int longest) {
    LatentDecodeArgs a{};
    std::vector<int32_t> lens(n);
    for (auto &v : lens) v = rng() % 16 == 0 ? (rng() % 2 ? -3 : 1 << 30) : (int)(rng() % (longest + 1));
    a.seq_lens = lens.data(), a.n_seqs = n, a.max_pages = longest / 16 + 1, a.page_shift = 4;

    std::vector<int> request;  // of each tile
    for (int i = 0; i < n; ++i) request.insert(request.end(), tiles_of<TILE>(a, lens[i]), i);
    const int total = (int)request.size(), ranges = std::min(ranges_most, total);
    const Cut cut(total, ranges);
    const bool by_request = n <= ranges_most;

    std::vector<Join> joins(ranges_most, Join{-77, 0, 0, 0});
    std::vector<int> range_of(total);
    for (int r = ranges_most - 1; r >= 0; --r) {  // in any order
        const int begin = cut.begin(std::min(r, ranges)), end = cut.begin(std::min(r + 1, ranges));
        if (begin == end && by_request) continue;
        int first = begin < total ? request[begin] : 0, off = 0;
        while (begin < total && off < begin && request[begin - 1 - off] == first) ++off;
        write_joins(Walk<TILE>{a, first, off, end - begin, lens[first], false}, cut, begin, r, by_request, joins.data());
        for (int t = begin; t < end; ++t) {
            range_of[t] = r;
            if (cut.range_of(t) != r) return printf("tile %d: range %d, not %d\n", t, cut.range_of(t), r), -1;
        }
    }
    std::vector<int> found(n, 0);
    for (int i = 0; i < std::min(n, ranges_most); ++i) {  // the entries that the join reads
        const Join j = joins[i];
        if (j.n == -77) return printf("entry %d is not written\n", i), -1;
        if (j.n < 0) continue;
        if (by_request && j.n != i) return printf("entry %d holds request %d\n", i, j.n), -1;
        ++found[j.n];
        int t0 = 0;
        while (request[t0] != j.n) ++t0;
        int t1 = t0;
        while (t1 + 1 < total && request[t1 + 1] == j.n) ++t1;
        if (j.first != range_of[t0] || j.last != range_of[t1] || j.first == j.last)
            return printf("request %d: ranges %d..%d, not %d..%d\n", j.n, j.first, j.last, range_of[t0], range_of[t1]), -1;
    }
    int crossing = 0;
    for (int i = 0, t = 0; i < n; ++i) {
        const int t1 = t + tiles_of<TILE>(a, lens[i]) - 1;
        const bool crosses = range_of[t] != range_of[t1];
        if (found[i] != crosses) return printf("request %d: %d records, crosses %d\n", i, found[i], crosses), -1;
        crossing += crosses;
        t = t1 + 1;
    }
    return crossing;
}

int main() {
    std::mt19937 rng(1);
    long crossing = 0;
    for (int k = 0; k < 3000; ++k) {
        const int n = 1 + rng() % (k % 3 == 0 ? 4 : 400), ranges = 1 + rng() % 152, longest = 1 + rng() % (n < 5 ? 9000 : 700);
        const int c = k % 2 ? check<48>(rng, n, ranges, longest) : check<64>(rng, n, ranges, longest);
        if (c < 0) return printf("%d requests, %d ranges, up to %d tokens\n", n, ranges, longest), 1;
        crossing += c;
    }
    printf("ok %ld\n", crossing);
}
