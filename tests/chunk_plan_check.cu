// The plan of a chunk attention call (kivi_chunk.cuh) against counting one by one: the
// weights of a sequence's items in closed form, and the CTAs' spans, which must
// hold every tile of every item once, in order.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "kivi_chunk.cuh"

using namespace kivi;

static int fail(const char* what) {
    std::printf("FAILED: %s\n", what);
    return 1;
}

int main() {
    std::mt19937 rng(7);
    auto pick = [&](long long lo, long long hi) { return lo + (long long)(rng() % (unsigned long long)(hi - lo + 1)); };
    for (int round = 0; round < 4000; ++round) {
        const int nqs[3] = {1, 2, 4};
        const int windows[6] = {0, 0, 1, (int)pick(2, 300), (int)pick(100, 5000), 128};
        ChunkPlan p{nqs[pick(0, 2)], (int)pick(1, 5), windows[pick(0, 5)]};
        const int n = (int)pick(1, 6);
        std::vector<ChunkSeq> s(n);
        long long w = 0, n_items = 0;
        struct Tile { int seq, m, head, tile; };
        std::vector<Tile> want;
        for (int i = 0; i < n; ++i) {
            const int len = (int)(pick(0, 1) ? pick(1, 9) : pick(1, 2000));
            s[i] = ChunkSeq{w, i, len, 0, (int)(32 * pick(0, pick(0, 1) ? 100 : 3)), (int)pick(0, 128), 0};
            long long sum = 0;
            const int items = item_count(p, len);
            for (int m = 0; m <= items; ++m) {
                if (items_weight(p, s[i], m) != sum * p.Hkv) return fail("closed form");
                if (m == items) break;
                const ChunkItem it = chunk_item(p, s[i], m);
                // the tiles that hold a key that a row of the item sees
                const long long c = (long long)s[i].n_quant + s[i].n_resid;
                long long lo = c + it.t0, hi = 0;
                for (int t = it.t0; t < it.t1; ++t) {
                    const long long a = p.window ? std::max(0LL, c + t - p.window + 1) : 0;
                    lo = std::min(lo, a);
                    hi = std::max(hi, c + t);
                }
                if (it.lo != lo / kTile || it.hi != hi / kTile + 1) return fail("tiles of an item");
                if (it.both != ((it.t1 - it.t0) * p.nq > kHalf)) return fail("item rows");
                for (int h = 0; h < p.Hkv; ++h)
                    for (int t = it.lo; t < it.hi; ++t) want.push_back({i, m, h, t});
                sum += it.total();
            }
            w += sum * p.Hkv;
            n_items += items;
        }
        // (as the call sizes its grid)
        const int ctas = chunk_ctas(w, n_items * p.Hkv, (int)(pick(0, 1) ? pick(1, 40) : 152));
        size_t at = 0;
        long long seen_parts = 0;
        int empty = 0;
        for (int c = 0; c < ctas; ++c) {
            ChunkWalk walk;
            walk.start(&p, s.data(), n, chunk_begin(w, ctas, c), chunk_begin(w, ctas, c + 1));
            int spans = 0, tiles = 0;
            while (walk.next()) {
                ++spans;
                const ChunkSpan& x = walk.s;
                if (x.first != 0 && spans > 1) return fail("a later span that starts inside an item");
                if (x.first != 0) ++seen_parts;
                for (int t = x.first; t < x.last; ++t, ++at, ++tiles) {
                    if (at >= want.size()) return fail("too many tiles");
                    const Tile& y = want[at];
                    if (y.seq != x.seq || y.m != x.m || y.head != x.head || y.tile != x.it.lo + t) return fail("order of tiles");
                }
            }
            empty += !tiles;
        }
        if (at != want.size()) return fail("tiles left over");
        // (a CTA without a tile lies between two items)
        if (empty > 2 * (long long)want.size()) return fail("empty CTAs");
        // the merge's parts of each split item are the spans that continue it
        long long parts = 0;
        for (int c = 1; c < ctas; ++c) {
            ChunkWalk walk;
            walk.start(&p, s.data(), n, chunk_begin(w, ctas, c), chunk_begin(w, ctas, c + 1));
            if (!walk.next()) continue;
            const MergeJob j = merge_job(walk, w, ctas, c);
            if (j.parts) parts += j.parts - 1;
        }
        if (parts != seen_parts) return fail("parts of the merge");
    }
    std::printf("OK\n");
    return 0;
}
