// The merge jobs of a chunk attention call (kivi_chunk.cuh) against the CTAs' spans listed one by one: each item that
// several CTAs work on has one job, at the second of them, with its parts, rows, first token and head; these CTAs follow
// each other, and no other CTA has a job.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "kivi_chunk.cuh"

using namespace kivi;

static int fail(const char* what, int round, int c) {
    std::printf("FAILED: %s (round %d, CTA %d)\n", what, round, c);
    return 1;
}

int main() {
    std::mt19937 rng(11);
    auto pick = [&](long long lo, long long hi) { return lo + (long long)(rng() % (unsigned long long)(hi - lo + 1)); };
    long long jobs = 0, most_parts = 0, idle = 0;
    for (int round = 0; round < 3000; ++round) {
        const int nqs[3] = {1, 2, 4};
        const int windows[6] = {0, 0, 1, (int)pick(2, 300), (int)pick(100, 5000), 128};
        ChunkPlan p{nqs[pick(0, 2)], (int)pick(1, 5), windows[pick(0, 5)]};
        const int n = (int)pick(1, 6);
        std::vector<ChunkSeq> s(n);
        long long w = 0, items = 0;
        int tok = (int)pick(0, 9);
        for (int i = 0; i < n; ++i) {
            const int len = (int)(pick(0, 1) ? pick(1, 9) : pick(1, 2000));
            s[i] = ChunkSeq{w, i, len, tok, (int)(32 * pick(0, pick(0, 1) ? 400 : 3)), (int)pick(0, 128), 0};
            tok += len + (int)pick(0, 3);                      // (sequences of the other kernel lie between)
            w += items_weight(p, s[i], item_count(p, len));
            items += item_count(p, len);
        }
        const int ctas = chunk_ctas(w, items * p.Hkv, (int)(pick(0, 1) ? pick(1, 40) : 152));
        struct Item { int seq, m, head; };
        struct Part { Item at; bool begins, ends; };
        std::vector<std::vector<Part>> of(ctas);
        std::vector<MergeJob> got(ctas, MergeJob{0, 0, 0, 0});
        for (int c = 0; c < ctas; ++c) {
            ChunkWalk walk;
            walk.start(&p, s.data(), n, chunk_begin(w, ctas, c), chunk_begin(w, ctas, c + 1));
            for (bool first = true; walk.next(); first = false) {
                if (first) got[c] = merge_job(walk, w, ctas, c);   // (as the kernel's planner does)
                const ChunkSpan& x = walk.s;
                of[c].push_back({{x.seq, x.m, x.head}, x.first == 0, x.last == x.it.hi - x.it.lo});
            }
            idle += of[c].empty();
        }
        std::vector<MergeJob> want(ctas, MergeJob{0, 0, 0, 0});
        for (int c = 0; c < ctas; ++c) {
            for (size_t k = 0; k < of[c].size(); ++k) {
                const Part& x = of[c][k];
                if (!x.begins && k) return fail("a later span that starts inside an item", round, c);
                if (x.ends || !x.begins) continue;
                if (k + 1 != of[c].size()) return fail("a span behind one that does not end", round, c);
                int last = c;                                  // the CTAs that go on with it
                do {
                    if (++last >= ctas) return fail("an item without an end", round, c);
                    if (of[last].empty()) return fail("a CTA without a tile inside an item", round, last);
                    const Part& y = of[last][0];
                    if (y.begins || y.at.seq != x.at.seq || y.at.m != x.at.m || y.at.head != x.at.head)
                        return fail("an item that goes on elsewhere", round, last);
                } while (!of[last][0].ends);
                const int per = kRows / p.nq, t0 = x.at.m * per;
                const int rows = std::min(per, s[x.at.seq].n - t0) * p.nq;
                want[c + 1] = MergeJob{last - c + 1, rows, s[x.at.seq].tok0 + t0, x.at.head};
            }
        }
        for (int c = 0; c < ctas; ++c) {
            if (got[c].parts != want[c].parts) return fail("parts", round, c);
            if (!want[c].parts) continue;
            if (got[c].rows != want[c].rows) return fail("rows", round, c);
            if (got[c].tok != want[c].tok) return fail("first token", round, c);
            if (got[c].head != want[c].head) return fail("head", round, c);
            ++jobs;
            most_parts = std::max<long long>(most_parts, want[c].parts);
        }
    }
    // (there were jobs of two parts and of many, and CTAs that lie in the lead of an item)
    if (jobs < 10000 || most_parts < 20 || !idle) return fail("nothing to check", 0, 0);
    std::printf("OK\n");
    return 0;
}
