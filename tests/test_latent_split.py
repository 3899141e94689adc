"""How absorbed attention's work is divided, replayed on the host with the functions that
the kernels use: every tile that a unit's rows see is taken once, a unit that a cut falls
into leaves its partial sums exactly where the merge looks for them, and nowhere twice."""
import pytest

from tests.host_util import run_host

HOST = r"""
#include "latent_split.h"
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <vector>
using namespace pkv_split;

struct Part { int worker, slot; };
struct Unit { std::vector<int> taken; std::vector<Part> parts; int kt = 0, lister = -1, listed = 0, wholes = 0; };

// counts of what the batches reach
static long cut_units, early_ends, moved, empty_ranges, long_ranges, wide_merges;

static const char *divide(const std::vector<Seq> &seqs, int heads, const Rule &r)
{
    const int S = (int)seqs.size();
    std::vector<int> begin(S + 1, 0);
    for (int s = 0; s < S; ++s) begin[s + 1] = begin[s] + seq_cost(seqs[s], heads, r.unit);
    const int W = begin[S], nc = sharers(W, r);
    const Cut cut = cut_of(W, nc);
    const int snap = snap_of(cut, r);
    std::map<std::pair<int, int>, Unit> units;
    for (int s = 0; s < S; ++s)
        for (int u = 0; u * r.unit < seqs[s].n * heads; ++u) units[{s, u}].taken.assign(seq_tiles(seqs[s]), 0);
    std::vector<int> used(2 * r.workers, 0);
    // a cut's place: as the thread finds it whose sequences hold it
    auto place = [&](int pos, int &s) -> Place {
        for (s = 0; pos >= begin[s + 1]; ++s) {}
        return moved_cut(pos, begin[s], seq_tiles(seqs[s]), snap);
    };
    for (int k = 0; k < r.workers; ++k) {
        const int w0 = k < nc ? cut.begin(k) : W, w1 = k < nc ? cut.begin(k + 1) : W;
        if (w0 >= w1) continue;
        int s, s1;
        const Place a = place(w0, s);
        const int end = w1 >= W ? W : place(w1, s1).pos;
        if (cut.owner(w0) != k || cut.owner(w1 - 1) != k) return "a tile's owner";
        if (a.pos != w0) ++moved;
        const int tiles = greater(0, end - a.pos);
        if (!tiles) ++empty_ranges;
        Walk w = {s, a.u, a.t, tiles};
        Item it;
        int lists = 0;
        while (next_item(S, heads, r.unit, w, it, [&](int i) { return seqs[i]; })) {
            if (it.s - s >= 40) ++long_ranges;
            Unit &x = units[{it.s, it.r0 / r.unit}];
            x.kt = it.kt;
            for (int j = it.j0; j < it.j1; ++j) ++x.taken[j];
            if (it.whole()) {
                ++x.wholes;
                continue;
            }
            const int slot = own_slot(k, it);
            if (used[slot]++) return "a slot used twice";
            x.parts.push_back({k, slot});
            if (it.j0 == 0) {
                if (lists++) return "two units in a worker's list";
                x.lister = k;
                x.listed = partials(cut, nc, snap, a.pos, tiles, it, k);
                if (it.kt < seq_tiles(it.q) && snap > 0) ++early_ends;
            }
        }
        if (w.left > 0 && k < nc) return "tiles left over";
    }
    for (auto &e : units) {
        const Unit &x = e.second;
        for (int j = 0; j < (int)x.taken.size(); ++j)
            if (x.taken[j] != (j < x.kt)) return x.taken[j] ? "a tile taken twice" : "a tile lost";
        if (x.wholes + (x.lister >= 0) != 1) return "neither whole nor listed";
        if (x.wholes) {
            if (!x.parts.empty()) return "partials of a whole unit";
            continue;
        }
        ++cut_units;
        if (x.listed > 16) ++wide_merges;
        if (x.listed != (int)x.parts.size()) return "partials listed and written differ";
        for (int i = 0; i < x.listed; ++i)
            if (x.parts[i].worker != x.lister + i || x.parts[i].slot != partial_slot(x.lister, i)) return "a partial elsewhere";
    }
    return nullptr;
}

int main(int, char **argv)
{
    const bool one = std::atoi(argv[1]);
    std::mt19937 g(std::atoi(argv[2]));
    auto pick = [&](int lo, int hi) { return lo + (int)(g() % (unsigned)(hi - lo + 1)); };
    auto spread = [&](int hi) { int x = hi; for (int i = pick(0, 6); i > 0; --i) x = pick(0, x); return x; };
    for (int batch = 0; batch < std::atoi(argv[3]); ++batch) {
        const int heads = one ? pick(1, 64) : pick(1, 128), S = 1 + spread(one ? 400 : 200), kind = pick(0, 4);
        std::vector<Seq> seqs;
        int row = 0;
        for (int s = 0; s < S; ++s) {
            int L = kind == 0 ? spread(200) : spread(9000), n = 1;
            if (kind == 2) n = spread(600);
            if (kind == 3) n = pick(0, 3);
            if (kind == 4) n = pick(0, 20) ? 0 : pick(1, 70);
            if (L > 0 && L < n) L = n + spread(300);
            seqs.push_back({row, n, L});
            row += n;
        }
        if (const char *wrong = divide(seqs, heads, one ? ONE : PAIR)) {
            std::printf("%s: %d heads,", wrong, heads);
            for (const Seq &q : seqs) std::printf(" %d/%d", q.n, q.L);
            std::printf("\n");
            return 0;
        }
    }
    std::printf("ok %ld %ld %ld %ld %ld %ld\n", cut_units, early_ends, moved, empty_ranges, long_ranges, wide_merges);
}
"""


@pytest.mark.parametrize("one", [0, 1])
@pytest.mark.parametrize("seed", [1, 2])
def test_every_tile_once_and_every_partial_merged(tmp_path, one, seed):
    out = run_host(tmp_path, HOST, one, seed, 3000).split()
    assert out[0] == "ok", " ".join(out)
    # cut units, among them ones whose causal end comes before their sequence's last tile; cuts that
    # moved, workers left without a tile, ranges of more sequences than are tabled, merges of many
    assert all(int(n) > 0 for n in out[1:]), out
