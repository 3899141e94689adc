"""What the prompt kernel's producer waits for when it gives up, at every point at which
it can: the loads that may be in flight, and nothing that was never asked for (a phase
without loads never completes, and holds the CTA for the whole limit)."""
from tests.host_util import run_host

# The producer's order: per item its first query tile, per key tile the three parts, and
# before the first tile's values the second query tile.  `stop` requests are made.
HOST = r"""
#include "latent_loads.h"
#include <cstdio>
#include <set>
#include <utility>
using namespace pkv_loads;
int main()
{
    const int items[][2] = {{1, 5}, {4, 1}, {3, 3}};      // key tiles of the items, by run
    for (const auto &run : items)
        for (int stop = 0; stop <= 64; ++stop) {
            Asked a;
            std::set<std::pair<int, int>> made;           // (barrier, phase)
            int left = stop, t = 0;
            auto part = [&](int p) {
                if (left-- <= 0) return false;
                a.tiles[p] = t + 1;
                made.insert({2 * p + (t & 1), t >> 1});
                return true;
            };
            auto query = [&](int g) {
                if (left-- <= 0) return false;
                made.insert({2 * PARTS + g, a.queries[g]++});
                return true;
            };
            bool ok = true;
            for (int k = 0; ok && k < 2; ++k) {
                ok = query(0);
                for (int j = 0; ok && j < run[k]; ++j, t += ok)
                    ok = part(KEY0) && part(KEYS) && (j > 0 || query(1)) && part(VALUES);
            }
            std::set<std::pair<int, int>> waited;
            a.drain([&](int p, int x) { waited.insert({2 * p + (x & 1), x >> 1}); },
                    [&](int g, int x) { waited.insert({2 * PARTS + g, x}); });
            // the last phase of every barrier that has one, and no other
            std::set<std::pair<int, int>> last;
            for (const auto &m : made)
                if (!made.count({m.first, m.second + 1})) last.insert(m);
            if (waited != last) {
                std::printf("stop %d: %zu waited for, %zu in flight\n", stop, waited.size(), last.size());
                return 0;
            }
        }
    std::printf("ok\n");
}
"""


def test_the_producer_waits_for_what_it_asked_for(tmp_path):
    assert run_host(tmp_path, HOST) == "ok\n"
