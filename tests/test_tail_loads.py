"""What the tails' producer waits for before it leaves, at the end of its items and at
every point at which it can give up: the loads that may be in flight (a consumer that
gave up does not wait for them), and no phase that never completes or that another has
followed on its barrier."""
from tests.host_util import run_host

# The producer's order: per item a wait for the slot's last item to be read, its queries,
# then its blocks, each after a wait for its stage; at the end a mark in the next slot.
# `stop` waits succeed.
HOST = r"""
#include "tail_loads.h"
#include <cstdio>
#include <map>
#include <set>
#include <utility>
int main()
{
    const int runs[][4] = {{0, 0, 0, 0}, {1, 0, 0, 0}, {3, 1, 0, 0}, {1, 1, 1, 0}, {9, 2, 5, 1}, {2, 7, 1, 4}};
    for (int ring : {2, 4})
        for (const auto &run : runs)
            for (int stop = 0; stop <= 60; ++stop) {
                constexpr int SLOTS = 2;
                std::map<int, int> stage, slot;      // barrier -> its last phase
                std::set<int> loads;                 // slots whose last phase has loads
                int left = stop, u = 0, asked = 0, k = 0;
                bool ok = true;
                for (;; ++k) {
                    if (k >= SLOTS && !(ok = left-- > 0)) break;
                    slot[k % SLOTS] = k / SLOTS;
                    loads.erase(k % SLOTS);
                    if (k == 4 || run[k] == 0) break;                    // the mark
                    loads.insert(k % SLOTS);
                    asked = k + 1;
                    for (int j = 0; ok && j < run[k]; ++j) {
                        if (u >= ring && !(ok = left-- > 0)) break;
                        stage[u % ring] = u / ring;
                        ++u;
                    }
                    if (!ok) break;
                }
                std::set<std::pair<int, int>> want, got;
                for (const auto &x : stage) want.insert({x.first, x.second});
                for (int s : loads) want.insert({100 + s, slot[s]});
                pkv_tail::drain(u, ring, asked, SLOTS, ok, [&](int i) { got.insert({i % ring, i / ring}); },
                                [&](int i) { got.insert({100 + i % SLOTS, i / SLOTS}); });
                if (want != got) {
                    std::printf("ring %d, %d items, stop %d: %zu waited for, %zu in flight\n", ring, asked, stop, got.size(), want.size());
                    return 0;
                }
            }
    std::printf("ok\n");
}
"""


def test_the_producer_waits_for_what_it_asked_for(tmp_path):
    assert run_host(tmp_path, HOST) == "ok\n"
