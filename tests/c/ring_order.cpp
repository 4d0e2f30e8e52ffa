// Host check of csrc/ring_order.h: a ring filled by one or two copying threads
// is stopped at any moment, and what has to be waited for is compared with what
// is still in flight.
#include <cstdio>
#include <cstdlib>
#include <set>
#include <vector>

#include "ring_order.h"

int main() {
    unsigned seed = 1;
    auto rnd = [&](unsigned n) {
        seed = seed * 1664525u + 1013904223u;
        return (seed >> 8) % n;
    };
    for (int copiers = 1; copiers <= 2; ++copiers)
        for (int stages = copiers; stages <= 16; ++stages)
            for (int trial = 0; trial < 400; ++trial) {
                std::vector<int64_t> put(copiers, 0), holds(stages, -1);
                std::set<int64_t> flight;
                int64_t read = 0;  // entries read so far, in order
                const int moves = (int)rnd(12 * stages + 1);
                for (int m = 0; m < moves; ++m) {
                    const unsigned what = rnd(3);
                    if (what == 0) {  // a thread puts its next entry where the stage's last one was read
                        const int c = (int)rnd(copiers);
                        const int64_t u = c + put[c] * copiers;
                        if (u >= stages && u - stages >= read) continue;
                        holds[u % stages] = u;
                        flight.insert(u);
                        ++put[c];
                    } else if (what == 1 && !flight.empty()) {  // one lands
                        auto it = flight.begin();
                        std::advance(it, rnd((unsigned)flight.size()));
                        flight.erase(it);
                    } else if (holds[read % stages] == read && !flight.count(read)) {  // the next is read
                        ++read;
                    }
                }
                std::set<int64_t> waited;
                for (int i = 0; i < stages; ++i) {
                    const int64_t u = shmm_ring::last_entry(i, stages, copiers, put.data());
                    if (u != holds[i]) {
                        std::printf("stages %d copiers %d stage %d: %lld, holds %lld\n", stages, copiers, i, (long long)u,
                                    (long long)holds[i]);
                        return 1;
                    }
                    waited.insert(u);
                }
                for (int64_t u : flight)
                    if (!waited.count(u)) {
                        std::printf("stages %d copiers %d: entry %lld is in flight\n", stages, copiers, (long long)u);
                        return 1;
                    }
            }
    std::printf("ok\n");
    return 0;
}
