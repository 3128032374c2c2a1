// launch_grid_check.cpp -- the grids of launch_grid.hpp next to the limit of
// 2^32 threads along x.  Built and run by tests/test_launch_grid.py.
#include <cstdio>
#include <cstdlib>

#include "launch_grid.hpp"

#define CHECK(c)                                                             \
    do {                                                                     \
        if (!(c)) {                                                          \
            std::fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__); \
            std::abort();                                                    \
        }                                                                    \
    } while (0)

int main() {
    const int64_t limit = int64_t(1) << 32;
    for (const int threads : {64, 128, 256, 512, 1024}) {
        const int64_t edge = limit / threads;
        for (const int64_t blocks : {int64_t(1), int64_t(7), edge - 1, edge, edge + 1, 3 * edge + 5,
                                     int64_t(0x7FFFFFFF)}) {
            if (blocks > 0x7FFFFFFF) continue;
            const dim3 g = dgc::grid_of(blocks, threads);
            CHECK(g.z == 1 && int64_t(g.x) * threads < limit);
            const int64_t all = int64_t(g.x) * g.y;
            CHECK(all >= blocks && all - blocks < dgc::kGridRow);
            CHECK(g.y == 1 ? all == blocks : g.x % 8 == 0);
            CHECK((g.y == 1) == (blocks * threads < limit));
        }
    }
    std::printf("grid check: ok\n");
    return 0;
}
