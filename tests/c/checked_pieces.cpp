// Host check of csrc/checked.cuh's comparisons, with SHMM_CHECKED: an access
// of several values is inside its buffer only as a whole.
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#define SHMM_CHECKED
#define __device__
#define __forceinline__ inline
static int atomicCAS(int *p, int expected, int v) {
    const int old = *p;
    if (old == expected) *p = v;
    return old;
}

#include "checked.cuh"

#define CHECK(x)                                        \
    do {                                                \
        if (!(x)) {                                     \
            std::printf("line %d: %s\n", __LINE__, #x); \
            return 1;                                   \
        }                                               \
    } while (0)

int main() {
    using namespace shmm_dev;
    const int64_t big = (int64_t)1 << 40;
    for (const int64_t extent : {(int64_t)8, (int64_t)100, big})
        for (int64_t first = extent - 12; first <= extent + 4; ++first)
            for (int64_t left = 1; left <= 12; ++left) {
                int status = 0;
                const int64_t one_by_one = left < 8 ? left : 8;
                CHECK(piece_in_bounds<true>(&status, first, left, extent) == (first >= 0 && first + 8 <= extent));
                CHECK((status != 0) == !(first >= 0 && first + 8 <= extent));
                status = 0;
                CHECK(piece_in_bounds<false>(&status, first, left, extent) == (first >= 0 && first + one_by_one <= extent));
                CHECK((status != 0) == !(first >= 0 && first + one_by_one <= extent));
            }
    std::printf("ok\n");
    return 0;
}
