// Which entries of a shared-memory ring are its stages' last ones: plain
// arithmetic, for the kernels and for host tests.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SHMM_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SHMM_HOST_DEVICE inline
#endif

namespace shmm_ring {

// A ring of `stages` stages holds entry u in stage u % stages.  Copying thread
// c of `copiers` has put entries c, c + copiers, ..., put[c] of them.  Returns
// the last entry put into `stage`, -1 if there is none.  When the number of
// stages is no multiple of the copiers, a stage's entries come from all of
// them in turn.
template <typename Put>
SHMM_HOST_DEVICE int64_t last_entry(int stage, int stages, int copiers, const Put *put) {
    int64_t last = -1;
    for (int c = 0; c < copiers; ++c) {
        int64_t i = put[c] - 1;
        for (int back = 0; back < stages && i >= 0; ++back, --i) {
            const int64_t u = c + i * copiers;
            if (u % stages != stage) continue;
            if (u > last) last = u;
            break;
        }
    }
    return last;
}

}  // namespace shmm_ring
