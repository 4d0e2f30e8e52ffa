// Low-rank adapters of many requests beside a shared (sharded) projection,
// and their gradient.  Row t of the batch uses adapter a = ids[t] (none when
// a is outside [0, n)), a pair of factors down[a] (R x J) and up[a] (R x K):
//   low[t] = A[t] . down[a]^T,       C[t] = base[t] + scale[a] low[t] . up[a]
// and, for the gradient dC of C,
//   dlow[t]  = scale[a] dC[t] . up[a]^T,   dA[t] = base[t] + dlow[t] . down[a]
//   dup[a]   = scale[a] sum over a's rows of low[t]^T dC[t]
//   ddown[a] = sum over a's rows of dlow[t]^T A[t]
// Both factors lie as [n][R][columns], so three kernels make all of it (and a
// fourth sorts the rows by adapter for the last one):
//   project  out[t] = X[t] . W[a]^T     (low, dlow)
//   expand   O[t] = base[t] + S[t] . W[a]   (C, dA)
//   outer    G[a] = sum S[t]^T X[t]     (dup, ddown)
// R is at most 64, so a row's X and O move 2 bytes per 2 R operations, or per
// 6 R where the low values go in three parts: 64 to 192 operations per byte at
// R = 64, against 280 at the rate of tcgen05 and about half of that at that of
// warp instructions.  So all three are bound by HBM up to R = 16; expand, on
// warp instructions, by those too at R = 32 and above.  What each is made of
// follows from where its operands come from:
//   project of few rows, and expand: warp matrix instructions (mma.sync, bf16
//   operands, fp32 accumulators) whose operands come straight from global
//   memory in 16-byte pieces.  The order of the summed index is free, so each
//   thread takes eight consecutive values where the instruction's own layout
//   would give it scattered pairs.  Every byte is used by one thread, once.
//   project of many rows, and outer: tcgen05.  Both operands go through shared
//   memory as they lie (one needs a row tile against all its adapters' factors,
//   the other a group of rows against 128 columns), the sums stay in the TMEM
//   for 16 instructions and then go on in registers.
//   fp32 operands: CUDA cores.
//
// The low-rank rows stay fp32 between the kernels.  Where they are matrix
// operands they are split into three bf16 parts, high bits first: 8 + 8 + 8
// bits, all of an fp32 value's 24, so a product with a bf16 factor loses
// nothing before it is added.  (Two parts would lose up to 2^-16 of it,
// rounding to bf16 2^-8.)
//
// Rows of other adapters never mix: a row's result takes only products with
// its own adapter, and rows of an adapter are gathered by index for its
// gradient, so infinities or NaN in one adapter or row stay there.

#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "checked.cuh"
#include "device_wait.cuh"
#include "pdl.cuh"
#include "shmm_internal.h"
#include "tcgen05.cuh"

namespace {

namespace cg = cooperative_groups;
using bf16 = __nv_bfloat16;
using shmm_dev::in_bounds;
using shmm_dev::piece_in_bounds;
using shmm_pdl::launch_pdl;
using shmm_pdl::launch_pdl_cluster;
using shmm_pdl::pdl_enter;
using shmm_pdl::pdl_release;
using shmm_pdl::pdl_wait;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// A [rows, cols] array as a grid of equal blocks (ranks' shards), row-major
// grid of b1 blocks per row of blocks.
struct Blocks {
    const void *at[SHMM_MAX_RANKS];
    int b1;
    int64_t brows, bcols;
};

struct ProjK {
    Blocks x;
    const void *w;        // [n][R][cols]
    const int *ids;
    const float *scale;   // multiplies the result, or NULL
    float *out;           // [rows][R]
    int *clear;           // set to 0 (for arrange_kernel), or NULL
    int n, R;
    int64_t rows, cols;
    int *status;
};

constexpr int kMaxMaps = 16;  // blocks a tensor-memory projection takes
struct ProjTcK {
    CUtensorMap x[kMaxMaps];  // block i of X: boxes of 128 rows x 64 columns
    CUtensorMap w;            // [n R][cols]: boxes of 16, 32 or 64 rows x 64 columns
    const int *ids;
    const float *scale;
    float *out;
    int *clear;
    int n, R, b1, row_tiles, per_block, chunks;  // row tiles of a block; 64-column chunks of a block, of X
    int64_t brows, bcols, rows;
    int *status;
};

struct ExpandK {
    const void *base[SHMM_MAX_RANKS];  // or NULL: zero
    void *out[SHMM_MAX_RANKS];
    int row0[SHMM_MAX_RANKS], col0[SHMM_MAX_RANKS];  // the rank's box, in blocks
    int64_t brows, bcols;
    const void *w;        // [n][R][cols]
    const int *ids;
    const float *scale;   // or NULL
    const float *s;       // [rows][R]
    int n, R, row_tiles, mt;  // CTAs per box's rows; 16-row tiles of a CTA
    int beside;           // runs beside the kernel before it (see expand_end)
    int64_t rows, cols;
    int *status;
};

struct OuterJob {
    Blocks x;
    const float *s;       // [rows][R]
    const bf16 *parts;    // s by adapter, in parts: [rows][3 RP] (see arrange_kernel)
    const float *scale;   // or NULL
    float *out;           // [n][R][cols]
    int64_t cols;
    int tiles;            // column tiles of the launch
};
// How the CTAs of a column tile share the rows of an adapter that has more of
// them than one CTA's part of all the work: the shares have places, numbered
// over all such adapters, whose CTAs come after those of the n adapters.  The
// host knows the rows, not whose they are, and one adapter with all of them is
// a common batch: 6540 rows of one of 17 adapters, 160 x 544, took 298 us with
// CTAs counted for equal adapters, 66 with these.  (Clusters large enough for
// that, whose idle CTAs leave at once, cost equal adapters 32 us instead of 23:
// they have to find room together.)
struct Shares {
    int2 *of;             // [n]: the adapter's first place and its number of CTAs (1: no places)
    int2 *at;             // [most]: adapter and share of a place (adapter -1: none)
    int *taken;           // places given out
    int *arrived;         // [tiles][most]: CTAs done, counted at the adapter's first place
    float *sums;          // [tiles][most]: their sums
    int most, tiles;      // places and column tiles (times the pieces of R, where CTAs share that too)
    int group, least;     // rows of a group; groups of a CTA
    int64_t room;         // CTAs that the card holds at once
};
struct OuterK {
    OuterJob job[2];
    Shares sh;
    const int *order;     // [rows]: the rows with an adapter, by adapter, each one's ascending
    const int *start;     // [n + 1]: adapter a's are order[start[a]] .. order[start[a + 1] - 1]
    int n, R;
    int64_t rows;
    int *status;
};
struct ArrangeK {
    Shares sh;
    const int *ids;
    const float *s[2];    // either may be NULL
    bf16 *parts[2];
    int *order, *start;
    int n, R;
    int64_t rows;
    int *status;
};

// ---- pieces shared by the kernels -------------------------------------------

struct Raw8 {  // eight bf16 values as they lie in memory
    uint32_t w[4];
};

// Values [c, c + 8) of a row, c < cols; past the row's end, zeros.  VEC: rows
// are whole 16-byte vectors.
template <bool VEC>
__device__ __forceinline__ Raw8 load8(const bf16 *row, int64_t c, int64_t cols) {
    Raw8 r;
    if constexpr (VEC) {
        const uint4 v = *reinterpret_cast<const uint4 *>(row + c);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(row);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = c + 2 * i < cols ? p[c + 2 * i] : 0, hi = c + 2 * i + 1 < cols ? p[c + 2 * i + 1] : 0;
            r.w[i] = lo | (hi << 16);
        }
    }
    return r;
}

// A thread's own queue of 16-byte pieces in shared memory, filled by
// asynchronous copies: more loads in flight than registers would hold.  Every
// piece is read by the thread that asked for it, at [piece][thread], so no
// barrier is needed and no banks conflict.  ok == false: the piece is zeros.
__device__ __forceinline__ void queue16(uint32_t at, const void *from, bool ok) {
    const uint32_t bytes = ok ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void queue_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>  // waits until at most LEFT of this thread's groups are in flight
__device__ __forceinline__ void queue_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}
__device__ __forceinline__ Raw8 read16(const uint4 *p) {
    const uint4 v = *p;
    return Raw8{{v.x, v.y, v.z, v.w}};
}

__device__ __forceinline__ void mma(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// High part of a split: v with its low 16 bits cut (never rounds up to
// infinity).  The rest, v - high, is exact; it is 0 for an infinity, whose
// own difference would be NaN.
__device__ __forceinline__ float cut(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }
__device__ __forceinline__ float rest(float v, float high) { return v == high ? 0.0f : v - high; }
__device__ __forceinline__ uint32_t pack_cut(float lo, float hi) {
    return (__float_as_uint(lo) >> 16) | (__float_as_uint(hi) & 0xffff0000u);
}
// Part `i` of the split of (lo, hi), packed.
template <int PARTS>
__device__ __forceinline__ void split(float lo, float hi, uint32_t *out) {
#pragma unroll
    for (int i = 0; i < PARTS - 1; ++i) {
        const float a = cut(lo), b = cut(hi);
        out[i] = pack_cut(a, b);
        lo = rest(lo, a);
        hi = rest(hi, b);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    out[PARTS - 1] = *reinterpret_cast<const uint32_t *>(&h);
}

// Distinct adapters of the ROWS rows from row t0, in order of first use, into
// list (returns how many); ids[i] = the row's adapter, -1 for none or no row.
template <int ROWS>
__device__ __forceinline__ int distinct(const int *gids, int64_t t0, int64_t rows, int n, int *ids, int *list,
                                        int *count, int *status) {
    if (threadIdx.x < ROWS) {
        const int64_t t = t0 + threadIdx.x;
        int a = -1;
        if (t < rows && in_bounds(status, t, 1, rows)) a = gids[t];
        ids[threadIdx.x] = a >= 0 && a < n ? a : -1;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int have = 0;
#pragma unroll
        for (int i0 = 0; i0 < ROWS; i0 += 32) {
            const int i = i0 + threadIdx.x, a = i < ROWS ? ids[i < ROWS ? i : 0] : -1;
            const unsigned same = __match_any_sync(0xffffffffu, a);
            bool first = a >= 0 && __ffs(same) - 1 == (int)threadIdx.x;
            if (first)
                for (int j = 0; j < have; ++j)
                    if (list[j] == a) {
                        first = false;
                        break;
                    }
            const unsigned m = __ballot_sync(0xffffffffu, first);
            if (first) list[have + __popc(m & ((1u << threadIdx.x) - 1))] = a;
            have += __popc(m);
            __syncwarp();
        }
        if (threadIdx.x == 0) *count = have;
    }
    __syncthreads();
    return *count;
}

// Sums `v` (N values per thread) over the CTA's warps into warp 0, halving
// the warps per step, in a fixed order.  sh holds kWarps / 2 * N * 32 floats.
template <int N>
__device__ __forceinline__ void sum_warps(float *v, float *sh) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
#pragma unroll
    for (int h = kWarps / 2; h > 0; h /= 2) {
        if (warp >= h && warp < 2 * h)
#pragma unroll
            for (int i = 0; i < N; ++i) sh[((warp - h) * N + i) * 32 + lane] = v[i];
        __syncthreads();
        if (warp < h)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += sh[(warp * N + i) * 32 + lane];
        __syncthreads();
    }
}

// Sum over the cluster's CTAs, in order, of the value at `at` in each one's
// shared memory; the loads go out together.
__device__ __forceinline__ float sum_cluster(cg::cluster_group &cluster, float *at, int cs) {
    float v[8], t = 0.0f;
#pragma unroll
    for (int b = 0; b < 8; ++b)
        if (b < cs) v[b] = *cluster.map_shared_rank(at, b);
#pragma unroll
    for (int b = 0; b < 8; ++b)
        if (b < cs) t += v[b];
    return t;
}

// ---- project ---------------------------------------------------------------

// A CTA takes 16 MT rows; its warps share the columns in chunks of 32, and so
// do the CTAs of a cluster along y when there are few rows (their sums meet
// through distributed shared memory, so no partial sum goes to HBM).
// blockIdx.z strides over the tile's distinct adapters.  X and W pieces run
// ST - 1 chunks ahead through the threads' queues, across adapters too.
// 96 rows of 64 adapters, 8192 columns, rank 16: 9.9 us for 27 MB; a launch,
// two dependent reads (the row adapters, then the first chunk) and the join of
// warps and cluster are some 5 of them.  A factor that several row tiles use is
// read, and its sums joined, once in each.
template <int MT, int NT>
struct ProjShape {
    static constexpr int kPieces = 2 * MT + NT;  // per thread and chunk
    static constexpr int kStages = kPieces <= 8 ? 3 : 2;
    static constexpr size_t kQueue = (size_t)kStages * kPieces * kThreads * 16;
    static constexpr size_t kSums = (size_t)kWarps / 2 * MT * NT * 4 * 32 * sizeof(float);
    static constexpr size_t kSmem = kQueue + kSums;
};

template <int MT, int NT, bool VEC>
__global__ void __launch_bounds__(kThreads) project_mma_kernel(const __grid_constant__ ProjK k) {
    pdl_enter();
    using Shape = ProjShape<MT, NT>;
    constexpr int ROWS = 16 * MT, P = Shape::kPieces, ST = Shape::kStages;
    __shared__ int ids[ROWS], list[ROWS], count;
    extern __shared__ __align__(16) uint8_t smem[];
    float *sh = reinterpret_cast<float *>(smem + Shape::kQueue);
    const uint4 *queue = reinterpret_cast<const uint4 *>(smem) + threadIdx.x;  // [stage * P + piece][thread]
    const uint32_t queue_at = shmm_dev::smem_u32(smem) + threadIdx.x * 16;
    cg::cluster_group cluster = cg::this_cluster();
    const int cr = (int)cluster.block_rank(), cs = (int)cluster.num_blocks();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, q = lane & 3, g = lane >> 2;
    const int64_t t0 = (int64_t)blockIdx.x * ROWS;
    if (k.clear && threadIdx.x == 0) *k.clear = 0;
    const int nd = distinct<ROWS>(k.ids, t0, k.rows, k.n, ids, list, &count, k.status);
    // rows without an adapter: zeros
    if (blockIdx.z == 0 && cr == 0)
        for (int i = threadIdx.x; i < ROWS * k.R; i += kThreads)
            if (ids[i / k.R] < 0 && t0 + i / k.R < k.rows && in_bounds(k.status, t0 * k.R + i, 1, k.rows * k.R))
                k.out[t0 * k.R + i] = 0.0f;
    int br[2 * MT], id[2 * MT];
    int64_t off[2 * MT];  // of the row in its block
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
        int64_t t = t0 + (i / 2) * 16 + (i & 1) * 8 + g;
        if (t >= k.rows) t = k.rows - 1;  // never loaded: its adapter is -1
        br[i] = (int)((uint32_t)t / (uint32_t)k.x.brows) * k.x.b1;
        off[i] = (int64_t)((uint32_t)t % (uint32_t)k.x.brows) * k.x.bcols;
        id[i] = ids[(i / 2) * 16 + (i & 1) * 8 + g];
    }
    const int bcols = (int)k.x.bcols, per_block = (bcols + 31) / 32, chunks = per_block * k.x.b1;
    const int step = kWarps * cs, ch0 = warp + kWarps * cr;
    // Piece i of X (row i % 2 MT) and j of W for columns c.. of block blk:
    // its address, and whether it exists.
    auto x_piece = [&](int i, int a, int blk, int c, bool *ok) {
        *ok = id[i] == a && c < bcols && piece_in_bounds<VEC>(k.status, off[i] + c, bcols - c, k.x.brows * k.x.bcols);
        return (const bf16 *)k.x.at[br[i] + blk] + off[i];
    };
    auto w_piece = [&](int j, int a, int blk, int c, bool *ok) {
        const int r = j * 8 + g;
        const int64_t at = ((int64_t)a * k.R + r) * k.cols + (int64_t)blk * bcols;
        *ok = r < k.R && c < bcols && piece_in_bounds<VEC>(k.status, at + c, bcols - c, (int64_t)k.n * k.R * k.cols);
        return (const bf16 *)k.w + at;
    };
    int ask_d = blockIdx.z, ask_ch = ch0;  // the next chunk to ask for
    auto ask = [&](int stage) {
        if (VEC && ch0 < chunks && ask_d < nd) {
            const int a = list[ask_d];
            const int blk = k.x.b1 == 1 ? 0 : ask_ch / per_block, c = (ask_ch - blk * per_block) * 32 + q * 8;
            uint32_t at = queue_at + (uint32_t)(stage * P) * kThreads * 16;
            bool ok;
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i, at += kThreads * 16) {
                const bf16 *p = x_piece(i, a, blk, c, &ok);
                queue16(at, ok ? p + c : (const bf16 *)k.w, ok);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j, at += kThreads * 16) {
                const bf16 *p = w_piece(j, a, blk, c, &ok);
                queue16(at, ok ? p + c : (const bf16 *)k.w, ok);
            }
            ask_ch += step;
            if (ask_ch >= chunks) {
                ask_ch = ch0;
                ask_d += gridDim.z;
            }
        }
        queue_commit();
    };
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) ask(i);
    int stage = 0;
    for (int d = blockIdx.z; d < nd; d += gridDim.z) {
        const int a = list[d];
        float acc[MT * NT * 4];
#pragma unroll
        for (int i = 0; i < MT * NT * 4; ++i) acc[i] = 0.0f;
        for (int ch = ch0; ch < chunks; ch += step) {
            ask(stage == 0 ? ST - 1 : stage - 1);
            queue_wait<ST - 1>();
            const int blk = k.x.b1 == 1 ? 0 : ch / per_block, c = (ch - blk * per_block) * 32 + q * 8;
            Raw8 x[2 * MT];
            const uint4 *from = queue + stage * P * kThreads;
            bool ok;
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
                if constexpr (VEC) {
                    x[i] = read16(from + i * kThreads);
                } else {
                    const bf16 *p = x_piece(i, a, blk, c, &ok);
                    x[i] = ok ? load8<false>(p, c, bcols) : Raw8{{0, 0, 0, 0}};
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                Raw8 b;
                if constexpr (VEC) {
                    b = read16(from + (2 * MT + j) * kThreads);
                } else {
                    const bf16 *p = w_piece(j, a, blk, c, &ok);
                    b = ok ? load8<false>(p, c, bcols) : Raw8{{0, 0, 0, 0}};
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    // A chunk's own sum first, then added: the matrix
                    // instructions cut what they add to (see kTcSegment),
                    // this addition rounds.
                    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    const Raw8 &lo = x[2 * m], &hi = x[2 * m + 1];
                    mma(s, lo.w[0], hi.w[0], lo.w[1], hi.w[1], b.w[0], b.w[1]);
                    mma(s, lo.w[2], hi.w[2], lo.w[3], hi.w[3], b.w[2], b.w[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[(m * NT + j) * 4 + i] += s[i];
                }
            }
            stage = stage + 1 == ST ? 0 : stage + 1;
        }
        sum_warps<MT * NT * 4>(acc, sh);
        if (warp == 0)
#pragma unroll
            for (int i = 0; i < MT * NT * 4; ++i) sh[i * 32 + lane] = acc[i];
        if (cs > 1) cluster.sync();
        else __syncthreads();
        const float scale = k.scale ? k.scale[a] : 1.0f;
        const int part = MT * NT * 4 * 32 / cs;
        for (int e = cr * part + threadIdx.x; e < (cr + 1) * part; e += kThreads) {
            const float v = cs > 1 ? sum_cluster(cluster, sh + e, cs) : sh[e];
            const int i = e / 32, l = e & 31, c = i & 3, j = (i / 4) % NT, m = i / (4 * NT);
            const int row = m * 16 + (l >> 2) + (c >> 1) * 8, r = j * 8 + (l & 3) * 2 + (c & 1);
            if (ids[row] == a && r < k.R && in_bounds(k.status, (t0 + row) * k.R + r, 1, k.rows * k.R))
                k.out[(t0 + row) * k.R + r] = k.scale ? v * scale : v;
        }
        if (cs > 1) cluster.sync();  // nobody overwrites, or leaves with, what another CTA still reads
        else __syncthreads();
    }
    queue_wait<0>();
}

// Many rows: 128 rows per CTA on tcgen05.  One thread streams X in boxes of
// 128 rows x 64 columns, with the boxes of the adapters the tile uses (128
// factor rows per pass, each a product of its own into its own TMEM
// columns), through a ring of shared-memory stages; one thread issues the
// products; eight warps read the result out of TMEM, a row per thread.  A
// cluster along y shares the columns, its sums meeting through distributed
// shared memory in order.  Beside the warp instructions above it: the factor
// is read once per 128 rows instead of per 32, and no thread spends
// instructions on addresses, which bounded them.
// 8192 rows: 64 us at 16384 columns, rank 32 (268 MB, 4.2 TB/s); 90 us at 28672
// columns, rank 16 (470 MB, 5.2 TB/s).  What is left is the start and the join of
// each cluster (5 us of 17 at 4096 rows of 4096 columns) and the places that
// clusters of a power of two leave empty (256 of 304 taken in these).  Ranks to
// 32 spill 16 bytes a thread.
constexpr int kTcThreads = 320, kTcStages = 3;
// Chunks summed in the tensor memory before their sum is added in registers:
// 16 instructions.  The tensor core's own fp32 additions cut instead of
// rounding, so their error grows with their number (some 4e-8 of the sum per
// instruction: 1e-5 over a 7168-column share); in registers they round.
constexpr int kTcSegment = 4;
constexpr int kTcSum = 132;  // fp32 of a row of sums: whole 16-byte vectors
// Two CTAs per SM (61 us against 72 with one and twice the stages, at 8192 x
// 16384, rank 32).  A pass takes 128 factor rows, whose sums are 64 registers a
// thread: a smaller one would make the tile with the most adapters, which then
// streams X twice, the one that ends last.
constexpr int kTcCols = 128;
constexpr uint32_t kTcStage = 16384 + kTcCols * 128, kTcRing = kTcStages * kTcStage;
constexpr size_t kTcSmem = kTcRing + 1024;
static_assert(128 * kTcSum * 4 <= kTcRing, "the sums take the ring's memory");

template <int RP>
__global__ void __launch_bounds__(kTcThreads, 2) project_tc_kernel(const __grid_constant__ ProjTcK k) {
    pdl_wait();
    constexpr int ROWS = 128, PER = kTcCols / RP, S = kTcStages, MINE = kTcCols / 2;  // MINE: of a reading warp
    __shared__ int ids[ROWS], list[ROWS], count, abort_flag;
    __shared__ float scales[PER];
    __shared__ __align__(8) uint64_t bars[2 * S + 5];
    __shared__ uint32_t tmem_at;
    extern __shared__ uint8_t raw_smem[];
    uint8_t *tiles = raw_smem + (1024 - (shmm_dev::smem_u32(raw_smem) & 1023)) % 1024;
    const uint32_t tiles_at = shmm_dev::smem_u32(tiles);
    cg::cluster_group cluster = cg::this_cluster();
    const int cr = (int)cluster.block_rank(), cs = (int)cluster.num_blocks();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    auto full = [&](int s) { return shmm_dev::smem_u32(&bars[s]); };
    auto empty = [&](int s) { return shmm_dev::smem_u32(&bars[S + s]); };
    auto done = [&](int b) { return shmm_dev::smem_u32(&bars[2 * S + b]); };         // a segment is in buffer b
    auto drained = [&](int b) { return shmm_dev::smem_u32(&bars[2 * S + 2 + b]); };  // and has been read (8 warps)
    const uint32_t finished = shmm_dev::smem_u32(&bars[2 * S + 4]);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * S + 5; ++i)
            shmm_dev::mbar_init(shmm_dev::smem_u32(&bars[i]), i == 2 * S + 2 || i == 2 * S + 3 ? 8 : 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        shmm_tc::fence_async();
    }
    if (warp == 1) shmm_tc::tmem_alloc(shmm_dev::smem_u32(&tmem_at), 256);
    shmm_tc::fence_before();
    const int brow = blockIdx.x / k.row_tiles, l0 = (int)(blockIdx.x % k.row_tiles) * ROWS;
    const int64_t t0 = brow * k.brows + l0, t1 = (brow + 1) * k.brows;
    if (k.clear && threadIdx.x == 0) *k.clear = 0;
    const int nd = distinct<ROWS>(k.ids, t0, t1, k.n, ids, list, &count, k.status);
    shmm_tc::fence_after();
    // Only now may the next kernel's CTAs come: one that takes all of an SM's
    // TMEM and then waits for this kernel must not get there first.
    pdl_release();
    const uint32_t tmem = tmem_at;
    if (cr == 0)  // rows without an adapter: zeros
        for (int i = threadIdx.x; i < ROWS * k.R; i += kTcThreads)
            if (ids[i / k.R] < 0 && t0 + i / k.R < t1 && in_bounds(k.status, t0 * k.R + i, 1, k.rows * k.R))
                k.out[t0 * k.R + i] = 0.0f;
    const int lo = (int)((int64_t)k.chunks * cr / cs), hi = (int)((int64_t)k.chunks * (cr + 1) / cs);
    // Producer and issuer are one thread each, so their own instructions are
    // what a chunk costs them (a division or two each made it 1500 cycles):
    // both walk stages and blocks by counting.
    uint32_t stage = 0, phase = 0, asked = 0;
    uint32_t uses = 0;  // segments so far; segment u is the (u / 2)-th in buffer u % 2
    const int blk0 = k.b1 == 1 ? 0 : lo / k.per_block;
    bool ok = true;
    for (int p0 = 0, pass = 0; p0 < nd; p0 += PER, ++pass) {
        const int na = nd - p0 < PER ? nd - p0 : PER;
        if (warp == 2 && lane < na) scales[lane] = k.scale ? k.scale[list[p0 + lane]] : 1.0f;
        if (warp == 0 && lane == 0) {
            const CUtensorMap *x = &k.x[brow * k.b1 + blk0];
            int c = (lo - blk0 * k.per_block) * 64, wc = (int)(blk0 * k.bcols) + c;
            const int w_row = list[p0] * k.R;
            const uint32_t bytes = 16384 + na * RP * 128;
            for (int ch = lo; ch < hi; ++ch) {
                ok = ok && shmm_dev::mbar_wait(empty(stage), phase ^ 1, &abort_flag, k.status);
                if (!ok) break;
                const uint32_t at = tiles_at + stage * kTcStage, bar = full(stage);
                shmm_dev::mbar_expect_tx(bar, bytes);
                shmm_tc::load_box(at, x, bar, c, l0);
                shmm_tc::load_box(at + 16384, &k.w, bar, wc, w_row);
                for (int i = 1; i < na; ++i)
                    shmm_tc::load_box(at + 16384 + i * RP * 128, &k.w, bar, wc, list[p0 + i] * k.R);
                ++asked;
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
                c += 64;
                wc += 64;
                if (c >= k.bcols) {  // the next block
                    wc += (int)k.bcols - c;
                    c = 0;
                    ++x;
                }
            }
        } else if (warp == 1 && lane == 0) {
            // The pass's factors lie below one another: one operand of na RP
            // rows.  An instruction takes some 130 cycles however narrow it
            // is, so one for all of them, not one each.
            const uint64_t base = shmm_tc::operand(tiles_at, 16, 1024);
            const uint32_t idesc = shmm_tc::instruction(na * RP, false, false);
            int left = 0;  // chunks of the segment still to come
            for (int ch = lo; ch < hi; ++ch) {
                const uint32_t buf = uses & 1;
                const bool start = left == 0;
                if (start) {
                    left = kTcSegment;
                    if (uses >= 2) ok = ok && shmm_dev::mbar_wait(drained(buf), (uses / 2 - 1) & 1, &abort_flag, k.status);
                }
                ok = ok && shmm_dev::mbar_wait(full(stage), phase, &abort_flag, k.status);
                if (!ok) break;
                shmm_tc::fence_after();
                const uint64_t xa = base + ((stage * kTcStage) >> 4);  // addresses in units of 16 bytes
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    shmm_tc::mma_issue(tmem + buf * 128, xa + kk * 2, xa + 1024 + kk * 2, idesc, !start || kk > 0);
                shmm_tc::mma_commit(empty(stage));
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
                if (--left == 0 || ch + 1 == hi) {
                    left = 0;
                    shmm_tc::mma_commit(done(buf));
                    ++uses;
                }
            }
            // Not cut short by an abort: the products in flight read shared memory.
            shmm_tc::mma_commit(finished);
            shmm_dev::mbar_wait(finished, pass & 1, &abort_flag, k.status, false);
        }
        __syncwarp();
        float *sums = reinterpret_cast<float *>(tiles);  // [row][kTcSum], once the products are done
        if (warp >= 2) {
            // Warp: 32 rows, half of the columns, from c0 on.
            const int quad = warp & 3, row = quad * 32 + lane, c0 = (warp - 2) / 4 * MINE;
            float acc[MINE];
#pragma unroll
            for (int c = 0; c < MINE; ++c) acc[c] = 0.0f;
            for (int ch = lo; ch < hi; ch += kTcSegment, ++uses) {
                const uint32_t buf = uses & 1;
                ok = ok && shmm_dev::mbar_wait(done(buf), uses / 2 & 1, &abort_flag, k.status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                shmm_tc::fence_after();
#pragma unroll
                for (int c = 0; c < MINE; c += 16) {
                    if (c0 + c >= na * RP) continue;
                    float v[16];
                    shmm_tc::tmem_read16(tmem + ((uint32_t)(quad * 32) << 16) + buf * 128 + c0 + c, v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[c + j] += v[j];
                }
                shmm_tc::fence_before();
                __syncwarp();
                if (lane == 0) shmm_dev::mbar_arrive(drained(buf));
            }
            // The ring's memory takes the sums once every warp's last segment
            // is done, which the last product is part of.
            asm volatile("bar.sync 1, 256;" ::: "memory");
#pragma unroll
            for (int c = 0; c < MINE; c += 16) {
                if (c0 + c >= na * RP) continue;
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    *reinterpret_cast<float4 *>(sums + row * kTcSum + c0 + c + j) =
                        make_float4(acc[c + j], acc[c + j + 1], acc[c + j + 2], acc[c + j + 3]);
            }
        }
        cluster.sync();
        const int r0 = ROWS * cr / cs, r1 = ROWS * (cr + 1) / cs;
        const int vecs = na * RP / 4;
        for (int e = threadIdx.x; e < (r1 - r0) * vecs; e += kTcThreads) {
            const int row = r0 + e / vecs, c = e % vecs * 4, i = c / RP, r = c % RP;
            if (r >= k.R || ids[row] != list[p0 + i]) continue;
            float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1  // at 96 registers a thread
            for (int b = 0; b < cs; ++b) {
                const float4 v = *cluster.map_shared_rank(reinterpret_cast<float4 *>(sums + row * kTcSum + c), b);
                t.x += v.x;
                t.y += v.y;
                t.z += v.z;
                t.w += v.w;
            }
            const float *u = &t.x;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (r + j < k.R && in_bounds(k.status, (t0 + row) * k.R + r + j, 1, k.rows * k.R))
                    k.out[(t0 + row) * k.R + r + j] = k.scale ? u[j] * scales[i] : u[j];
        }
        // The sums are read, by other CTAs too: after this barrier the stages
        // may be filled again.  That is the async proxy's writing, so every
        // reader orders its loads, remote ones among them, before the barrier
        // and the copying thread its copies after it; a fence of the CTA's own
        // shared memory would say nothing about a peer's.
        shmm_tc::fence_async_cluster();
        cluster.sync();
        shmm_tc::fence_async_cluster();
        shmm_tc::fence_after();
    }
    // Never leave a load into shared memory in flight.
    if (warp == 0 && lane == 0)
        for (uint32_t u = asked > S ? asked - S : 0; u < asked; ++u)
            shmm_dev::mbar_wait(full(u % S), u / S & 1, &abort_flag, k.status, false);
    __syncwarp();
    shmm_tc::fence_before();
    __syncthreads();
    shmm_tc::fence_after();
    if (warp == 1) shmm_tc::tmem_free(tmem, 256);
}

template <typename T>
__device__ __forceinline__ float as_float(T v) { return (float)v; }

// acc += s[0..3] x, the four values of s (in shared memory) in one load.
__device__ __forceinline__ void fma4(float *acc, const float *s, float x) {
    const float4 v = *reinterpret_cast<const float4 *>(s);
    acc[0] = fmaf(v.x, x, acc[0]);
    acc[1] = fmaf(v.y, x, acc[1]);
    acc[2] = fmaf(v.z, x, acc[2]);
    acc[3] = fmaf(v.w, x, acc[3]);
}

// Any types, on CUDA cores: 32 rows x 16 NR adapter rows per CTA, columns in
// chunks of 32 through shared memory, the cluster sharing the chunks.  Shared
// memory is read four columns at a time (pitch 36: no bank conflicts): one
// load per value made its reads the bound.  A chunk is summed by itself and
// then added, so a long share's rounding grows with its chunks, not its columns.
template <typename TX, typename TW, int NR>
__global__ void __launch_bounds__(kThreads) project_simt_kernel(const __grid_constant__ ProjK k) {
    pdl_enter();
    constexpr int ROWS = 32, RP = 16 * NR;
    __shared__ int ids[ROWS], list[ROWS], count, block_row[ROWS];
    __shared__ int64_t row_at[ROWS];  // in its row of blocks
    __shared__ __align__(16) float xs[ROWS][36], ws[RP][36];
    __shared__ float part[ROWS * RP];
    cg::cluster_group cluster = cg::this_cluster();
    const int cr = (int)cluster.block_rank(), cs = (int)cluster.num_blocks();
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const int64_t t0 = (int64_t)blockIdx.x * ROWS;
    if (k.clear && threadIdx.x == 0) *k.clear = 0;
    const int nd = distinct<ROWS>(k.ids, t0, k.rows, k.n, ids, list, &count, k.status);
    if (blockIdx.z == 0 && cr == 0)
        for (int i = threadIdx.x; i < ROWS * k.R; i += kThreads)
            if (ids[i / k.R] < 0 && t0 + i / k.R < k.rows && in_bounds(k.status, t0 * k.R + i, 1, k.rows * k.R))
                k.out[t0 * k.R + i] = 0.0f;
    if (threadIdx.x < ROWS) {
        block_row[threadIdx.x] = (int)((t0 + threadIdx.x) / k.x.brows);
        row_at[threadIdx.x] = (t0 + threadIdx.x) % k.x.brows * k.x.bcols;
    }
    __syncthreads();
    const int bcols = (int)k.x.bcols, per_block = (bcols + 31) / 32, chunks = per_block * k.x.b1;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    for (int d = blockIdx.z; d < nd; d += gridDim.z) {
        const int a = list[d];
        const int64_t w_at = (int64_t)a * k.R * k.cols;
        const TW *w = (const TW *)k.w + w_at;
        float acc[2][NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) acc[0][i] = acc[1][i] = 0.0f;
        // A chunk's values, asked for while the one before it is computed.
        float xv[ROWS / kWarps], wv[RP / kWarps];
        auto fetch = [&](int ch) {
            const int blk = ch / per_block, c = (ch - blk * per_block) * 32 + lane;
            const bool in = ch < chunks && c < bcols;
#pragma unroll
            for (int i = 0; i < ROWS / kWarps; ++i) {
                const int row = warp + i * kWarps;
                const int64_t at = row_at[row] + c;
                xv[i] = in && ids[row] == a && in_bounds(k.status, at, 1, k.x.brows * k.x.bcols)
                            ? as_float(((const TX *)k.x.at[block_row[row] * k.x.b1 + blk])[at])
                            : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < RP / kWarps; ++i) {
                const int r = warp + i * kWarps;
                const int64_t at = r * k.cols + (int64_t)blk * bcols + c;
                wv[i] = in && r < k.R && in_bounds(k.status, w_at + at, 1, (int64_t)k.n * k.R * k.cols) ? as_float(w[at])
                                                                                                        : 0.0f;
            }
        };
        fetch(cr);
        for (int ch = cr; ch < chunks; ch += cs) {
#pragma unroll
            for (int i = 0; i < ROWS / kWarps; ++i) xs[warp + i * kWarps][lane] = xv[i];
#pragma unroll
            for (int i = 0; i < RP / kWarps; ++i) ws[warp + i * kWarps][lane] = wv[i];
            __syncthreads();
            fetch(ch + cs);
            float sum[2][NR];
#pragma unroll
            for (int i = 0; i < NR; ++i) sum[0][i] = sum[1][i] = 0.0f;
#pragma unroll
            for (int c2 = 0; c2 < 32; c2 += 4) {
                const float4 x0 = *reinterpret_cast<const float4 *>(&xs[ty][c2]);
                const float4 x1 = *reinterpret_cast<const float4 *>(&xs[ty + 16][c2]);
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const float4 v = *reinterpret_cast<const float4 *>(&ws[tx + 16 * i][c2]);
                    sum[0][i] = fmaf(x0.w, v.w, fmaf(x0.z, v.z, fmaf(x0.y, v.y, fmaf(x0.x, v.x, sum[0][i]))));
                    sum[1][i] = fmaf(x1.w, v.w, fmaf(x1.z, v.z, fmaf(x1.y, v.y, fmaf(x1.x, v.x, sum[1][i]))));
                }
            }
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                acc[0][i] += sum[0][i];
                acc[1][i] += sum[1][i];
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            part[ty * RP + tx + 16 * i] = acc[0][i];
            part[(ty + 16) * RP + tx + 16 * i] = acc[1][i];
        }
        if (cs > 1) cluster.sync();
        else __syncthreads();
        const int share = ROWS * RP / cs;
        for (int e = cr * share + threadIdx.x; e < (cr + 1) * share; e += kThreads) {
            const float v = cs > 1 ? sum_cluster(cluster, part + e, cs) : part[e];
            const int row = e / RP, r = e % RP;
            if (ids[row] == a && r < k.R && in_bounds(k.status, (t0 + row) * k.R + r, 1, k.rows * k.R))
                k.out[(t0 + row) * k.R + r] = k.scale ? v * k.scale[a] : v;
        }
        if (cs > 1) cluster.sync();
        else __syncthreads();
    }
}

// ---- expand ----------------------------------------------------------------

// Eight consecutive values of base and output, as they lie in memory.
template <typename T, bool VEC>
struct Out8 {
    static constexpr int W = sizeof(T) / 2;  // 16-byte vectors
    uint4 b[W];
    __device__ void load(const T *p, int left) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < W; ++i) b[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
        } else if constexpr (sizeof(T) == 4) {
            uint32_t *w = reinterpret_cast<uint32_t *>(b);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = i < left ? __float_as_uint(p[i]) : 0;
        } else {
            const Raw8 r = load8<false>(p, 0, left);
            b[0] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        }
    }
    __device__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) b[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ void add(const float *v) {  // rounds once
        uint32_t *w = reinterpret_cast<uint32_t *>(b);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) + v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(w[i] << 16) + v[2 * i],
                                                               __uint_as_float(w[i] & 0xffff0000u) + v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
    }
    __device__ void store(T *p, int left) const {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < W; ++i) __stcs(reinterpret_cast<uint4 *>(p) + i, b[i]);
        } else {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(b);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) {
                    if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t *>(p)[i] = w[i];
                    else reinterpret_cast<uint16_t *>(p)[i] = (uint16_t)(w[i / 2] >> (i & 1) * 16);
                }
        }
    }
};

// A CTA takes k.mt row tiles of 16 of one rank's box x 512 columns (64 per
// warp; FEW: one row tile, many adapters).  An
// adapter's 16 KT x 64 piece stays in registers until a row tile needs
// another's.  The product's columns are dealt out
// so that each thread ends with two runs of eight consecutive ones, and four
// threads with 64 bytes of a row side by side: base and output move in whole
// sectors.  The base of up to kRing row tiles is in flight through the
// threads' queues from the start.
// 86 us for 537 MB at rank 16 (6.2 TB/s): HBM.  205 us for 8192 x 4096 to each of
// 8 ranks at rank 32 (1.07 GB, 5.2 TB/s): HBM and the matrix instructions of
// three parts (two would take 182, and 82 at rank 16, and lose 2^-16 of the low
// values).  Few rows (96, 8192 columns, 64 adapters): 13 us, one of them beside
// the projection; latency as in project_mma_kernel.
// blockIdx.x: rank x row tile; blockIdx.z strides over a row tile's adapters
// (and z = 0 copies the rows without one).
constexpr int kMaxRowTiles = 16;
template <bool FEW, int KT, typename TO>
struct ExpandShape {
    static constexpr int kParts = 3;  // of the low values: all their bits (see the top)
    static constexpr int kPitch = 16 * KT + 8;  // bf16: a row's start moves by 4 banks, fragments do not conflict
    static constexpr int kWords = sizeof(TO) / 2;  // 16-byte pieces of eight outputs
    static constexpr int kRing = FEW ? 1 : kWords == 1 ? 3 : 2;
    static constexpr size_t kBase = (size_t)kRing * 4 * kWords * kThreads * 16;
    // FEW: factor pieces of the next kAhead adapters queued too.
    static constexpr int kAhead = !FEW ? 0 : KT == 1 ? 4 : 2;
    static constexpr size_t kQueue = kBase + (size_t)kAhead * 4 * KT * kThreads * 16;
    static size_t smem(int row_tiles) { return kQueue + (size_t)kParts * 16 * row_tiles * kPitch * 2; }
};

// What may be done before the kernel in front of this one is over.  In both
// calls that kernel has itself waited for everything that the call was given,
// so row adapters, factors and base can be read, and factors and base are on
// their way when it ends; the forward call's is the projection, whose low rows
// are waited for.  The backward call's is the factor gradients' kernel, of
// which expand needs nothing, while it writes none of that one's inputs (dA is
// neither A nor dC): its CTAs work on the SMs that kernel's last ones leave
// empty, and wait for it at their end, so that the end of this kernel is the
// end of both.
__device__ __forceinline__ void expand_low(const ExpandK &k) {
    if (!k.beside) pdl_wait();
}
__device__ __forceinline__ void expand_end(const ExpandK &k) {
    if (k.beside) pdl_wait();
}

template <bool FEW, int KT, bool VEC, typename TO>
__global__ void __launch_bounds__(kThreads, sizeof(TO) == 4 || KT > 2 ? 1 : 2)
    expand_mma_kernel(const __grid_constant__ ExpandK k) {
    pdl_release();
    using Shape = ExpandShape<FEW, KT, TO>;
    constexpr int RP = 16 * KT, PITCH = Shape::kPitch, PARTS = Shape::kParts;
    constexpr int RING = Shape::kRing, WORDS = Shape::kWords;
    constexpr int AHEAD = FEW && VEC ? Shape::kAhead : 0;
    const int MT = FEW ? 1 : k.mt, ROWS = 16 * MT;
    __shared__ int ids[16 * kMaxRowTiles];
    __shared__ float row_scale[16 * kMaxRowTiles];
    extern __shared__ __align__(16) uint8_t smem[];
    bf16 *ss = reinterpret_cast<bf16 *>(smem + Shape::kQueue);  // [PARTS][ROWS][PITCH]
    const uint4 *queue = reinterpret_cast<const uint4 *>(smem) + threadIdx.x;  // [(slot * 4 + i) * WORDS + w][thread]
    const uint32_t queue_at = shmm_dev::smem_u32(smem) + threadIdx.x * 16;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, q = lane & 3, g = lane >> 2;
    const int rank = blockIdx.x / k.row_tiles;
    const int64_t l0 = (int64_t)(blockIdx.x % k.row_tiles) * ROWS;  // in the rank's box
    const int64_t t0 = k.row0[rank] * k.brows + l0;                 // in the batch
    const int nrows = (int)(k.brows - l0 < ROWS ? k.brows - l0 : ROWS);
    const int64_t c0 = (int64_t)blockIdx.y * 512 + warp * 64;
    const TO *base = (const TO *)k.base[rank];
    TO *out = (TO *)k.out[rank];
    // Piece i of row tile m: row half i / 2, columns 32 (i % 2) + 8 q of the
    // warp's 64.  `at`: its place in the box.
    const int64_t at0 = (l0 + g) * k.bcols + c0 + 8 * q;
    const int left0 = (int)(k.bcols - c0 - 8 * q);
    auto has = [&](int m, int i, int64_t *at, int *left) {
        *at = at0 + (int64_t)(m * 16 + (i >> 1) * 8) * k.bcols + 32 * (i & 1);
        *left = left0 - 32 * (i & 1);
        return m * 16 + (i >> 1) * 8 + g < nrows && *left > 0 &&
               piece_in_bounds<VEC>(k.status, *at, *left, k.brows * k.bcols);
    };
    auto ask = [&](int m, int slot) {  // row tile m into a slot of the queue
        if (VEC && m < MT) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                int64_t at;
                int left;
                const bool ok = has(m, i, &at, &left) && base;
#pragma unroll
                for (int w = 0; w < WORDS; ++w)
                    queue16(queue_at + (uint32_t)((slot * 4 + i) * WORDS + w) * kThreads * 16,
                            ok ? (const void *)(base + at + w * 8 / WORDS) : k.w, ok);
            }
        }
        queue_commit();
    };
#pragma unroll
    for (int m = 0; m < RING; ++m) ask(m, m);
    int my_id = -1;  // of row threadIdx.x
    if ((int)threadIdx.x < nrows && in_bounds(k.status, t0 + threadIdx.x, 1, k.rows)) my_id = k.ids[t0 + threadIdx.x];
    auto low_rows = [&] {  // their parts into shared memory
        expand_low(k);
#pragma unroll 4
        for (int i = threadIdx.x; i < ROWS * RP / 2; i += kThreads) {
            const int row = i / (RP / 2), r = (i % (RP / 2)) * 2;
            float lo = 0.0f, hi = 0.0f;
            if (row < nrows) {
                const int64_t at = (t0 + row) * k.R + r;
                if (r < k.R && in_bounds(k.status, at, 1, k.rows * k.R)) lo = k.s[at];
                if (r + 1 < k.R && in_bounds(k.status, at + 1, 1, k.rows * k.R)) hi = k.s[at + 1];
            }
            uint32_t p[PARTS];
            split<PARTS>(lo, hi, p);
#pragma unroll
            for (int h = 0; h < PARTS; ++h) *reinterpret_cast<uint32_t *>(ss + (h * ROWS + row) * PITCH + r) = p[h];
        }
    };
    // FEW: waited for after the first factor pieces are on their way.  Else at
    // once, while the row adapters are (after them it costs a start of its own:
    // 10 us of the longest case above).
    if constexpr (!FEW) low_rows();
    if ((int)threadIdx.x < ROWS) {
        my_id = my_id >= 0 && my_id < k.n ? my_id : -1;
        ids[threadIdx.x] = my_id;
        row_scale[threadIdx.x] = k.scale && my_id >= 0 ? k.scale[my_id] : 1.0f;
    }
    __syncthreads();
    if (c0 >= k.bcols) {
        if constexpr (FEW) {
            low_rows();
            __syncthreads();
        }
        queue_wait<0>();
        expand_end(k);
        return;
    }
    const int64_t col = k.col0[rank] * k.bcols;  // of the box in the factor
    int held = -1;                               // the adapter in b
    uint32_t b[KT][8][2];
    Raw8 raw[KT][4];
    const uint4 *w_queue = queue + Shape::kBase / 16;
    // Adapter a's pieces, into registers or (to >= 0) into place `to` of the
    // queue.
    auto load_w = [&](int a, int to = -1) {
        const bf16 *w = (const bf16 *)k.w + (int64_t)a * k.R * k.cols + col;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = kt * 16 + 2 * q + (i & 1) + (i >> 1) * 8;
                const int64_t c = c0 + 32 * (g & 1) + 8 * (g >> 1);  // product column j of lane group g: this one + j
                const bool ok = r < k.R && c < k.bcols &&
                                piece_in_bounds<VEC>(k.status, ((int64_t)a * k.R + r) * k.cols + col + c, k.bcols - c,
                                                     (int64_t)k.n * k.R * k.cols);
                if (AHEAD && to >= 0) {
                    queue16(queue_at + (uint32_t)Shape::kBase + (uint32_t)((to * KT + kt) * 4 + i) * kThreads * 16,
                            ok ? (const void *)(w + r * k.cols + c) : k.w, ok);
                } else {
                    raw[kt][i] = Raw8{{0, 0, 0, 0}};
                    if (ok) raw[kt][i] = load8<VEC>(w + r * k.cols, c, k.bcols);
                }
            }
    };
    int slot = 0;
#pragma unroll 1
    for (int m = 0; m < MT; ++m) {
        const int id = ids[m * 16 + (lane & 15)];
        const unsigned with = __ballot_sync(0xffffffffu, id >= 0) & 0xffffu;
        // The next of this CTA's adapters of the row tile (-1: none left)
        // and its rows.
        struct Left {
            unsigned todo;
            int d;
        };
        auto advance = [&](Left &left, unsigned *rows) {
            while (left.todo) {
                const int a = __shfl_sync(0xffffffffu, id, __ffs(left.todo) - 1);
                *rows = __ballot_sync(0xffffffffu, id == a) & 0xffffu;
                left.todo &= ~*rows;
                if (left.d++ % gridDim.z == blockIdx.z) return a;
            }
            return -1;
        };
        Left left{with, 0}, ahead{with, 0};
        int w_at = 0;  // the place of the next adapter in the queue
        auto ask_w = [&](int to) {
            unsigned rows;
            const int a = advance(ahead, &rows);
            if (a >= 0) load_w(a, to);
            queue_commit();
        };
        if constexpr (AHEAD > 0) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) ask_w(i);
        }
        if constexpr (FEW) {  // one row tile
            low_rows();
            __syncthreads();
        }
        queue_wait<RING - 1 + AHEAD>();
        Out8<TO, VEC> now[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (VEC) {
#pragma unroll
                for (int w = 0; w < WORDS; ++w) now[i].b[w] = queue[((slot * 4 + i) * WORDS + w) * kThreads];
            } else {
                int64_t at;
                int left;
                if (has(m, i, &at, &left) && base) now[i].load(base + at, left);
                else now[i].zero();
            }
        }
        if (blockIdx.z == 0 && base != out) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                int64_t at;
                int left;
                if (!(with >> ((i >> 1) * 8 + g) & 1) && has(m, i, &at, &left)) now[i].store(out + at, left);
            }
        }
        unsigned rows = 0;
        for (int a = advance(left, &rows); a >= 0; a = advance(left, &rows)) {
            if constexpr (AHEAD > 0) {
                queue_wait<AHEAD - 1>();
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) raw[kt][i] = read16(w_queue + ((w_at * KT + kt) * 4 + i) * kThreads);
            }
            if (AHEAD || a != held) {
                held = a;
                if (!AHEAD) load_w(a);
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const Raw8 *v = raw[kt];
                        b[kt][j][0] = __byte_perm(v[0].w[j / 2], v[1].w[j / 2], (j & 1) ? 0x7632 : 0x5410);
                        b[kt][j][1] = __byte_perm(v[2].w[j / 2], v[3].w[j / 2], (j & 1) ? 0x7632 : 0x5410);
                    }
            }
            float acc[8][4];
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int h = PARTS - 1; h >= 0; --h) {
                    uint32_t f[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        f[i] = *reinterpret_cast<const uint32_t *>(ss + (h * ROWS + m * 16 + g + (i & 1) * 8) * PITCH +
                                                                   kt * 16 + 2 * q + (i >> 1) * 8);
#pragma unroll
                    for (int j = 0; j < 8; ++j) mma(acc[j], f[0], f[1], f[2], f[3], b[kt][j][0], b[kt][j][1]);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                int64_t at;
                int left;
                if (!(rows >> ((i >> 1) * 8 + g) & 1) || !has(m, i, &at, &left)) continue;
                const float scale = row_scale[m * 16 + (i >> 1) * 8 + g];
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = acc[j][i] * scale;
                now[i].add(v);
                now[i].store(out + at, left);
            }
            if constexpr (AHEAD > 0) {
                ask_w(w_at);
                w_at = w_at + 1 == AHEAD ? 0 : w_at + 1;
            }
        }
        ask(m + RING, slot);
        slot = slot + 1 == RING ? 0 : slot + 1;
    }
    queue_wait<0>();
    expand_end(k);
}

// Rows of the tile without an adapter: base as it is.
template <typename T, int NROWS>
__device__ __forceinline__ void copy_rows(const ExpandK &k, int rank, const int *ids, int64_t l0, int64_t lrows,
                                          int64_t c0) {
    const T *base = (const T *)k.base[rank];
    T *out = (T *)k.out[rank];
    const int64_t c = c0 + threadIdx.x;  // width: kThreads
    if (base == out || c >= k.bcols) return;
    T v[NROWS];
#pragma unroll
    for (int i = 0; i < NROWS; ++i) {
        const int64_t at = (l0 + i) * k.bcols + c;
        if (ids[i] < 0 && l0 + i < lrows && in_bounds(k.status, at, 1, k.brows * k.bcols))
            v[i] = base ? base[at] : T(0.0f);
    }
#pragma unroll
    for (int i = 0; i < NROWS; ++i) {
        const int64_t at = (l0 + i) * k.bcols + c;
        if (ids[i] < 0 && l0 + i < lrows && in_bounds(k.status, at, 1, k.brows * k.bcols)) out[at] = v[i];
    }
}

// Any types, on CUDA cores: 16 rows x 256 columns, a column per thread.
template <typename TW, typename TO>
__global__ void __launch_bounds__(kThreads) expand_simt_kernel(const __grid_constant__ ExpandK k) {
    pdl_release();
    constexpr int ROWS = 16, RMAX = 64;
    __shared__ int ids[ROWS], list[ROWS], count;
    __shared__ __align__(16) float ss[RMAX][ROWS];
    const int rank = blockIdx.x / k.row_tiles;
    const int64_t l0 = (int64_t)(blockIdx.x % k.row_tiles) * ROWS;
    const int64_t t0 = k.row0[rank] * k.brows + l0, t1 = (k.row0[rank] + 1) * k.brows;
    const int nd = distinct<ROWS>(k.ids, t0, t1 < k.rows ? t1 : k.rows, k.n, ids, list, &count, k.status);
    expand_low(k);
    if (blockIdx.z == 0) copy_rows<TO, ROWS>(k, rank, ids, l0, k.brows, (int64_t)blockIdx.y * 256);
    for (int i = threadIdx.x; i < ROWS * k.R; i += kThreads) {
        const int row = i / k.R, r = i % k.R;
        const int64_t at = (t0 + row) * k.R + r;
        ss[r][row] = ids[row] >= 0 && in_bounds(k.status, at, 1, k.rows * k.R) ? k.s[at] : 0.0f;
    }
    __syncthreads();
    const int64_t c = (int64_t)blockIdx.y * 256 + threadIdx.x;
    if (c >= k.bcols) {
        expand_end(k);
        return;
    }
    const TO *base = (const TO *)k.base[rank];
    TO *out = (TO *)k.out[rank];
    for (int d = blockIdx.z; d < nd; d += gridDim.z) {
        const int a = list[d];
        const int64_t w_at = (int64_t)a * k.R * k.cols + k.col0[rank] * k.bcols + c;
        const TW *w = (const TW *)k.w + w_at;
        float acc[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) acc[i] = 0.0f;
        for (int r0 = 0; r0 < k.R; r0 += 8) {
            float v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                v[r] = r0 + r < k.R && in_bounds(k.status, w_at + (r0 + r) * k.cols, 1, (int64_t)k.n * k.R * k.cols)
                           ? as_float(w[(r0 + r) * k.cols])
                           : 0.0f;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                if (r0 + r >= k.R) break;
#pragma unroll
                for (int i = 0; i < ROWS; i += 4) fma4(acc + i, &ss[r0 + r][i], v[r]);
            }
        }
        const float scale = k.scale ? k.scale[a] : 1.0f;
        float old[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int64_t at = (l0 + i) * k.bcols + c;
            old[i] = base && ids[i] == a && in_bounds(k.status, at, 1, k.brows * k.bcols) ? as_float(base[at]) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int64_t at = (l0 + i) * k.bcols + c;
            if (ids[i] == a && in_bounds(k.status, at, 1, k.brows * k.bcols)) out[at] = TO(old[i] + acc[i] * scale);
        }
    }
    expand_end(k);
}

// ---- outer -----------------------------------------------------------------

// Rows of an adapter.  A CTA marks them in a bit mask over a window of
// kWindow rows (one read of the row adapters), with how many lie before each
// 32-row word, then turns the marks into lists of up to kList rows, ascending.
constexpr int kWindow = 16384, kList = 1024;
// CTAs of one adapter and column tile.  One adapter, rank 16, with at most 16
// and 32 of them: 36.9 and 38.4 us for 8192 rows of 512 + 512 columns, 71.6 and
// 62.7 for 32768 of 256 + 256 (the whole gradient).
constexpr int kMostShares = 16;
struct Marks {
    uint32_t bits[kWindow / 32];
    int before[kWindow / 32];
    int warp_sum[16];
};

// Marks the window's rows with adapter a; returns how many.  A lane reads four
// rows, eight lanes make a word, a warp 128 rows at a time; all of a warp's
// rows of a window of 8 * 128 WARPS are asked for before any is looked at.
template <int WARPS>
__device__ __forceinline__ int mark_rows(const int *ids, int64_t w0, int64_t rows, int a, Marks &marks, int *status) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int n = (int)(rows - w0 < kWindow ? rows - w0 : kWindow), words = (n + 31) / 32;
    const int per = (words + 4 * WARPS - 1) / (4 * WARPS), first = warp * per;  // in units of 128 rows
    const bool whole = (reinterpret_cast<uintptr_t>(ids + w0) & 15) == 0;
    int mine = 0;
    for (int u0 = 0; u0 < per; u0 += 8) {
        int4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int t = (first + u0 + u) * 128 + lane * 4;
            v[u] = make_int4(-1, -1, -1, -1);
            if (u0 + u >= per || t >= n || !in_bounds(status, w0 + t, n - t < 4 ? n - t : 4, rows)) continue;
            if (whole && t + 4 <= n) {
                v[u] = *reinterpret_cast<const int4 *>(ids + w0 + t);
            } else {
                v[u].x = ids[w0 + t];
                if (t + 1 < n) v[u].y = ids[w0 + t + 1];
                if (t + 2 < n) v[u].z = ids[w0 + t + 2];
                if (t + 3 < n) v[u].w = ids[w0 + t + 3];
            }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (u0 + u >= per) break;
            uint32_t m = (uint32_t)((v[u].x == a) | (v[u].y == a) << 1 | (v[u].z == a) << 2 | (v[u].w == a) << 3)
                         << (lane & 7) * 4;
#pragma unroll
            for (int o = 1; o < 8; o *= 2) m |= __shfl_xor_sync(0xffffffffu, m, o);
            const int c0 = __popc(__shfl_sync(0xffffffffu, m, 0)), c1 = __popc(__shfl_sync(0xffffffffu, m, 8)),
                      c2 = __popc(__shfl_sync(0xffffffffu, m, 16)), c3 = __popc(__shfl_sync(0xffffffffu, m, 24));
            const int word = (first + u0 + u) * 4 + lane / 8;
            if ((lane & 7) == 0 && word < words) {
                marks.bits[word] = m;
                marks.before[word] = mine + (lane > 0 ? c0 : 0) + (lane > 8 ? c1 : 0) + (lane > 16 ? c2 : 0);
            }
            mine += c0 + c1 + c2 + c3;
        }
    }
    if (lane == 0) marks.warp_sum[warp] = mine;
    __syncthreads();
    int total = 0, before = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        if (i < warp) before += marks.warp_sum[i];
        total += marks.warp_sum[i];
    }
    for (int i = first * 4 + lane; i < (first + per) * 4 && i < words; i += 32) marks.before[i] += before;
    __syncthreads();
    return total;
}

// The marked rows number [from, to) of the window, at most kList, into list.
template <int WARPS>
__device__ __forceinline__ void list_rows(const Marks &marks, int64_t w0, int64_t rows, int from, int to, int *list) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int words = (int)((rows - w0 < kWindow ? rows - w0 : kWindow) + 31) / 32;
    __syncthreads();  // list is free
#pragma unroll 4
    for (int i = warp; i < words; i += WARPS) {
        const uint32_t m = marks.bits[i];
        const int place = marks.before[i] + __popc(m & ((1u << lane) - 1));
        if ((m >> lane & 1) && place >= from && place < to) list[place - from] = (int)(w0 + i * 32 + lane);
    }
    __syncthreads();
}

// Sorts the rows by adapter for the kernels that sum over an adapter's rows,
// and lays their low-rank values down in that order as those kernels' operand:
// three bf16 parts of RP values each (zeros past R), per row.  A CTA takes one
// adapter, and CTAs along y share its rows; every CTA counts for itself, from
// the ids alone, so that they need nothing of one another.  Latency: 6 us by
// itself for 4096 rows, 10 for 8192 at rank 32, all but 3 to 4 of it beside the
// projection.
template <int RP>
__global__ void __launch_bounds__(512) arrange_kernel(const __grid_constant__ ArrangeK k) {
    __shared__ Marks marks;
    __shared__ int list[kList], sum[16], valid_sum[16];
    const int a = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    // rows of the adapters below this one, where its own begin, and of all
    int below = 0, valid = 0;
    const int64_t n4 = (reinterpret_cast<uintptr_t>(k.ids) & 15) ? 0 : k.rows / 4;
    auto count = [&](int id) {
        below += (unsigned)id < (unsigned)a;
        valid += (unsigned)id < (unsigned)k.n;
    };
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < n4; i += 512) {
        const int4 v = in_bounds(k.status, i * 4, 4, k.rows) ? reinterpret_cast<const int4 *>(k.ids)[i] : make_int4(-1, -1, -1, -1);
        count(v.x);
        count(v.y);
        count(v.z);
        count(v.w);
    }
    for (int64_t i = n4 * 4 + threadIdx.x; i < k.rows; i += 512)
        if (in_bounds(k.status, i, 1, k.rows)) count(k.ids[i]);
    below = __reduce_add_sync(0xffffffffu, below);
    valid = __reduce_add_sync(0xffffffffu, valid);
    if (lane == 0) {
        sum[warp] = below;
        valid_sum[warp] = valid;
    }
    __syncthreads();
    below = valid = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        below += sum[i];
        valid += valid_sum[i];
    }
    if (a == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < k.sh.tiles * k.sh.most; i += 512) k.sh.arrived[i] = 0;
    int at = below;  // place of the window's first row
    for (int64_t w0 = 0; w0 < k.rows; w0 += kWindow) {
        const int total = mark_rows<16>(k.ids, w0, k.rows, a, marks, k.status);
        const int lo = (int)((int64_t)total * blockIdx.y / gridDim.y), hi = (int)((int64_t)total * (blockIdx.y + 1) / gridDim.y);
        // The ids and the forward call's values are from before the kernel that
        // this one follows (which has itself waited for what was before it);
        // the gradient of the low values is that kernel's.
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (j == 1) pdl_wait();
            for (int l0 = lo; l0 < hi; l0 += kList) {
                const int have = hi - l0 < kList ? hi - l0 : kList;
                if (j == 0 || hi - lo > kList) list_rows<16>(marks, w0, k.rows, l0, l0 + have, list);
                if (j == 0)
                    for (int i = threadIdx.x; i < have; i += 512)
                        if (in_bounds(k.status, at + l0 + i, 1, k.rows)) k.order[at + l0 + i] = list[i];
                if (!k.s[j]) continue;
#pragma unroll 2
                for (int e = threadIdx.x; e < have * (RP / 2); e += 512) {
                    const int i = e / (RP / 2), r = e % (RP / 2) * 2;
                    const int64_t from = (int64_t)list[i] * k.R;
                    if (!in_bounds(k.status, from, k.R, k.rows * k.R)) continue;
                    const float *v = k.s[j] + from;
                    uint32_t p[3];
                    split<3>(r < k.R ? v[r] : 0.0f, r + 1 < k.R ? v[r + 1] : 0.0f, p);
                    const int64_t to = ((int64_t)at + l0 + i) * (3 * RP) + r;
                    if (!in_bounds(k.status, to, 2 * RP + 2, k.rows * 3 * RP)) continue;  // the three parts' places
#pragma unroll
                    for (int h = 0; h < 3; ++h) *reinterpret_cast<uint32_t *>(k.parts[j] + to + h * RP) = p[h];
                }
            }
        }
        at += total;
    }
    pdl_release();
    if (threadIdx.x == 0 && blockIdx.y == 0) {
        k.start[a] = below;
        if (a == k.n - 1) k.start[k.n] = at;
        // A CTA's part of all the work, and how many of them this adapter is.
        // Which places it gets depends on who asks first; the sums do not.
        int first = 0, want = 1;
        if (k.sh.most) {
            const int64_t groups = (at - below + k.sh.group - 1) / k.sh.group, all = (valid + k.sh.group - 1) / k.sh.group;
            int64_t each = (all * k.sh.tiles + k.sh.room - 1) / k.sh.room;
            if (each < k.sh.least) each = k.sh.least;
            const int64_t w = groups / each;  // whole parts only: all CTAs still fit the card at once
            want = (int)(w < 1 ? 1 : w > kMostShares ? kMostShares : w);
            if (want > 1) {
                first = atomicAdd(k.sh.taken, want);
                const bool fits = first + want <= k.sh.most;  // always (see Grain)
                for (int i = 0; i < want && first + i < k.sh.most; ++i) k.sh.at[first + i] = make_int2(fits ? a : -1, i);
                if (!fits) want = 1;
            }
        }
        k.sh.of[a] = make_int2(first, want);
    }
}

// What the CTAs of a factor gradient's kernel do at the start: which adapter
// and share blockIdx.y is (false: none) ...
__device__ __forceinline__ bool take_share(const OuterK &k, int *a, int *share, int2 *of) {
    *a = blockIdx.y;
    *share = 0;
    if (*a >= k.n) {
        const int place = *a - k.n;
        if (place >= *k.sh.taken) return false;
        const int2 at = k.sh.at[place];
        if (at.x < 0 || at.y == 0) return false;
        *a = at.x;
        *share = at.y;
    }
    *of = k.sh.of[*a];
    return true;
}
// ... and at the end, with their own sums of `values` floats in memory: true
// for the last of an adapter's CTAs, which then adds all of them in order.
__device__ __forceinline__ bool last_share(const OuterK &k, int tile, int2 of, int *flag) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) *flag = atomicAdd(&k.sh.arrived[tile * k.sh.most + of.x], 1) == of.y - 1;
    __syncthreads();
    __threadfence();
    return *flag;
}

// A CTA takes one adapter, or a share of its rows, and 128 columns.
// Rows go in groups of 64, on tcgen05.  Both operands are MN-major, as their
// rows lie in memory: X's, gathered by index, 64 x 128; and the arranged low
// values', whose three parts stand beside one another, 64 x 3 RP, so that one
// product of 128 rows does all parts (RP = 64: a second one the third) and the
// parts' rows are added at the end.  The factor side, 3 RP columns, would be
// the bound of warp matrix instructions at RP = 32 and above (about half their
// rate), and its operands of their shared-memory reads.
// 80 us for 8192 rows of 20480 columns at rank 32 (336 MB, 4.2 TB/s), 24 us for
// 4096 of 8192 at rank 16.  What bounds it is a group's own chain, some 2400
// cycles in each of two CTAs: waiting for its copies, its products, asking for
// the next (800 of them: ten copies a thread, whose addresses spill: 84 bytes a
// thread, 148 to 188 in the element form), reading sums.  Not HBM (rows brought into the L2 six groups early:
// 84 us), not the L2 (22 % busy), issue slots (33 %) or the CTA's barrier (only
// the issuing warp waiting for the others: 85).  Other copies were slower: the
// low values split and the rows listed in every column tile (256 columns, one
// CTA per SM), 124 us; TMA gathers of four rows, 131 (65 cycles each).
constexpr int kOuterThreads = 256, kOuterCols = 128;  // two CTAs per SM
template <int RP>
struct OuterShape {
    static constexpr int kWidth = 3 * RP;                    // parts of a row
    static constexpr int kBoxes = (kWidth + 63) / 64;        // 64 x 64 boxes of them
    static constexpr int kRows = RP == 64 ? 128 : kWidth;    // TMEM lanes that hold something
    static constexpr int kBands = kRows / RP;
    static constexpr uint32_t kX = kBoxes * 8192;            // X's place in a stage, behind them
    static constexpr uint32_t kStage = kX + 16384;
    static constexpr int kStages = RP == 16 ? 4 : RP == 32 ? 3 : 2;
    static constexpr uint32_t kRing = kStages * kStage;
    static constexpr uint32_t kZeros = RP == 64 ? 8192 : 0;  // the lower half of the third part's product
    static constexpr int kPitch = 132;                       // fp32
    static constexpr size_t kResult = (size_t)kRows * kPitch * 4;
    static constexpr size_t kSmem = (kResult > kRing + kZeros ? kResult : kRing + kZeros) + 1024;
};
constexpr int kOuterSegment = 4;  // groups summed in the tensor memory before registers take them (see kTcSegment)
constexpr int kOuterList = 1024;  // row addresses at hand: 16 groups, half of them ahead

template <int RP, bool VEC>
__global__ void __launch_bounds__(kOuterThreads, 2) outer_tc_kernel(const __grid_constant__ OuterK k) {
    pdl_wait();
    using Shape = OuterShape<RP>;
    constexpr int S = Shape::kStages;
    constexpr int AHEAD = S - 1;  // groups asked for early
    __shared__ int abort_flag, last;
    __shared__ const bf16 *row_at[kOuterList];  // rows' first values of this tile's block, by place in the share
    __shared__ uint32_t tmem_at;
    __shared__ __align__(8) uint64_t bars[S];  // a stage's products are done
    extern __shared__ uint8_t raw_smem[];
    uint8_t *smem = raw_smem + (1024 - (shmm_dev::smem_u32(raw_smem) & 1023)) % 1024;
    const uint32_t smem_at = shmm_dev::smem_u32(smem);
    int a, cr;  // share cr of the adapter's
    int2 of;
    if (!take_share(k, &a, &cr, &of)) return;
    const int cs = of.y;
    const int which = (int)blockIdx.x >= k.job[0].tiles;
    const OuterJob &J = k.job[which];
    const int tile = blockIdx.x - (which ? k.job[0].tiles : 0);
    const int bcols = (int)J.x.bcols, per_block = (bcols + kOuterCols - 1) / kOuterCols, blk = tile / per_block;
    const int c0 = (tile - blk * per_block) * kOuterCols;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) shmm_dev::mbar_init(shmm_dev::smem_u32(&bars[i]), 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) shmm_tc::tmem_alloc(shmm_dev::smem_u32(&tmem_at), 2 * kOuterCols);
    if constexpr (Shape::kZeros > 0)
        for (int i = threadIdx.x; i < (int)Shape::kZeros / 16; i += kOuterThreads)
            *reinterpret_cast<uint4 *>(smem + Shape::kRing + i * 16) = make_uint4(0, 0, 0, 0);
    // This CTA's share of the adapter's rows, in whole groups of 64.
    const int first = k.start[a], total = k.start[a + 1] - first, groups = (total + 63) / 64;
    const int lo = (int)((int64_t)groups * cr / cs) * 64, end = (int)((int64_t)groups * (cr + 1) / cs) * 64;
    const int have = (end < total ? end : total) - lo, ngroups = (have + 63) / 64;
    const int *order = k.order + first + lo;
    const bf16 *parts = J.parts + (int64_t)(first + lo) * Shape::kWidth;
    auto find_rows = [&](int i0) {  // the addresses of 512 rows from i0 on
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = i0 + u * kOuterThreads + threadIdx.x;
            if (i >= have) continue;
            const uint32_t t = in_bounds(k.status, first + lo + i, 1, k.rows) ? order[i] : 0, b = t / (uint32_t)J.x.brows;
            const int64_t off = (int64_t)(t - b * (uint32_t)J.x.brows) * bcols;
            row_at[i % kOuterList] = in_bounds(k.status, off, bcols, J.x.brows * J.x.bcols)
                                         ? (const bf16 *)J.x.at[b * J.x.b1 + blk] + off
                                         : (const bf16 *)nullptr;
        }
    };
    find_rows(0);
    shmm_tc::fence_before();
    __syncthreads();
    shmm_tc::fence_after();
    pdl_release();  // after the TMEM is held (see project_tc_kernel)
    const uint32_t tmem = tmem_at;
    // This thread's pieces of a group: of X, eight columns of the rows xr + 16 i;
    // of the parts, every fourth eight of row pr.
    const int xr = threadIdx.x / 16, cx = c0 + (threadIdx.x & 15) * 8;
    const uint32_t x_to = Shape::kX + (threadIdx.x & 15) / 8 * 8192 + xr * 128 + (((threadIdx.x & 7) ^ (xr & 7)) * 16);
    const int pr = threadIdx.x / 4, pc = threadIdx.x & 3;
    bool ok = true;
    // The sums so far: TMEM lane 32 (warp % 4) + lane, columns 64 (warp / 4)..
    const int quad = warp & 3, part = warp >> 2;
    float acc[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) acc[i] = 0.0f;
    // Adds segment q (group `last` its last) from its buffer.
    auto drain = [&](uint32_t q, uint32_t last) {
        ok = shmm_dev::mbar_wait(shmm_dev::smem_u32(&bars[last % S]), (last / S) & 1, &abort_flag, k.status) && ok;
        __syncwarp();
        shmm_tc::fence_after();
        if (quad * 32 >= Shape::kRows) return;
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
            float v[16];
            shmm_tc::tmem_read16(tmem + ((uint32_t)(quad * 32) << 16) + (q & 1) * kOuterCols + part * 64 + c, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[c + j] += v[j];
        }
        shmm_tc::fence_before();  // the barrier before the next product into this buffer follows
    };
    // Asks for group f, once the products of the stage's last one are done.
    auto ask = [&](uint32_t f) {
        const uint32_t s = f % S;
        if (f >= S) ok = shmm_dev::mbar_wait(shmm_dev::smem_u32(&bars[s]), (f / S - 1) & 1, &abort_flag, k.status) && ok;
        const uint32_t at0 = s * Shape::kStage;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = f * 64 + i * 16 + xr;
            const bf16 *row = at < have && cx < bcols ? row_at[at % kOuterList] : (const bf16 *)nullptr;
            if constexpr (VEC) {
                queue16(smem_at + x_to + at0 + i * 2048, row ? (const void *)(row + cx) : parts, row != nullptr);
            } else {
                const Raw8 v = row ? load8<false>(row, cx, bcols) : Raw8{{0, 0, 0, 0}};
                *reinterpret_cast<uint4 *>(smem + x_to + at0 + i * 2048) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
            }
        }
        const bool real = (int)f * 64 + pr < have &&
                          in_bounds(k.status, (int64_t)(first + lo + (int)f * 64 + pr) * Shape::kWidth, Shape::kWidth,
                                    k.rows * Shape::kWidth);
        const bf16 *from = parts + (int64_t)(real ? f * 64 + pr : 0) * Shape::kWidth + pc * 8;
#pragma unroll
        for (int i = 0; i < (Shape::kWidth + 31) / 32; ++i) {
            const int c = pc + 4 * i;
            if (c < Shape::kWidth / 8)
                queue16(smem_at + at0 + (c / 8) * 8192 + pr * 128 + (((c & 7) ^ (pr & 7)) * 16), from + i * 32, real);
        }
        queue_commit();
    };
#pragma unroll 1
    for (int f = 0; f < AHEAD; ++f) {
        if (f < ngroups) ask(f);
        else queue_commit();
    }
    for (int f = 0; f < ngroups; ++f) {
        queue_wait<AHEAD - 1>();
        shmm_tc::fence_async();
        shmm_tc::fence_before();
        __syncthreads();
        const uint32_t q = f / kOuterSegment;
        if (threadIdx.x == 0) {
            shmm_tc::fence_after();
            const uint32_t at = smem_at + (f % S) * Shape::kStage, zeros = smem_at + Shape::kRing;  // RP = 64
            constexpr uint32_t idesc = shmm_tc::instruction(kOuterCols, true, true);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint64_t x = shmm_tc::operand(at + Shape::kX + kk * 2048, 8192, 1024);
                // RP = 16 has one box: X's first one fills the 64 rows that nobody reads
                shmm_tc::mma_issue(tmem + (q & 1) * kOuterCols, shmm_tc::operand(at + kk * 2048, 8192, 1024), x, idesc,
                                   f % kOuterSegment > 0 || kk > 0);
                if constexpr (RP == 64)
                    shmm_tc::mma_issue(tmem + (q & 1) * kOuterCols,
                                       shmm_tc::operand(at + 16384 + kk * 2048, zeros - at - 16384 - kk * 2048, 1024), x,
                                       idesc, true);
            }
            shmm_tc::mma_commit(shmm_dev::smem_u32(&bars[f % S]));
        }
        if (f % 8 == 0) find_rows((f + 8) * 64);  // asked for after the next barrier at the earliest
        if (f + AHEAD < ngroups) ask(f + AHEAD);
        else queue_commit();
        // The segment before this one, while its successor's first products
        // run (they go into the other buffer).
        if (f % kOuterSegment == 0 && f > 0) drain(q - 1, f - 1);
    }
    if (ngroups > 0) drain((ngroups - 1) / kOuterSegment, ngroups - 1);
    // Every product is done before its operands' memory is used again.
    for (int f = ngroups > S ? ngroups - S : 0; f < ngroups; ++f)
        shmm_dev::mbar_wait(shmm_dev::smem_u32(&bars[f % S]), (f / S) & 1, &abort_flag, k.status, false);
    __syncthreads();
    // Result through shared memory, the parts' rows added there; then the
    // shares' sums.
    const float scale = J.scale && total > 0 ? J.scale[a] : 1.0f;  // no rows: zeros whatever it is
    float *out = J.out + (int64_t)a * k.R * J.cols + (int64_t)blk * bcols + c0;
    const bool whole = (J.cols & 3) == 0 && (bcols & 3) == 0 && (reinterpret_cast<uintptr_t>(J.out) & 15) == 0;
    auto put = [&](int r, int c, float4 v) {  // four columns from c of row r
        const int left = bcols - c0 - c;
        if (left <= 0 || !in_bounds(k.status, ((int64_t)a * k.R + r) * J.cols + (int64_t)blk * bcols + c0 + c,
                                    left < 4 ? left : 4, (int64_t)k.n * k.R * J.cols))
            return;
        float *o = out + (int64_t)r * J.cols + c;
        v = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
        if (whole) {
            *reinterpret_cast<float4 *>(o) = v;
        } else {
            o[0] = v.x;
            if (left > 1) o[1] = v.y;
            if (left > 2) o[2] = v.z;
            if (left > 3) o[3] = v.w;
        }
    };
    float *piece = reinterpret_cast<float *>(smem);                // [kRows][kPitch]
    float *sums = k.sh.sums + ((int64_t)blockIdx.x * k.sh.most + of.x) * (RP * kOuterCols);  // the first share's
    auto add = [](float4 &t, const float4 &v) {
        t.x += v.x;
        t.y += v.y;
        t.z += v.z;
        t.w += v.w;
    };
    const int my_row = quad * 32 + lane;
    if (my_row < Shape::kRows)
#pragma unroll
        for (int j = 0; j < 64; j += 4)
            *reinterpret_cast<float4 *>(piece + my_row * Shape::kPitch + part * 64 + j) =
                make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
    __syncthreads();
    for (int e = threadIdx.x; e < k.R * 32; e += kOuterThreads) {
        const int r = e / 32, j = e % 32 * 4;
        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int h = Shape::kBands - 1; h >= 0; --h)
            add(t, *reinterpret_cast<const float4 *>(piece + (h * RP + r) * Shape::kPitch + j));
        if (cs == 1) put(r, j, t);
        else if (in_bounds(k.status, (sums - k.sh.sums) + (int64_t)cr * RP * kOuterCols + r * kOuterCols + j, 4,
                           (int64_t)k.sh.tiles * k.sh.most * RP * kOuterCols))
            __stcg(reinterpret_cast<float4 *>(sums + (int64_t)cr * RP * kOuterCols + r * kOuterCols + j), t);
    }
    if (cs > 1 && last_share(k, blockIdx.x, of, &last))
        for (int e = threadIdx.x; e < k.R * 32; e += kOuterThreads) {
            float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int b = 0; b < cs; ++b)
                add(t, __ldcg(reinterpret_cast<const float4 *>(sums + (int64_t)b * RP * kOuterCols + e * 4)));
            put(e / 32, e % 32 * 4, t);
        }
    shmm_tc::fence_before();
    __syncthreads();
    shmm_tc::fence_after();
    if (warp == 0) shmm_tc::tmem_free(tmem, 2 * kOuterCols);
}

// Any types, on CUDA cores: one adapter, 128 columns and 16 adapter rows per
// CTA, or a share of the adapter's rows; the halves of a CTA take every other
// group of 16 of them.
template <typename TX>
__global__ void __launch_bounds__(kThreads) outer_simt_kernel(const __grid_constant__ OuterK k) {
    pdl_enter();
    __shared__ __align__(16) float ss[2][16][16];
    __shared__ float sums[16 * 128];
    __shared__ int last;
    int a, cr;  // share cr of the adapter's
    int2 of;
    if (!take_share(k, &a, &cr, &of)) return;
    const int cs = of.y;
    const int which = (int)blockIdx.x >= k.job[0].tiles;
    const OuterJob &J = k.job[which];
    const int tile = blockIdx.x - (which ? k.job[0].tiles : 0), r0 = blockIdx.z * 16;
    const int half = threadIdx.x / 128, th = threadIdx.x % 128;
    const int bcols = (int)J.x.bcols, per_block = (bcols + 127) / 128, blk = tile / per_block;
    const int c0 = (tile - blk * per_block) * 128, c = c0 + th;
    const int first = k.start[a], total = k.start[a + 1] - first, groups = (total + 31) / 32;
    const int lo = (int)((int64_t)groups * cr / cs) * 32, end = (int)((int64_t)groups * (cr + 1) / cs) * 32;
    const int have = (end < total ? end : total) - lo;
    const int *order = k.order + first + lo;
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    for (int64_t s0 = 0; s0 < have; s0 += 32) {
        const int64_t s = s0 + half * 16;
        float x[16], v[2];
#pragma unroll
        for (int u = 0; u < 16; ++u) {
            x[u] = 0.0f;
            if (s + u < have && c < bcols && in_bounds(k.status, first + lo + s + u, 1, k.rows)) {
                const uint32_t t = order[s + u], b = t / (uint32_t)J.x.brows;
                const int64_t at = (int64_t)(t - b * (uint32_t)J.x.brows) * bcols + c;
                if (in_bounds(k.status, at, 1, J.x.brows * bcols))
                    x[u] = as_float(((const TX *)J.x.at[b * J.x.b1 + blk])[at]);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int u = th / 16 + i * 8, r = r0 + th % 16;
            v[i] = 0.0f;
            if (s + u < have && r < k.R && in_bounds(k.status, first + lo + s + u, 1, k.rows)) {
                const int64_t at = (int64_t)order[s + u] * k.R + r;
                if (in_bounds(k.status, at, 1, k.rows * k.R)) v[i] = J.s[at];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) ss[half][th / 16 + i * 8][th % 16] = v[i];
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 16; ++u)
#pragma unroll
            for (int i = 0; i < 16; i += 4) fma4(acc + i, &ss[half][u][i], x[u]);
    }
    if (half)
#pragma unroll
        for (int i = 0; i < 16; ++i) sums[i * 128 + th] = acc[i];
    __syncthreads();
    if (!half)
#pragma unroll
        for (int i = 0; i < 16; ++i) sums[i * 128 + th] += acc[i];
    __syncthreads();
    const float scale = J.scale && total > 0 ? J.scale[a] : 1.0f;  // no rows: zeros whatever it is
    const int piece = blockIdx.z * gridDim.x + blockIdx.x;  // a tile's 16 adapter rows
    float *shared_sums = k.sh.sums + ((int64_t)piece * k.sh.most + of.x) * (16 * 128);
    if (cs > 1) {
        for (int e = threadIdx.x; e < 16 * 128; e += kThreads)
            if (in_bounds(k.status, (shared_sums - k.sh.sums) + cr * (16 * 128) + e, 1,
                          (int64_t)k.sh.tiles * k.sh.most * (16 * 128)))
                __stcg(shared_sums + cr * (16 * 128) + e, sums[e]);
        if (!last_share(k, piece, of, &last)) return;
    }
    for (int e = threadIdx.x; e < 16 * 128; e += kThreads) {
        float v = cs > 1 ? 0.0f : sums[e];
        if (cs > 1)
#pragma unroll 4
            for (int b = 0; b < cs; ++b) v += __ldcg(shared_sums + b * (16 * 128) + e);
        const int r = r0 + e / 128, col = c0 + e % 128;
        const int64_t at = ((int64_t)a * k.R + r) * J.cols + (int64_t)blk * bcols + col;
        if (r < k.R && col < bcols && in_bounds(k.status, at, 1, (int64_t)k.n * k.R * J.cols)) J.out[at] = v * scale;
    }
}

// ---- launches --------------------------------------------------------------

int sms() {
    static shmm::PerDevice<int> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= shmm::kMaxDevices) return 152;
    int n = cache.get(dev);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
        cache.set(dev, n);
    }
    return n;
}

// Lets `kern` take `bytes` of dynamic shared memory on the current device.
template <typename K>
cudaError_t opt_in(K kern, size_t bytes, shmm::PerDevice<int> *done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= shmm::kMaxDevices) return cudaErrorInvalidDevice;
    if (done->get(dev)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done->set(dev, 1);
    return e;
}

void fill(Blocks *b, const shmm::BlockGrid &g) {
    for (int i = 0; i < g.b0 * g.b1; ++i) b->at[i] = g.at[i];
    b->b1 = g.b1;
    b->brows = g.brows;
    b->bcols = g.bcols;
}

// CTAs of kThreads threads and `smem` bytes of shared memory that the card
// holds at once.
int64_t slots_for(size_t smem) {
    const int64_t per = (227 * 1024) / (int64_t)(smem + 3 * 1024);
    return sms() * (per < 1 ? 1 : per > 4 ? 4 : per);
}

// Spreads `tiles` CTAs of work over the card in one wave: a tile's adapters
// over z CTAs (at most `most`, as many as it has rows or the call adapters),
// then its columns over a cluster of c (at most `split`).  One wave of equal
// CTAs ends together; two leave the second part empty.
// `few`: a batch of single tokens, most rows with an adapter of their own, so
// the adapters come first (96 rows of 64 adapters at random, 8192 columns, rank
// 16: 14.2 us forward against 15.2 columns first; 256 rows 22.4 against 28.3).
// In longer ones a tile is meant to have one or two; where it has many all the
// same, columns first costs (512 rows of 64 adapters: 49.6 us against 35.9).
void spread(int64_t tiles, int64_t slots, int64_t most, int64_t split, bool few, int *c, int *z) {
    *c = *z = 1;
    auto adapters = [&] {
        const int64_t left = slots / (tiles * *c);
        *z = (int)(left < 1 ? 1 : left < most ? left : most);
    };
    if (few) adapters();
    while (*c < 8 && tiles * *z * *c * 2 <= slots && *c * 2 <= split) *c *= 2;
    if (!few) adapters();
}
constexpr int64_t kFewRows = 256;

template <int MT, int NT, bool VEC>
cudaError_t project_mma(const ProjK &k, cudaStream_t s) {
    using Shape = ProjShape<MT, NT>;
    auto kern = project_mma_kernel<MT, NT, VEC>;
    static shmm::PerDevice<int> done;
    cudaError_t e = opt_in(kern, Shape::kSmem, &done);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (k.rows + 16 * MT - 1) / (16 * MT);
    int c, z;
    // two chunks of 32 columns per warp at least
    spread(tiles, slots_for(Shape::kSmem), k.n < 16 * MT ? k.n : 16 * MT, k.cols / (64 * kWarps),
           k.rows < kFewRows, &c, &z);
    return launch_pdl_cluster(kern, dim3((unsigned)tiles, c, z), dim3(1, c, 1), dim3(kThreads), Shape::kSmem, s, k);
}

template <int NT, bool VEC>
cudaError_t project_rows(const ProjK &k, cudaStream_t s) {
    // Two row tiles per warp halve the factor's share of the loads; they
    // need rows enough to fill the card.
    return k.rows >= 16 * sms() ? project_mma<2, NT, VEC>(k, s) : project_mma<1, NT, VEC>(k, s);
}

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
    static std::once_flag once;
    static EncodeFn fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
    });
    return fn;
}

// A row-major rows x cols bf16 matrix in boxes of box_rows x 64.
bool make_map(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int box_rows) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)cols * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, one[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int RP>
cudaError_t project_tc(const ProjK &k, int b0, cudaStream_t s) {
    auto kern = project_tc_kernel<RP>;
    static shmm::PerDevice<int> done;
    cudaError_t e = opt_in(kern, kTcSmem, &done);
    if (e != cudaSuccess) return e;
    ProjTcK t;
    for (int i = 0; i < b0 * k.x.b1; ++i)
        if (!make_map(&t.x[i], k.x.at[i], k.x.brows, k.x.bcols, 128)) return cudaErrorNotSupported;
    if (!make_map(&t.w, k.w, (int64_t)k.n * k.R, k.cols, RP)) return cudaErrorNotSupported;
    t.ids = k.ids;
    t.scale = k.scale;
    t.out = k.out;
    t.clear = k.clear;
    t.n = k.n;
    t.R = k.R;
    t.b1 = k.x.b1;
    t.row_tiles = (int)((k.x.brows + 127) / 128);
    t.per_block = (int)((k.x.bcols + 63) / 64);
    t.chunks = t.per_block * k.x.b1;
    t.brows = k.x.brows;
    t.bcols = k.x.bcols;
    t.rows = k.rows;
    t.status = k.status;
    const int64_t tiles = (int64_t)t.row_tiles * b0;
    int c, z;
    spread(tiles, 2 * sms(), 1, t.chunks / 4, false, &c, &z);
    return launch_pdl_cluster(kern, dim3((unsigned)tiles, c), dim3(1, c, 1), dim3(kTcThreads), kTcSmem, s, t);
}

template <bool VEC>
cudaError_t project_vec(const ProjK &k, cudaStream_t s) {
    // tcgen05 from 2048 rows on: 16 row tiles, whose clusters of 8 reach most
    // SMs.  Forward, 4096 x 64, four adapters, tcgen05 and warp instructions:
    // rank 64 18.6 and 16.8 us at 1024 rows, 20.6 and 25.7 at 2048, 32.6 and
    // 64.3 at 8192; rank 16 15.6 and 12.2 at 2048, 16.7 and 15.3 at 4096, 20.9
    // and 24.7 at 8192: one border for all ranks, late for high, early for low.
    const int b0 = (int)(k.rows / k.x.brows);
    if (VEC && k.rows >= 2048 && k.x.brows >= 128 && b0 * k.x.b1 <= kMaxMaps && k.cols >= 512) {
        if (k.R <= 16) return project_tc<16>(k, b0, s);
        return k.R <= 32 ? project_tc<32>(k, b0, s) : project_tc<64>(k, b0, s);
    }
    if (k.R <= 8) return project_rows<1, VEC>(k, s);
    if (k.R <= 16) return project_rows<2, VEC>(k, s);
    if (k.R <= 32) return project_rows<4, VEC>(k, s);
    return project_rows<8, VEC>(k, s);
}

template <typename TX, typename TW>
cudaError_t project_simt(const ProjK &k, cudaStream_t s) {
    const int64_t tiles = (k.rows + 31) / 32;
    int cluster, z;
    spread(tiles, 4 * sms(), k.n < 32 ? k.n : 32, k.cols / 64, k.rows < kFewRows, &cluster, &z);
    const dim3 g((unsigned)tiles, cluster, z), c(1, cluster, 1);
    if (k.R <= 16) return launch_pdl_cluster(project_simt_kernel<TX, TW, 1>, g, c, dim3(kThreads), 0, s, k);
    if (k.R <= 32) return launch_pdl_cluster(project_simt_kernel<TX, TW, 2>, g, c, dim3(kThreads), 0, s, k);
    return launch_pdl_cluster(project_simt_kernel<TX, TW, 4>, g, c, dim3(kThreads), 0, s, k);
}

cudaError_t project(const ProjK &k, shmm_dtype_t xt, shmm_dtype_t wt, cudaStream_t s) {
    shmm::count_launch();
    if (xt == SHMM_BF16 && wt == SHMM_BF16)
        return k.cols % 8 == 0 && k.x.bcols % 8 == 0 ? project_vec<true>(k, s) : project_vec<false>(k, s);
    if (xt == SHMM_F32) return wt == SHMM_F32 ? project_simt<float, float>(k, s) : project_simt<float, bf16>(k, s);
    return project_simt<bf16, float>(k, s);
}

template <bool FEW, int KT, bool VEC, typename TO>
cudaError_t expand_mma(ExpandK k, int nranks, cudaStream_t s) {
    using Shape = ExpandShape<FEW, KT, TO>;
    auto kern = expand_mma_kernel<FEW, KT, VEC, TO>;
    static shmm::PerDevice<int> done;
    cudaError_t e = opt_in(kern, Shape::smem(FEW ? 1 : kMaxRowTiles), &done);
    if (e != cudaSuccess) return e;
    const int64_t cols = (k.bcols + 511) / 512;
    k.row_tiles = (int)((k.brows + 16 * k.mt - 1) / (16 * k.mt));
    int c, z = 1;
    if (FEW) spread((int64_t)k.row_tiles * nranks * cols, 2 * sms(), k.n < 16 ? k.n : 16, 1, true, &c, &z);
    return launch_pdl(kern, dim3((unsigned)(k.row_tiles * nranks), (unsigned)cols, z), dim3(kThreads),
                      Shape::smem(k.mt), s, k);
}

template <bool VEC, typename TO>
cudaError_t expand_vec(ExpandK k, int nranks, cudaStream_t s) {
    // A CTA of more row tiles reads a factor's piece and the low rows' split
    // less often (its start costs some 3 us), while the last wave of CTAs
    // leaves less of the card empty the more of them there are: 16 row tiles
    // where that makes six waves of two CTAs per SM, 8 for three, else 4, and
    // one below half a wave.  Forward, 64 x 4096, rank 16, at the borders: 58368
    // rows 190 us with 16 and 196 with 8; 14592 rows 50.8 with 8, 56.5 with 4 (56.4
    // with 16); 1216 rows 9.0 with 4, 9.7 with 1.
    auto waves = [&](int mt) {
        return (double)((k.brows + 16 * mt - 1) / (16 * mt) * nranks * ((k.bcols + 511) / 512)) / (2 * sms());
    };
    k.mt = waves(16) >= 6 ? 16 : waves(8) >= 3 ? 8 : waves(4) >= 0.5 ? 4 : 1;
    if (k.mt == 1) {
        if (k.R <= 16) return expand_mma<true, 1, VEC, TO>(k, nranks, s);
        return k.R <= 32 ? expand_mma<true, 2, VEC, TO>(k, nranks, s) : expand_mma<true, 4, VEC, TO>(k, nranks, s);
    }
    if (k.R <= 16) return expand_mma<false, 1, VEC, TO>(k, nranks, s);
    return k.R <= 32 ? expand_mma<false, 2, VEC, TO>(k, nranks, s) : expand_mma<false, 4, VEC, TO>(k, nranks, s);
}

template <typename TO>
cudaError_t expand_type(ExpandK k, int nranks, shmm_dtype_t wt, cudaStream_t s) {
    if (wt == SHMM_BF16)
        return k.cols % 8 == 0 && k.bcols % 8 == 0 ? expand_vec<true, TO>(k, nranks, s)
                                                   : expand_vec<false, TO>(k, nranks, s);
    k.row_tiles = (int)((k.brows + 15) / 16);
    const int64_t tiles = (int64_t)k.row_tiles * nranks * ((k.bcols + 255) / 256);
    int c, z;
    spread(tiles, 2 * sms(), k.n < 16 ? k.n : 16, 1, true, &c, &z);
    return launch_pdl(expand_simt_kernel<float, TO>,
                      dim3((unsigned)(k.row_tiles * nranks), (unsigned)((k.bcols + 255) / 256), z), dim3(kThreads),
                      0, s, k);
}

cudaError_t expand(const ExpandK &k, int nranks, shmm_dtype_t wt, shmm_dtype_t ot, cudaStream_t s) {
    shmm::count_launch();
    return ot == SHMM_F32 ? expand_type<float>(k, nranks, wt, s) : expand_type<bf16>(k, nranks, wt, s);
}

template <int RP, bool VEC>
cudaError_t outer_tc(const OuterK &k, cudaStream_t s) {
    using Shape = OuterShape<RP>;
    auto kern = outer_tc_kernel<RP, VEC>;
    static shmm::PerDevice<int> done;
    cudaError_t e = opt_in(kern, Shape::kSmem, &done);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)(k.job[0].tiles + k.job[1].tiles), (unsigned)(k.n + k.sh.most)),
                      dim3(kOuterThreads), Shape::kSmem, s, k);
}

int padded(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : 64; }  // adapter rows of a product

cudaError_t arrange(const ArrangeK &k, cudaStream_t s) {
    shmm::count_launch();
    // CTAs for a wave of two per SM, of 64 rows and more.
    int64_t y = 2 * sms() / k.n, most = k.rows / 64;
    if (y > most) y = most;
    const dim3 g((unsigned)k.n, (unsigned)(y > 1 ? y : 1));
    if (k.R <= 16) return launch_pdl(arrange_kernel<16>, g, dim3(512), 0, s, k);
    if (k.R <= 32) return launch_pdl(arrange_kernel<32>, g, dim3(512), 0, s, k);
    return launch_pdl(arrange_kernel<64>, g, dim3(512), 0, s, k);
}

// One or both gradient products (job[1].cols == 0: one) of one type.
cudaError_t outer(OuterK k, shmm_dtype_t xt, cudaStream_t s) {
    shmm::count_launch();
    if (xt == SHMM_F32)
        return launch_pdl(outer_simt_kernel<float>,
                          dim3((unsigned)(k.job[0].tiles + k.job[1].tiles), (unsigned)(k.n + k.sh.most), (k.R + 15) / 16),
                          dim3(kThreads), 0, s, k);
    bool vec = true;
    for (const OuterJob &j : k.job)
        if (j.cols) vec = vec && j.x.bcols % 8 == 0;
    if (k.R <= 16) return vec ? outer_tc<16, true>(k, s) : outer_tc<16, false>(k, s);
    if (k.R <= 32) return vec ? outer_tc<32, true>(k, s) : outer_tc<32, false>(k, s);
    return vec ? outer_tc<64, true>(k, s) : outer_tc<64, false>(k, s);
}

void fill_expand(ExpandK *k, const shmm::AdapterArgs &a, const shmm::RankBoxes &b) {
    for (int r = 0; r < b.nranks; ++r) {
        k->base[r] = b.base ? b.base[r] : nullptr;
        k->out[r] = b.out[r];
        k->row0[r] = b.row0[r];
        k->col0[r] = b.col0[r];
    }
    k->brows = b.brows;
    k->bcols = b.bcols;
    k->ids = a.ids;
    k->n = a.n;
    k->R = a.R;
    k->rows = a.rows;
}

}  // namespace

namespace shmm {

// Places for shares (see Shares).  An adapter with w >= 2 of them has w parts'
// worth of groups, the last one perhaps of a single row: at most twice as many
// as its rows fill.  So all places together are at most 2 (room / tiles) per
// column tile.  None when half the card's CTAs or more have a column tile of
// their own, or for few rows.
// The card's SMs are a constant here, not asked of the current device: the
// workspace's size follows from them, and it is the same wherever it is asked
// for.  (Nothing waits for all CTAs to be there at once.)
struct Grain {
    static constexpr int kSms = 152;
    int per_sm, group, least;  // CTAs per SM, rows of a group, groups of a CTA
    int64_t room() const { return (int64_t)per_sm * kSms; }
    bool shared(int64_t rows) const { return rows > (int64_t)group * least; }
    int most(int64_t rows, int64_t n, int64_t tiles) const {
        if (tiles * 2 > room() || !shared(rows)) return 0;
        const int64_t most = 2 * room() / tiles + 2;
        return n + most > 65535 ? 0 : (int)most;
    }
};
static Grain grain(bool tc) { return tc ? Grain{2, 64, 4} : Grain{4, 32, 1}; }

// Workspace of the backward call: the gradient of the low values, then the
// rows' arrangement and the shares'.
struct Rooms {
    size_t start, order, of, at, taken, arrived, sums, parts[2], all;
};
static Rooms rooms(int64_t rows, int n, int R, bool tc) {
    auto up = [](int64_t bytes) { return (size_t)((bytes + 255) / 256 * 256); };
    const Grain g = grain(tc);
    const int64_t room = g.room(), places = g.shared(rows) ? 3 * room : 0;  // over all tiles: most * tiles <= 3 room
    Rooms r;
    r.start = up(rows * R * 4);
    r.order = r.start + up(((int64_t)n + 1) * 4);
    r.of = r.order + up(rows * 4);
    r.at = r.of + up((int64_t)n * 8);
    r.taken = r.at + (places ? up((2 * room + 2) * 8) : 0);
    r.arrived = r.taken + 256;
    r.sums = r.arrived + up(places * 4);
    r.parts[0] = r.sums + up(places * (tc ? padded(R) : 16) * 128 * 4);
    r.parts[1] = r.parts[0] + (tc ? up(rows * 6 * padded(R)) : 0);
    r.all = rows ? r.parts[1] + (tc ? up(rows * 6 * padded(R)) : 0) : 0;
    return r;
}

size_t adapters_workspace_bytes(int64_t rows, int n, int R, bool tc) { return rooms(rows, n, R, tc).all; }

int launch_adapters_forward(const AdapterArgs &a, const BlockGrid &A, const RankBoxes &C, shmm_dtype_t in_dt,
                            shmm_dtype_t out_dt, int *status, void *stream) {
    if (a.rows == 0) return 0;
    cudaStream_t s = (cudaStream_t)stream;
    ProjK p = {};
    fill(&p.x, A);
    p.w = a.down;
    p.ids = a.ids;
    p.out = a.low;
    p.n = a.n;
    p.R = a.R;
    p.rows = a.rows;
    p.cols = a.J;
    p.status = status;
    cudaError_t e = project(p, in_dt, in_dt, s);
    if (e != cudaSuccess) return (int)e;
    ExpandK x = {};
    fill_expand(&x, a, C);
    x.w = a.up;
    x.scale = a.scale;
    x.s = a.low;
    x.cols = a.K;
    x.status = status;
    return (int)expand(x, C.nranks, in_dt, out_dt, s);
}

int launch_adapters_backward(const AdapterArgs &a, const BlockGrid &dC, const BlockGrid &A, const RankBoxes &dA,
                             shmm_dtype_t in_dt, shmm_dtype_t out_dt, int *status, void *stream) {
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (a.rows == 0) {  // nothing to read, and no workspace
        const size_t factor = (size_t)a.n * a.R * 4;
        e = cudaMemsetAsync(a.ddown, 0, factor * a.J, s);
        return (int)(e != cudaSuccess ? e : cudaMemsetAsync(a.dup, 0, factor * a.K, s));
    }
    ProjK p = {};
    fill(&p.x, dC);
    p.w = a.up;
    p.ids = a.ids;
    p.scale = a.scale;
    p.out = a.dlow;
    p.n = a.n;
    p.R = a.R;
    p.rows = a.rows;
    p.cols = a.K;
    p.status = status;
    const bool tc[2] = {out_dt == SHMM_BF16, in_dt == SHMM_BF16};  // dup, ddown
    const Rooms at = rooms(a.rows, a.n, a.R, tc[0] || tc[1]);
    char *ws = reinterpret_cast<char *>(a.dlow);
    p.clear = reinterpret_cast<int *>(ws + at.taken);
    if ((e = project(p, out_dt, in_dt, s)) != cudaSuccess) return (int)e;
    OuterK o = {};
    o.order = reinterpret_cast<int *>(ws + at.order);
    o.start = reinterpret_cast<int *>(ws + at.start);
    o.n = a.n;
    o.R = a.R;
    o.rows = a.rows;
    o.status = status;
    OuterJob up = {}, down = {};
    fill(&up.x, dC);
    up.s = a.low;
    up.parts = reinterpret_cast<bf16 *>(ws + at.parts[0]);
    up.scale = a.scale;
    up.out = a.dup;
    up.cols = a.K;
    fill(&down.x, A);
    down.s = a.dlow;
    down.parts = reinterpret_cast<bf16 *>(ws + at.parts[1]);
    down.out = a.ddown;
    down.cols = a.J;
    const bool one = in_dt == out_dt;  // one launch for both
    for (int j = 0; j < 2; ++j) {
        OuterJob &J = j ? down : up;
        J.tiles = (int)((J.x.bcols + kOuterCols - 1) / kOuterCols * J.x.b1);
    }
    Shares &sh = o.sh;
    sh.of = reinterpret_cast<int2 *>(ws + at.of);
    sh.at = reinterpret_cast<int2 *>(ws + at.at);
    sh.taken = reinterpret_cast<int *>(ws + at.taken);
    sh.arrived = reinterpret_cast<int *>(ws + at.arrived);
    sh.sums = reinterpret_cast<float *>(ws + at.sums);
    if (one) {
        const int64_t tiles = (int64_t)(up.tiles + down.tiles) * (tc[0] ? 1 : (a.R + 15) / 16);
        const Grain g = grain(tc[0]);
        sh.room = g.room();
        sh.group = g.group;
        sh.least = g.least;
        sh.most = g.most(a.rows, a.n, tiles);
        sh.tiles = (int)tiles;
    }
    ArrangeK g = {};
    g.sh = sh;
    g.ids = a.ids;
    g.order = reinterpret_cast<int *>(ws + at.order);
    g.start = reinterpret_cast<int *>(ws + at.start);
    g.s[0] = tc[0] ? a.low : nullptr;
    g.s[1] = tc[1] ? a.dlow : nullptr;
    for (int j = 0; j < 2; ++j) g.parts[j] = reinterpret_cast<bf16 *>(ws + at.parts[j]);
    g.n = a.n;
    g.R = a.R;
    g.rows = a.rows;
    g.status = status;
    if ((e = arrange(g, s)) != cudaSuccess) return (int)e;
    o.job[0] = up;
    if (one) o.job[1] = down;
    if ((e = outer(o, out_dt, s)) != cudaSuccess) return (int)e;
    if (!one) {
        o.job[0] = down;
        if ((e = outer(o, in_dt, s)) != cudaSuccess) return (int)e;
    }
    ExpandK x = {};
    fill_expand(&x, a, dA);
    x.beside = 1;
    x.w = a.down;
    x.s = a.dlow;
    x.cols = a.J;
    x.status = status;
    return (int)expand(x, dA.nranks, in_dt, in_dt, s);
}

}  // namespace shmm
