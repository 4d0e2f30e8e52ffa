// Layer normalisation for training: the forward pass that keeps each row's
// statistics (with a residual added on the way, or with the rows gathered to
// every rank), and its gradient (with the reduce-scatter that is the adjoint
// of that gather, and the reduction of the gain's and bias's gradient).
//
// For a row t of n values, with gain gamma and bias beta:
//   mean = sum(t) / n,  rstd = 1 / sqrt(sum((t - mean)^2) / n + eps)
//   xh   = (t - mean) rstd,  y = xh gamma + beta
// and with dy the gradient of y, w = dy gamma:
//   dt     = rstd (w - sum(w) / n - xh sum(w xh) / n)
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Both passes are HBM-bound (8 to 14 operations per element), so each reads
// every element once: a CTA (or, for rows of up to 512 columns, a warp) holds
// a row in registers between its reduction and its output, and every thread
// keeps the same columns in every row of the CTA's walk, so gamma, beta and
// the running dgamma, dbeta live in registers too.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "checked.cuh"
#include "device_wait.cuh"
#include "pdl.cuh"
#include "ring_order.h"
#include "shmm_internal.h"

namespace {

using shmm_dev::in_bounds;
using shmm_pdl::launch_pdl;
using shmm_pdl::pdl_enter;

// Columns one thread of the register kernels holds, and the most threads
// they give a row: rows of up to 8192 columns.  Wider rows take the
// re-reading kernels at the end.
constexpr int kCols = 16;
constexpr int kMaxThreads = 512;
// CTAs whose partial dgamma, dbeta rows the workspace holds: two per SM, more
// of narrower rows, whose CTAs are smaller.
int64_t max_parts(int64_t cols) { return cols >= 4096 ? 304 : cols >= 2048 ? 608 : 912; }

// Pointer tables: one entry for the plain call (a small parameter block
// keeps its launch short), one per rank for the gathered one.
template <int N>
struct FwdK {
    const void *src[N];   // [g*G + p]: block p of group g
    void *dst[N];         // [g*G + m]: every member's gathered buffer
    float *mean[N], *rstd[N];  // [g*G + p]
    const void *res;      // N == 1: residual, or NULL
    void *total;          // N == 1: x + residual, or NULL
    const float *gamma, *beta;
    float eps;
    int G;
    int64_t brows, cols, rows;  // rows over all blocks
    int *status;
};

template <int N>
struct BwdK {
    const void *grad[N];  // [g*G + m]: member m's gradient of the gathered rows
    const void *src[N];   // [g*G + p]: block p of group g
    const float *mean[N], *rstd[N];
    void *dst[N];
    const void *res;      // N == 1: gradient added to dt, or NULL
    const float *gamma;
    float *part;          // [gridDim.x][2][cols]
    int64_t part_floats;  // of them the workspace holds
    int G;
    int64_t brows, cols, rows;
    int *status;
};

// Two fp32 values in one register pair: one instruction for both (the issue
// slots, not the memory, bound these kernels with one value each).
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 pair(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 both(float a) { return pair(a, a); }
__device__ __forceinline__ float2 split(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// VW consecutive values as they lie in memory: one access of VW * sizeof(T)
// bytes (two for 8 fp32 values), kept packed until they are used.
template <typename T, int VW>
struct Raw {
    static constexpr int W = VW * (int)sizeof(T) / 4;  // 32-bit words
    uint32_t w[W];
    __device__ void load(const T *p) {
        if constexpr (W >= 4) {
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
                w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
            }
        }
    }
    __device__ void store(T *p) const {
#pragma unroll
        for (int i = 0; i < W / 4; ++i)
            __stcs(reinterpret_cast<uint4 *>(p) + i, make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
    }
    __device__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    __device__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
    }
    __device__ F2 get2(int i) const {  // values 2 i and 2 i + 1
        if constexpr (sizeof(T) == 4) return pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else return pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    __device__ void set2(int i, F2 v) {
        const float2 f = split(v);
        if constexpr (sizeof(T) == 4) {
            w[2 * i] = __float_as_uint(f.x);
            w[2 * i + 1] = __float_as_uint(f.y);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    __device__ void set(const float *v) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < VW; ++i) w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < VW / 2; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
    }
};
template <typename T>
struct Raw<T, 1> {
    T v;
    __device__ void load(const T *p) { v = *p; }
    __device__ void store(T *p) const { *p = v; }
    __device__ void zero() { v = T(0.0f); }
    __device__ float get(int) const { return (float)v; }
    __device__ void set(const float *f) {
        if constexpr (sizeof(T) == 4) v = *f;
        else v = __float2bfloat16_rn(*f);
    }
};

// Where row t lives: block s = g*G + p, row rr of the block, and its row in
// the gathered buffers of group g.
template <int N>
__device__ __forceinline__ void locate(int64_t t, int64_t brows, int G, int *s, int *g, int64_t *rr, int64_t *grow) {
    if constexpr (N == 1) {
        *s = 0;
        *g = 0;
        *rr = *grow = t;
    } else {
        int64_t q;
        if (t < ((int64_t)1 << 31) && brows < ((int64_t)1 << 31)) q = (uint32_t)t / (uint32_t)brows;
        else q = t / brows;
        *s = (int)q;
        *g = *s / G;
        *rr = t - q * brows;
        *grow = (int64_t)(*s - *g * G) * brows + *rr;
    }
}

// The warps' sums in order; the reads go out together.
__device__ __forceinline__ float2 sum_scratch(const float2 *s, int warps) {
    float2 t = make_float2(0.0f, 0.0f);
    for (int i0 = 0; i0 < warps; i0 += 8) {
        float2 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = i0 + i < warps ? s[i0 + i] : make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t.x += u[i].x;
            t.y += u[i].y;
        }
    }
    return t;
}

// Sum of two values over the threads of a row: shuffles, then (more than one
// warp) the warps' sums in order.  Every thread gets the same bits.
// `scratch` holds two float2 rows used in turn, so one barrier per sum is
// enough: a thread that is a sum ahead writes the other row, and a thread
// two sums ahead has passed a barrier that the slowest reader has reached.
template <bool ONEWARP>
__device__ __forceinline__ float2 row_sum(float2 v, float2 *scratch, int &turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if constexpr (ONEWARP) return v;
    float2 *s = scratch + turn * (kMaxThreads / 32);
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x / 32] = v;
    __syncthreads();
    return sum_scratch(s, blockDim.x / 32);
}

// Thread's first column of its access j: consecutive threads read
// consecutive accesses.
template <int VW, bool ONEWARP>
__device__ __forceinline__ int col_of(int j) {
    const int th = ONEWARP ? (threadIdx.x & 31) : threadIdx.x;
    const int nt = ONEWARP ? 32 : blockDim.x;
    return (th + j * nt) * VW;
}

// ---- rows in flight ----------------------------------------------------------

// Many rows: a warp or two keep whole rows coming through a ring in shared
// memory (bulk copies, an mbarrier pair per entry) while the other warps work
// on the rows that have landed, so the loads never wait for a row's two block
// sums.  An entry is one row of one buffer: x, a residual, or a member's
// gradient; copying warp i (one thread of it) takes entries i, i + COPIERS, ...
// With the rows in registers instead, what was in flight fell with every
// register the running sums took: 63 us forward and 81 us backward at 8192 x
// 4096 bf16 with a residual, where this takes 50 and 63 us (49 and 61 without the
// fence of ring_free).  Some of the gradient's kernels spill: fp32 rows of one
// block 84 to 156 bytes a thread, rows above 4096 columns up to 76.
constexpr int kMaxStages = 16;
// Forward, one block: three CTAs per SM under one another's chains of sums and
// barriers (54 -> 49 us at 8192 x 4096 bf16 with a residual; with a second
// copying warp they do not fit); gathered: two (98 against 101 us, 8 ranks).
// Backward: two, the third's registers would spill (57 against 77 us), and a
// second copying warp for its three entries a row.
constexpr int kForwardCopiers = 1, kBackwardCopiers = 2, kMaxCopiers = 2;
struct Ring {
    uint64_t full[kMaxStages], empty[kMaxStages];
    int64_t put[kMaxCopiers];  // entries of each copying thread, once it is done
    int abort_flag;
};

// One side's place in the ring.
struct Turn {
    int stage, phase;
    __device__ void next(int stages, int by = 1) {  // by <= stages
        stage += by;
        if (stage >= stages) {
            stage -= stages;
            phase ^= 1;
        }
    }
};

__device__ __forceinline__ void ring_init(Ring &ring, int stages, int readers) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            shmm_dev::mbar_init(shmm_dev::smem_u32(&ring.full[i]), 1);
            shmm_dev::mbar_init(shmm_dev::smem_u32(&ring.empty[i]), readers);
        }
        ring.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
}

// A copying thread: row `from` (or nothing, if the bounds-checked build found
// it outside its buffer) into its next entry.  False after an abort.
template <int COPIERS>
__device__ __forceinline__ bool ring_put(Ring &ring, Turn &turn, int stages, uint32_t entries, uint32_t entry_bytes,
                                         const void *from, uint32_t bytes, bool ok, int *status) {
    if (!shmm_dev::mbar_wait(shmm_dev::smem_u32(&ring.empty[turn.stage]), turn.phase ^ 1, &ring.abort_flag, status))
        return false;
    const uint32_t bar = shmm_dev::smem_u32(&ring.full[turn.stage]);
    if (ok) {
        shmm_dev::mbar_expect_tx(bar, bytes);
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                entries + turn.stage * entry_bytes),
            "l"(from), "r"(bytes), "r"(bar)
            : "memory");
    } else {
        shmm_dev::mbar_arrive(bar);
    }
    turn.next(stages, COPIERS);
    return true;
}

// The end, for every thread.  The working warps have waited for every entry,
// unless a wait was given up: then one thread (`waits`; a copying one, whose
// warp has the registers for it) waits, again with a limit, for every stage's
// last entry, so that no copy into shared memory stays in flight.  (An older
// entry of a stage was read before the last one was put.)
template <int COPIERS>
__device__ __forceinline__ void ring_end(Ring &ring, bool waits, int stages, int *status) {
    __syncwarp();
    __syncthreads();
    if (waits && *(volatile int *)&ring.abort_flag)
        for (int i = 0; i < stages; ++i) {
            const int64_t u = shmm_ring::last_entry(i, stages, COPIERS, ring.put);
            if (u >= 0)
                shmm_dev::mbar_wait(shmm_dev::smem_u32(&ring.full[i]), (uint32_t)(u / stages) & 1, &ring.abort_flag,
                                    status, false);
        }
}

// A working warp: the entry it is at has landed (after an abort it returns
// at once and what it reads is anything: the call reports the timeout) ...
__device__ __forceinline__ void ring_wait(Ring &ring, const Turn &turn, int *status) {
    shmm_dev::mbar_wait(shmm_dev::smem_u32(&ring.full[turn.stage]), turn.phase, &ring.abort_flag, status);
}
// ... and has been read.  The fence: the next copy into the entry goes through
// the async proxy, and a warp's shared-memory loads may still be in their
// queue when its arrival is counted (without it, one call in 25 had a first
// row with a piece of the third's).
__device__ __forceinline__ void ring_free(Ring &ring, Turn &turn, int stages) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if ((threadIdx.x & 31) == 0) shmm_dev::mbar_arrive(shmm_dev::smem_u32(&ring.empty[turn.stage]));
    turn.next(stages);
}

// row_sum over the first `n` threads (the working warps).
__device__ __forceinline__ float2 stream_sum(float2 v, float2 *scratch, int &turn, int n) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    float2 *s = scratch + turn * (kMaxThreads / 32);
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x / 32] = v;
    asm volatile("bar.sync 1, %0;" ::"r"(n) : "memory");
    return sum_scratch(s, n / 32);
}

// An access of VW values of T out of a ring entry.
template <typename T, int VW>
__device__ __forceinline__ void from_ring(Raw<T, VW> &r, const uint8_t *entry, int c) {
    const uint4 *p = reinterpret_cast<const uint4 *>(entry + (size_t)c * sizeof(T));
#pragma unroll
    for (int i = 0; i < Raw<T, VW>::W / 4; ++i) {
        const uint4 v = p[i];
        r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
    }
}

// ---- forward ---------------------------------------------------------------

template <typename T, int VW, int NV, int N, bool ONEWARP>
__global__ void __launch_bounds__(kMaxThreads) ln_forward_kernel(const __grid_constant__ FwdK<N> k) {
    pdl_enter();
    __shared__ float2 scratch[2 * kMaxThreads / 32];
    int turn = 0;
    const int cols = (int)k.cols;
    const float n = (float)cols;
    const int lanes_row = ONEWARP ? threadIdx.x / 32 : 0, per_cta = ONEWARP ? blockDim.x / 32 : 1;
    const int64_t step = (int64_t)gridDim.x * per_cta;
    float ga[NV][VW], be[NV][VW];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = col_of<VW, ONEWARP>(j);
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            ga[j][i] = c < cols ? k.gamma[c + i] : 0.0f;
            be[j][i] = c < cols ? k.beta[c + i] : 0.0f;
        }
    }
    const bool has_res = N == 1 && k.res;
    Raw<T, VW> v[NV], r[NV];
    auto load_row = [&](int64_t t) {
        int s, g;
        int64_t rr, grow;
        locate<N>(t, k.brows, k.G, &s, &g, &rr, &grow);
        const bool ok = in_bounds(k.status, rr * cols, cols, k.brows * cols);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = col_of<VW, ONEWARP>(j);
            v[j].zero();
            if (c < cols && ok) v[j].load((const T *)k.src[s] + rr * cols + c);
        }
        if constexpr (N == 1) {
            if (has_res) {
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int c = col_of<VW, ONEWARP>(j);
                    r[j].zero();
                    if (c < cols && ok) r[j].load((const T *)k.res + rr * cols + c);
                }
            }
        }
    };
    int64_t t = (int64_t)blockIdx.x * per_cta + lanes_row;
    if (t < k.rows) load_row(t);
    for (; t < k.rows; t += step) {
        int s, g;
        int64_t rr, grow;
        locate<N>(t, k.brows, k.G, &s, &g, &rr, &grow);
        if constexpr (N == 1) {
            // The sum is rounded to the stored type before anything is
            // computed from it: the backward pass reads the stored sum.
            if (has_res) {
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    float f[VW];
#pragma unroll
                    for (int i = 0; i < VW; ++i) f[i] = v[j].get(i) + r[j].get(i);
                    v[j].set(f);
                    const int c = col_of<VW, ONEWARP>(j);
                    if (c < cols && in_bounds(k.status, rr * cols + c, VW, k.brows * cols))
                        v[j].store((T *)k.total + rr * cols + c);
                }
            }
        }
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VW; ++i) sum.x += v[j].get(i);
        // Divided, not multiplied by 1 / n: a constant row whose sum is exact
        // then has deviations of exactly zero (rstd would magnify a last bit).
        const float mean = row_sum<ONEWARP>(sum, scratch, turn).x / n;
        float2 sq = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (col_of<VW, ONEWARP>(j) < cols)
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    const float d = v[j].get(i) - mean;
                    sq.x += d * d;
                }
        const float rstd = 1.0f / sqrtf(row_sum<ONEWARP>(sq, scratch, turn).x / n + k.eps);
        Raw<T, VW> y[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float f[VW];
#pragma unroll
            for (int i = 0; i < VW; ++i) f[i] = (v[j].get(i) - mean) * rstd * ga[j][i] + be[j][i];
            y[j].set(f);
        }
        if (t + step < k.rows) load_row(t + step);  // in flight while this row is written
        if (col_of<VW, ONEWARP>(0) == 0 && in_bounds(k.status, rr, 1, k.brows)) {
            k.mean[s][rr] = mean;
            k.rstd[s][rr] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = col_of<VW, ONEWARP>(j);
            if (c >= cols || !in_bounds(k.status, grow * cols + c, VW, k.G * k.brows * cols)) continue;
            for (int m = 0; m < k.G; ++m) y[j].store((T *)k.dst[g * k.G + m] + grow * cols + c);
        }
    }
}

// Many rows, through the ring.  blockDim.x - 32 kForwardCopiers threads work, the
// last warps copy.
template <typename T, int NV, int N, bool BIG>
__global__ void __launch_bounds__((BIG ? kMaxThreads : 256) + 32 * kForwardCopiers, BIG ? 1 : N == 1 ? 3 : 2)
    ln_forward_stream_kernel(const __grid_constant__ FwdK<N> k, int stages) {
    pdl_enter();
    constexpr int VW = 16 / (int)sizeof(T);
    extern __shared__ __align__(128) uint8_t entries[];
    __shared__ Ring ring;
    __shared__ float2 scratch[2 * kMaxThreads / 32];
    const int cols = (int)k.cols, work = blockDim.x - 32 * kForwardCopiers;
    const uint32_t bytes = (uint32_t)cols * sizeof(T);
    const bool has_res = N == 1 && k.res;
    ring_init(ring, stages, work / 32);
    if ((int)threadIdx.x >= work) {
        const int first = ((int)threadIdx.x - work) / 32;
        if ((threadIdx.x & 31) == 0) {
            // entries of a row: x, then the residual
            const uint32_t at = shmm_dev::smem_u32(entries);
            Turn turn{first, 0};
            int64_t t = blockIdx.x, put = 0;
            int e = first;
            for (bool ok = true; ok;) {
                const int per_row = has_res ? 2 : 1;
                while (e >= per_row) {
                    e -= per_row;
                    t += gridDim.x;
                }
                if (t >= k.rows) break;
                int s, g;
                int64_t rr, grow;
                locate<N>(t, k.brows, k.G, &s, &g, &rr, &grow);
                ok = ring_put<kForwardCopiers>(ring, turn, stages, at, bytes, (const T *)(e ? k.res : k.src[s]) + rr * cols, bytes,
                              in_bounds(k.status, rr * cols, cols, k.brows * cols), k.status);
                put += ok;
                e += kForwardCopiers;
            }
            ring.put[first] = put;
        }
        ring_end<kForwardCopiers>(ring, (int)threadIdx.x == work, stages, k.status);
        return;
    }
    Turn turn{0, 0};
    int sum_turn = 0;
    const float n = (float)cols;
    F2 ga[NV][VW / 2], be[NV][VW / 2];
    int col[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        col[j] = (threadIdx.x + j * work) * VW;
#pragma unroll
        for (int i = 0; i < VW / 2; ++i) {
            const bool in = col[j] < cols;
            ga[j][i] = in ? pair(k.gamma[col[j] + 2 * i], k.gamma[col[j] + 2 * i + 1]) : both(0.0f);
            be[j][i] = in ? pair(k.beta[col[j] + 2 * i], k.beta[col[j] + 2 * i + 1]) : both(0.0f);
        }
    }
    for (int64_t t = blockIdx.x; t < k.rows; t += gridDim.x) {
        int s, g;
        int64_t rr, grow;
        locate<N>(t, k.brows, k.G, &s, &g, &rr, &grow);
        Raw<T, VW> v[NV];
        ring_wait(ring, turn, k.status);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            v[j].zero();
            if (col[j] < cols) from_ring(v[j], entries + turn.stage * bytes, col[j]);
        }
        ring_free(ring, turn, stages);
        if constexpr (N == 1) {
            if (has_res) {  // rounded before anything is computed from it
                ring_wait(ring, turn, k.status);
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if (col[j] >= cols) continue;
                    Raw<T, VW> r;
                    from_ring(r, entries + turn.stage * bytes, col[j]);
#pragma unroll
                    for (int i = 0; i < VW / 2; ++i) v[j].set2(i, v[j].get2(i) + r.get2(i));
                    if (in_bounds(k.status, rr * cols + col[j], VW, k.brows * cols))
                        v[j].store((T *)k.total + rr * cols + col[j]);
                }
                ring_free(ring, turn, stages);
            }
        }
        F2 sum = both(0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VW / 2; ++i) sum = sum + v[j].get2(i);
        float2 part = split(sum);
        const float mean = stream_sum(make_float2(part.x + part.y, 0.0f), scratch, sum_turn, work).x / n;
        const F2 minus = both(-mean);
        F2 sq = both(0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (col[j] < cols)
#pragma unroll
                for (int i = 0; i < VW / 2; ++i) {
                    const F2 d = v[j].get2(i) + minus;
                    sq = fma(d, d, sq);
                }
        part = split(sq);
        const float rstd =
            1.0f / sqrtf(stream_sum(make_float2(part.x + part.y, 0.0f), scratch, sum_turn, work).x / n + k.eps);
        const F2 scale = both(rstd);
        if (threadIdx.x == 0 && in_bounds(k.status, rr, 1, k.brows)) {
            k.mean[s][rr] = mean;
            k.rstd[s][rr] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (col[j] >= cols || !in_bounds(k.status, grow * cols + col[j], VW, k.G * k.brows * cols)) continue;
            Raw<T, VW> y;
#pragma unroll
            for (int i = 0; i < VW / 2; ++i) y.set2(i, fma((v[j].get2(i) + minus) * scale, ga[j][i], be[j][i]));
            for (int m = 0; m < k.G; ++m) y.store((T *)k.dst[g * k.G + m] + grow * cols + col[j]);
        }
    }
    ring_end<kForwardCopiers>(ring, false, stages, k.status);
}

// Rows of any width: the row is read three times (from L2 after the first).
template <typename T, int N>
__global__ void __launch_bounds__(kMaxThreads) ln_forward_wide_kernel(const __grid_constant__ FwdK<N> k) {
    pdl_enter();
    __shared__ float2 scratch[2 * kMaxThreads / 32];
    int turn = 0;
    const float n = (float)k.cols;
    for (int64_t t = blockIdx.x; t < k.rows; t += gridDim.x) {
        int s, g;
        int64_t rr, grow;
        locate<N>(t, k.brows, k.G, &s, &g, &rr, &grow);
        if (!in_bounds(k.status, rr * k.cols, k.cols, k.brows * k.cols) ||
            !in_bounds(k.status, grow * k.cols, k.cols, k.G * k.brows * k.cols))
            continue;  // the same for the whole CTA
        const T *x = (const T *)k.src[s] + rr * k.cols;
        float2 sum = make_float2(0.0f, 0.0f);
        for (int64_t c = threadIdx.x; c < k.cols; c += blockDim.x) {
            float f = (float)x[c];
            if (N == 1 && k.res) {
                Raw<T, 1> o;
                f += (float)((const T *)k.res)[rr * k.cols + c];
                o.set(&f);
                o.store((T *)k.total + rr * k.cols + c);
                f = o.get(0);
            }
            sum.x += f;
        }
        if (N == 1 && k.res) x = (const T *)k.total + rr * k.cols;  // each thread reads back its own columns
        const float mean = row_sum<false>(sum, scratch, turn).x / n;
        float2 sq = make_float2(0.0f, 0.0f);
        for (int64_t c = threadIdx.x; c < k.cols; c += blockDim.x) {
            const float d = (float)x[c] - mean;
            sq.x += d * d;
        }
        const float rstd = 1.0f / sqrtf(row_sum<false>(sq, scratch, turn).x / n + k.eps);
        if (threadIdx.x == 0) {
            k.mean[s][rr] = mean;
            k.rstd[s][rr] = rstd;
        }
        for (int64_t c = threadIdx.x; c < k.cols; c += blockDim.x) {
            const float f = ((float)x[c] - mean) * rstd * k.gamma[c] + k.beta[c];
            Raw<T, 1> o;
            o.set(&f);
            for (int m = 0; m < k.G; ++m) o.store((T *)k.dst[g * k.G + m] + grow * k.cols + c);
        }
    }
}

// ---- backward --------------------------------------------------------------

template <typename T, typename GT, int VW, int NV, int N, bool ONEWARP>
__global__ void __launch_bounds__(kMaxThreads) ln_backward_kernel(const __grid_constant__ BwdK<N> k) {
    pdl_enter();
    __shared__ float2 scratch[2 * kMaxThreads / 32];
    int turn = 0;
    const int cols = (int)k.cols;
    const float inv_n = 1.0f / (float)cols;
    const int lanes_row = ONEWARP ? threadIdx.x / 32 : 0, per_cta = ONEWARP ? blockDim.x / 32 : 1;
    const int64_t step = (int64_t)gridDim.x * per_cta;
    float ga[NV][VW], dg[NV][VW], db[NV][VW];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = col_of<VW, ONEWARP>(j);
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            ga[j][i] = c < cols ? k.gamma[c + i] : 0.0f;
            dg[j][i] = db[j][i] = 0.0f;
        }
    }
    Raw<T, VW> x[NV];
    Raw<GT, VW> d0[NV];  // the first member's gradient
    auto load_row = [&](int64_t t) {
        int s, g;
        int64_t rr, grow;
        locate<N>(t, k.brows, k.G, &s, &g, &rr, &grow);
        const bool ok = in_bounds(k.status, rr * cols, cols, k.brows * cols) &&
                        in_bounds(k.status, grow * cols, cols, k.G * k.brows * cols);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = col_of<VW, ONEWARP>(j);
            x[j].zero();
            d0[j].zero();
            if (c < cols && ok) {
                x[j].load((const T *)k.src[s] + rr * cols + c);
                d0[j].load((const GT *)k.grad[g * k.G] + grow * cols + c);
            }
        }
    };
    int64_t t = (int64_t)blockIdx.x * per_cta + lanes_row;
    if (t < k.rows) load_row(t);
    for (; t < k.rows; t += step) {
        int s, g;
        int64_t rr, grow;
        locate<N>(t, k.brows, k.G, &s, &g, &rr, &grow);
        // x - mean before anything else, not x rstd - mean rstd: in a row whose
        // values differ little the second's own rounding would be the result.
        const bool known = in_bounds(k.status, rr, 1, k.brows);
        const float mean = known ? k.mean[s][rr] : 0.0f, rstd = known ? k.rstd[s][rr] : 0.0f;
        float dy[NV][VW];
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VW; ++i) dy[j][i] = d0[j].get(i);
        if constexpr (N > 1) {  // the members' gradients in rank order
#pragma unroll 4
            for (int m = 1; m < k.G; ++m) {
                Raw<GT, VW> d[NV];
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int c = col_of<VW, ONEWARP>(j);
                    d[j].zero();
                    if (c < cols && in_bounds(k.status, grow * cols + c, VW, k.G * k.brows * cols))
                        d[j].load((const GT *)k.grad[g * k.G + m] + grow * cols + c);
                }
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int i = 0; i < VW; ++i) dy[j][i] += d[j].get(i);
            }
        }
        float2 sum = make_float2(0.0f, 0.0f);  // of w and of w xh
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (col_of<VW, ONEWARP>(j) < cols)
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    const float xh = (x[j].get(i) - mean) * rstd, w = dy[j][i] * ga[j][i];
                    sum.x += w;
                    sum.y = fmaf(w, xh, sum.y);
                    dg[j][i] = fmaf(dy[j][i], xh, dg[j][i]);
                    db[j][i] += dy[j][i];
                }
        sum = row_sum<ONEWARP>(sum, scratch, turn);
        // xh before its factor, not (x - mean) times rstd^2, which overflows where
        // rows are small and eps is 0 (rstd above 2^64), though the result does not.
        const float k1 = -rstd * (sum.x * inv_n), k2 = -rstd * (sum.y * inv_n);
        float o[NV][VW];
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                o[j][i] = fmaf((x[j].get(i) - mean) * rstd, k2, fmaf(dy[j][i] * ga[j][i], rstd, k1));
            }
        if (t + step < k.rows) load_row(t + step);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = col_of<VW, ONEWARP>(j);
            if (c >= cols || !in_bounds(k.status, rr * cols + c, VW, k.brows * cols)) continue;
            if constexpr (N == 1) {
                if (k.res) {
                    Raw<T, VW> r;
                    r.load((const T *)k.res + rr * cols + c);
#pragma unroll
                    for (int i = 0; i < VW; ++i) o[j][i] += r.get(i);
                }
            }
            Raw<T, VW> y;
            y.set(o[j]);
            y.store((T *)k.dst[s] + rr * cols + c);
        }
    }
    // This CTA's rows' sums.  One warp per row: the warps' sums in order.
    if (!in_bounds(k.status, (int64_t)blockIdx.x * 2 * cols, 2 * cols, k.part_floats)) return;
    float *part = k.part + (int64_t)blockIdx.x * 2 * cols;
    if constexpr (ONEWARP) {
        __shared__ float sh[(kMaxThreads / 32) * 32 * NV * VW];
        const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, nw = blockDim.x / 32;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VW; ++i)
                    sh[warp * 32 * NV * VW + (lane + j * 32) * VW + i] = h ? db[j][i] : dg[j][i];
            __syncthreads();
            for (int c = threadIdx.x; c < cols; c += blockDim.x) {
                float a = 0.0f;
                for (int w = 0; w < nw; ++w) a += sh[w * 32 * NV * VW + c];
                part[h * cols + c] = a;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = col_of<VW, ONEWARP>(j);
            if (c >= cols) continue;
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                part[c + i] = dg[j][i];
                part[cols + c + i] = db[j][i];
            }
        }
    }
}

// Many rows, through the ring: per row the members' gradients in rank order,
// x, and the residual's gradient.
template <typename T, typename GT, int NV, int N, bool BIG>
__global__ void __launch_bounds__((BIG ? kMaxThreads : 256) + 32 * kBackwardCopiers, BIG ? 1 : 2)
    ln_backward_stream_kernel(const __grid_constant__ BwdK<N> k, int stages) {
    pdl_enter();
    constexpr int VW = 16 / (int)sizeof(T);
    extern __shared__ __align__(128) uint8_t entries[];
    __shared__ Ring ring;
    __shared__ float2 scratch[2 * kMaxThreads / 32];
    const int cols = (int)k.cols, work = blockDim.x - 32 * kBackwardCopiers;
    const uint32_t bytes = (uint32_t)cols * sizeof(T), gbytes = (uint32_t)cols * sizeof(GT);
    const uint32_t entry = gbytes > bytes ? gbytes : bytes;
    const bool has_res = N == 1 && k.res;
    // gamma: with one member in registers, with several, whose sum takes the
    // registers, in shared memory (8 fp32 members: 184 against 198 us; one
    // member: 57 in registers against 64).
    float *gains = reinterpret_cast<float *>(entries + (size_t)stages * entry);
    F2 gr[N == 1 ? NV : 1][VW / 2];
    ring_init(ring, stages, work / 32);
    if ((int)threadIdx.x >= work) {
        const int first = ((int)threadIdx.x - work) / 32;
        if ((threadIdx.x & 31) == 0) {
            const int per_row = k.G + 1 + (has_res ? 1 : 0);
            const uint32_t at = shmm_dev::smem_u32(entries);
            Turn turn{first, 0};
            int64_t t = blockIdx.x, put = 0;
            int e = first, s, g;  // the next entry: number e of row t
            int64_t rr, grow;
            if (t < k.rows) locate<N>(t, k.brows, k.G, &s, &g, &rr, &grow);
            for (bool ok = true; ok;) {
                if (e >= per_row) {  // kBackwardCopiers <= per_row: the next row
                    e -= per_row;
                    t += gridDim.x;
                    if (t < k.rows) locate<N>(t, k.brows, k.G, &s, &g, &rr, &grow);
                }
                if (t >= k.rows) break;
                if (e < k.G)
                    ok = ring_put<kBackwardCopiers>(ring, turn, stages, at, entry, (const GT *)k.grad[g * k.G + e] + grow * cols, gbytes,
                                  in_bounds(k.status, grow * cols, cols, k.G * k.brows * cols), k.status);
                else
                    ok = ring_put<kBackwardCopiers>(ring, turn, stages, at, entry,
                                  (const T *)(N == 1 && e > k.G ? k.res : k.src[s]) + rr * cols, bytes,
                                  in_bounds(k.status, rr * cols, cols, k.brows * cols), k.status);
                put += ok;
                e += kBackwardCopiers;
            }
            ring.put[first] = put;
        }
        ring_end<kBackwardCopiers>(ring, (int)threadIdx.x == work, stages, k.status);
        return;
    }
    Turn turn{0, 0};
    int sum_turn = 0;
    const float inv_n = 1.0f / (float)cols;
    F2 dg[NV][VW / 2], db[NV][VW / 2];
    int col[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        col[j] = (threadIdx.x + j * work) * VW;
#pragma unroll
        for (int i = 0; i < VW / 2; ++i) {
            dg[j][i] = db[j][i] = both(0.0f);
            const float2 two = col[j] < cols ? make_float2(k.gamma[col[j] + 2 * i], k.gamma[col[j] + 2 * i + 1])
                                             : make_float2(0.0f, 0.0f);
            if constexpr (N == 1) gr[j][i] = pair(two.x, two.y);
            else if (col[j] < cols) *reinterpret_cast<float2 *>(gains + col[j] + 2 * i) = two;
        }
    }
    auto ga = [&](int j, int i) {
        if constexpr (N == 1) return gr[j][i];
        else return F2{*reinterpret_cast<const uint64_t *>(gains + col[j] + 2 * i)};
    };
    float mean = 0.0f, rstd = 0.0f;  // read a row ahead
    auto read_stats = [&](int64_t t) {
        int s, g;
        int64_t rr, grow;
        locate<N>(t, k.brows, k.G, &s, &g, &rr, &grow);
        if (!in_bounds(k.status, rr, 1, k.brows)) return;
        mean = k.mean[s][rr];
        rstd = k.rstd[s][rr];
    };
    if ((int64_t)blockIdx.x < k.rows) read_stats(blockIdx.x);
    for (int64_t t = blockIdx.x; t < k.rows; t += gridDim.x) {
        int s, g;
        int64_t rr, grow;
        locate<N>(t, k.brows, k.G, &s, &g, &rr, &grow);
        // The members' gradients.  One member's stay packed until they are used.
        Raw<GT, VW> d0[NV];
        F2 dys[NV][VW / 2];
        for (int m = 0; m < k.G; ++m) {
            ring_wait(ring, turn, k.status);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if constexpr (N == 1) d0[j].zero();
                if (N > 1 && m == 0)
#pragma unroll
                    for (int i = 0; i < VW / 2; ++i) dys[j][i] = both(0.0f);
                if (col[j] >= cols) continue;
                if constexpr (N == 1) {
                    from_ring(d0[j], entries + turn.stage * entry, col[j]);
                } else {
                    Raw<GT, VW> d;
                    from_ring(d, entries + turn.stage * entry, col[j]);
#pragma unroll
                    for (int i = 0; i < VW / 2; ++i) dys[j][i] = m ? dys[j][i] + d.get2(i) : d.get2(i);
                }
            }
            ring_free(ring, turn, stages);
        }
        auto dy = [&](int j, int i) { return N == 1 ? d0[j].get2(i) : dys[j][i]; };
        Raw<T, VW> x[NV];
        ring_wait(ring, turn, k.status);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            x[j].zero();
            if (col[j] < cols) from_ring(x[j], entries + turn.stage * entry, col[j]);
        }
        ring_free(ring, turn, stages);
        const float rs = rstd;
        const F2 minus = both(-mean);  // x - mean first (see ln_backward_kernel)
        if (t + gridDim.x < k.rows) read_stats(t + gridDim.x);
        const F2 rs2 = both(rs);
        F2 sw = both(0.0f), swx = both(0.0f);  // of w and of w xh
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (col[j] < cols)
#pragma unroll
                for (int i = 0; i < VW / 2; ++i) {
                    const F2 d = dy(j, i), xh = (x[j].get2(i) + minus) * rs2, w = d * ga(j, i);
                    sw = sw + w;
                    swx = fma(w, xh, swx);
                    dg[j][i] = fma(d, xh, dg[j][i]);
                    db[j][i] = db[j][i] + d;
                }
        const float2 pw = split(sw), px = split(swx);
        const float2 sum = stream_sum(make_float2(pw.x + pw.y, px.x + px.y), scratch, sum_turn, work);
        const F2 k1 = both(-rs * (sum.x * inv_n)), k2 = both(-rs * (sum.y * inv_n));  // (see ln_backward_kernel)
        if (has_res) ring_wait(ring, turn, k.status);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (col[j] >= cols) continue;
            F2 o[VW / 2];
#pragma unroll
            for (int i = 0; i < VW / 2; ++i)
                o[i] = fma((x[j].get2(i) + minus) * rs2, k2, fma(dy(j, i) * ga(j, i), rs2, k1));
            if constexpr (N == 1) {
                if (has_res) {
                    Raw<T, VW> r;
                    from_ring(r, entries + turn.stage * entry, col[j]);
#pragma unroll
                    for (int i = 0; i < VW / 2; ++i) o[i] = o[i] + r.get2(i);
                }
            }
            Raw<T, VW> y;
#pragma unroll
            for (int i = 0; i < VW / 2; ++i) y.set2(i, o[i]);
            if (in_bounds(k.status, rr * cols + col[j], VW, k.brows * cols)) y.store((T *)k.dst[s] + rr * cols + col[j]);
        }
        if (has_res) ring_free(ring, turn, stages);
    }
    float *part = k.part + (int64_t)blockIdx.x * 2 * cols;
    const bool room = in_bounds(k.status, (int64_t)blockIdx.x * 2 * cols, 2 * cols, k.part_floats);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (col[j] >= cols || !room) continue;
#pragma unroll
        for (int i = 0; i < VW / 2; ++i) {
            *reinterpret_cast<float2 *>(part + col[j] + 2 * i) = split(dg[j][i]);
            *reinterpret_cast<float2 *>(part + cols + col[j] + 2 * i) = split(db[j][i]);
        }
    }
    ring_end<kBackwardCopiers>(ring, false, stages, k.status);
}

// Rows of any width: the row is read twice, and each thread adds its columns
// of dgamma and dbeta to the CTA's partial row, which it zeroes first.
template <typename T, typename GT, int N>
__global__ void __launch_bounds__(kMaxThreads) ln_backward_wide_kernel(const __grid_constant__ BwdK<N> k) {
    pdl_enter();
    __shared__ float2 scratch[2 * kMaxThreads / 32];
    int turn = 0;
    const float inv_n = 1.0f / (float)k.cols;
    if (!in_bounds(k.status, (int64_t)blockIdx.x * 2 * k.cols, 2 * k.cols, k.part_floats)) return;
    float *part = k.part + (int64_t)blockIdx.x * 2 * k.cols;
    for (int64_t c = threadIdx.x; c < k.cols; c += blockDim.x) part[c] = part[k.cols + c] = 0.0f;
    for (int64_t t = blockIdx.x; t < k.rows; t += gridDim.x) {
        int s, g;
        int64_t rr, grow;
        locate<N>(t, k.brows, k.G, &s, &g, &rr, &grow);
        if (!in_bounds(k.status, rr * k.cols, k.cols, k.brows * k.cols) ||
            !in_bounds(k.status, grow * k.cols, k.cols, k.G * k.brows * k.cols))
            continue;  // the same for the whole CTA
        const T *x = (const T *)k.src[s] + rr * k.cols;
        const bool known = in_bounds(k.status, rr, 1, k.brows);
        const float mean = known ? k.mean[s][rr] : 0.0f, rstd = known ? k.rstd[s][rr] : 0.0f;
        auto grad = [&](int64_t c) {
            float dy = (float)((const GT *)k.grad[g * k.G])[grow * k.cols + c];
            for (int m = 1; m < k.G; ++m) dy += (float)((const GT *)k.grad[g * k.G + m])[grow * k.cols + c];
            return dy;
        };
        float2 sum = make_float2(0.0f, 0.0f);
        for (int64_t c = threadIdx.x; c < k.cols; c += blockDim.x) {
            const float dy = grad(c), xh = ((float)x[c] - mean) * rstd, w = dy * k.gamma[c];
            sum.x += w;
            sum.y += w * xh;
            part[c] += dy * xh;
            part[k.cols + c] += dy;
        }
        sum = row_sum<false>(sum, scratch, turn);
        const float c1 = sum.x * inv_n, c2 = sum.y * inv_n;
        for (int64_t c = threadIdx.x; c < k.cols; c += blockDim.x) {
            const float xh = ((float)x[c] - mean) * rstd;
            float o = rstd * (grad(c) * k.gamma[c] - c1 - xh * c2);
            if (N == 1 && k.res) o += (float)((const T *)k.res)[rr * k.cols + c];
            Raw<T, 1> y;
            y.set(&o);
            y.store((T *)k.dst[s] + rr * k.cols + c);
        }
    }
}

// dgamma and dbeta: the CTAs' partial rows, column by column.  A CTA takes 32
// columns of the [parts][2 cols] array; warp y adds rows y, y + 32, ..., ten at
// a time in pairs, and the 32 sums are added in pairs: a fixed order, so one
// input gives one result, and few additions deep (in a row they were off by
// 1.5e-7 at 1031 rows, more than the sums that made them).  parts == 0 (no
// rows) writes zeros.
__global__ void __launch_bounds__(1024) ln_grad_sum_kernel(const float *part, int parts, int64_t part_floats, int64_t cols,
                                                           float *dgamma, float *dbeta, int *status) {
    pdl_enter();
    __shared__ float sh[32][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float a = 0.0f;
    if (c < 2 * cols) {
        constexpr int U = 10;  // loads in flight
        for (int p0 = threadIdx.y; p0 < parts; p0 += 32 * U) {
            float v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t at = (int64_t)(p0 + 32 * u) * 2 * cols + c;
                v[u] = p0 + 32 * u < parts && in_bounds(status, at, 1, part_floats) ? part[at] : 0.0f;
            }
            a += (((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]))) + (v[8] + v[9]);
        }
    }
    sh[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && c < 2 * cols) {
        float t[32];
#pragma unroll
        for (int y = 0; y < 32; ++y) t[y] = sh[y][threadIdx.x];
#pragma unroll
        for (int h = 16; h > 0; h /= 2)
#pragma unroll
            for (int y = 0; y < h; ++y) t[y] += t[y + h];
        if (c < cols) dgamma[c] = t[0];
        else dbeta[c - cols] = t[0];
    }
}

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

// Threads per row and accesses per thread for `cols` columns in accesses of
// VW values.  `spread` gives a row more threads with fewer columns each.
struct Shape {
    int nv, threads;
    bool onewarp;
};
Shape shape_for(int64_t cols, int vw, int want_cols) {
    const int nvec = (int)((cols + vw - 1) / vw);
    if (cols <= 32 * kCols && want_cols >= kCols) return {kCols / vw, 256, true};
    int nv = want_cols / vw;
    if (vw == 1 && nv < 4) nv = 4;
    while ((nvec + nv - 1) / nv > kMaxThreads) nv *= vw == 1 ? 4 : 2;
    const int threads = ((nvec + nv - 1) / nv + 31) / 32 * 32;
    return {nv, threads, false};
}

// Launch shape of the ring kernels: CTAs per SM for `threads` working threads,
// and the ring's entries of `entry` bytes in each CTA's share of an SM.
struct StreamShape {
    int threads, per_sm, stages;
    size_t smem;
};
StreamShape stream_shape(int64_t cols, int64_t entry, int64_t extra, int most) {  // most: CTAs of 256 threads
    StreamShape h;
    h.threads = (int)((cols + kCols * 32 - 1) / (kCols * 32)) * 32;
    h.per_sm = h.threads > 256 ? 1 : most * 256 / h.threads > 6 ? 6 : most * 256 / h.threads;
    const int64_t budget = (220 * 1024) / h.per_sm - 2048 - extra;
    h.stages = (int)(budget / entry < kMaxStages ? budget / entry : kMaxStages);
    h.smem = (size_t)(h.stages * entry + extra);
    return h;
}

template <typename K>
cudaError_t launch_stream(void (*kern)(K, int), const K &k, const StreamShape &h, int copiers, int64_t grid, cudaStream_t s,
                          shmm::PerDevice<int> *done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= shmm::kMaxDevices) return cudaErrorInvalidDevice;
    if (!done->get(dev)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
        if (e != cudaSuccess) return e;
        done->set(dev, 1);
    }
    return launch_pdl(kern, dim3((unsigned)grid), dim3((unsigned)h.threads + 32 * copiers), h.smem, s, k, h.stages);
}

// Rows enough for the ring kernels: every CTA has three rows or more to keep
// in flight.
bool stream_rows(int64_t rows, int64_t cols) { return cols > 32 * kCols && rows >= 6 * sms(); }

template <typename T, int N, bool BIG>
cudaError_t forward_stream(const FwdK<N> &k, cudaStream_t s) {
    constexpr int VW = 16 / (int)sizeof(T);
    static shmm::PerDevice<int> done;
    const StreamShape h = stream_shape(k.cols, k.cols * (int64_t)sizeof(T), 0, N == 1 ? 3 : 2);
    return launch_stream(ln_forward_stream_kernel<T, kCols / VW, N, BIG>, k, h, kForwardCopiers,
                         (int64_t)sms() * h.per_sm, s, &done);
}

template <typename T, typename GT, int N, bool BIG>
cudaError_t backward_stream(const BwdK<N> &k, int *parts, cudaStream_t s) {
    constexpr int VW = 16 / (int)sizeof(T);
    static shmm::PerDevice<int> done;
    const StreamShape h = stream_shape(k.cols, k.cols * (int64_t)(sizeof(T) > sizeof(GT) ? sizeof(T) : sizeof(GT)),
                                       N == 1 ? 0 : k.cols * 4, 2);
    int64_t grid = (int64_t)sms() * h.per_sm;
    if (grid > max_parts(k.cols)) grid = max_parts(k.cols);
    *parts = (int)grid;
    return launch_stream(ln_backward_stream_kernel<T, GT, kCols / VW, N, BIG>, k, h, kBackwardCopiers, grid, s, &done);
}

template <typename T, int VW, int N>
cudaError_t forward_vec(const FwdK<N> &k, cudaStream_t s) {
    const bool few = k.rows < sms();
    const Shape h = shape_for(k.cols, VW, few ? VW : kCols);
    const int64_t per_cta = h.onewarp ? h.threads / 32 : 1;
    int64_t grid = (k.rows + per_cta - 1) / per_cta;
    const int64_t cap = (int64_t)sms() * (1024 / h.threads > 0 ? 1024 / h.threads : 1);
    if (grid > cap) grid = cap;
    const dim3 g((unsigned)grid), b((unsigned)h.threads);
    constexpr int kMost = kCols / VW;  // accesses of a thread that holds kCols columns
    if (h.onewarp) return launch_pdl(ln_forward_kernel<T, VW, kMost, N, true>, g, b, 0, s, k);
    if (h.nv == kMost) return launch_pdl(ln_forward_kernel<T, VW, kMost, N, false>, g, b, 0, s, k);
    if (h.nv == kMost / 2 && VW > 1) return launch_pdl(ln_forward_kernel<T, VW, (VW > 1 ? kMost / 2 : kMost), N, false>, g, b, 0, s, k);
    if (h.nv == kMost / 4 && VW < 8) return launch_pdl(ln_forward_kernel<T, VW, (VW < 8 ? kMost / 4 : kMost), N, false>, g, b, 0, s, k);
    return cudaErrorInvalidValue;
}

template <typename T, int N>
cudaError_t forward(const FwdK<N> &k, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    if (k.cols > (int64_t)kMaxThreads * kCols) {
        const int64_t cap = (int64_t)sms() * 2;
        const dim3 g((unsigned)(k.rows < cap ? k.rows : cap));
        return launch_pdl(ln_forward_wide_kernel<T, N>, g, dim3(kMaxThreads), 0, s, k);
    }
    if (k.cols % V) return forward_vec<T, 1, N>(k, s);
    if (!stream_rows(k.rows, k.cols)) return forward_vec<T, V, N>(k, s);
    return k.cols > 256 * kCols ? forward_stream<T, N, true>(k, s) : forward_stream<T, N, false>(k, s);
}

template <typename T, typename GT, int VW, int N>
cudaError_t backward_vec(const BwdK<N> &k, int *parts, cudaStream_t s) {
    const Shape h = shape_for(k.cols, VW, kCols);
    const int64_t per_cta = h.onewarp ? h.threads / 32 : 1;
    int64_t grid = (k.rows + per_cta - 1) / per_cta;
    int64_t cap = (int64_t)sms() * (h.threads > 256 ? 1 : 512 / h.threads > 6 ? 6 : 512 / h.threads);
    if (cap > max_parts(k.cols)) cap = max_parts(k.cols);
    if (grid > cap) grid = cap;
    *parts = (int)grid;
    const dim3 g((unsigned)grid), b((unsigned)h.threads);
    constexpr int kMost = kCols / VW;  // accesses of a thread that holds kCols columns
    if (h.onewarp) return launch_pdl(ln_backward_kernel<T, GT, VW, kMost, N, true>, g, b, 0, s, k);
    return launch_pdl(ln_backward_kernel<T, GT, VW, kMost, N, false>, g, b, 0, s, k);
}

template <typename T, typename GT, int N>
cudaError_t backward(const BwdK<N> &k, int *parts, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    if (k.cols > (int64_t)kMaxThreads * kCols) {
        int64_t cap = (int64_t)sms();
        if (cap > max_parts(k.cols)) cap = max_parts(k.cols);
        *parts = (int)(k.rows < cap ? k.rows : cap);
        return launch_pdl(ln_backward_wide_kernel<T, GT, N>, dim3((unsigned)*parts), dim3(kMaxThreads), 0, s, k);
    }
    if (k.cols % V) return backward_vec<T, GT, 1, N>(k, parts, s);
    if (!stream_rows(k.rows, k.cols)) return backward_vec<T, GT, V, N>(k, parts, s);
    return k.cols > 256 * kCols ? backward_stream<T, GT, N, true>(k, parts, s)
                                : backward_stream<T, GT, N, false>(k, parts, s);
}

template <int N>
cudaError_t run_forward(const shmm::NormForwardArgs &a, int *status, cudaStream_t s) {
    FwdK<N> k;
    for (int i = 0; i < a.ngroups * a.G; ++i) {
        k.src[i] = a.src[i];
        k.dst[i] = a.dst[i];
        k.mean[i] = a.mean[i];
        k.rstd[i] = a.rstd[i];
    }
    k.res = a.res;
    k.total = a.total;
    k.gamma = a.gamma;
    k.beta = a.beta;
    k.eps = a.eps;
    k.G = a.G;
    k.brows = a.brows;
    k.cols = a.cols;
    k.rows = (int64_t)a.ngroups * a.G * a.brows;
    k.status = status;
    shmm::count_launch();
    return a.dt == SHMM_F32 ? forward<float, N>(k, s) : forward<__nv_bfloat16, N>(k, s);
}

template <int N>
cudaError_t run_backward(const shmm::NormBackwardArgs &a, int *status, cudaStream_t s) {
    BwdK<N> k;
    for (int i = 0; i < a.ngroups * a.G; ++i) {
        k.grad[i] = a.grad[i];
        k.src[i] = a.src[i];
        k.dst[i] = a.dst[i];
        k.mean[i] = a.mean[i];
        k.rstd[i] = a.rstd[i];
    }
    k.res = a.res;
    k.gamma = a.gamma;
    k.part = a.workspace;
    k.part_floats = (int64_t)(shmm::norm_workspace_bytes((int64_t)a.ngroups * a.G * a.brows, a.cols) / sizeof(float));
    k.G = a.G;
    k.brows = a.brows;
    k.cols = a.cols;
    k.rows = (int64_t)a.ngroups * a.G * a.brows;
    k.status = status;
    int parts = 0;
    cudaError_t e = cudaSuccess;
    if (k.rows > 0) {
        shmm::count_launch();
        if (a.dt == SHMM_F32) {
            e = backward<float, float, N>(k, &parts, s);
        } else if (a.grad_dt == SHMM_BF16) {
            e = backward<__nv_bfloat16, __nv_bfloat16, N>(k, &parts, s);
        } else {  // partial sums of several members
            if constexpr (N > 1) e = backward<__nv_bfloat16, float, N>(k, &parts, s);
            else e = cudaErrorInvalidValue;
        }
        if (e != cudaSuccess) return e;
    }
    shmm::count_launch();
    return launch_pdl(ln_grad_sum_kernel, dim3((unsigned)((2 * a.cols + 31) / 32)), dim3(32, 32), 0, s,
                      (const float *)a.workspace, parts, k.part_floats, a.cols, a.dgamma, a.dbeta, status);
}

}  // namespace

namespace shmm {

size_t norm_workspace_bytes(int64_t rows, int64_t cols) {
    const int64_t most = max_parts(cols), parts = rows < most ? rows : most;
    return (size_t)(parts * 2 * cols * 4);
}

int launch_norm_forward(const NormForwardArgs &a, int *status, void *stream) {
    if (a.ngroups * a.G > SHMM_MAX_RANKS) return (int)cudaErrorInvalidValue;
    if (a.brows == 0 || a.cols == 0) return 0;
    return (int)(a.ngroups * a.G == 1 ? run_forward<1>(a, status, (cudaStream_t)stream)
                                      : run_forward<SHMM_MAX_RANKS>(a, status, (cudaStream_t)stream));
}

int launch_norm_backward(const NormBackwardArgs &a, int *status, void *stream) {
    if (a.ngroups * a.G > SHMM_MAX_RANKS) return (int)cudaErrorInvalidValue;
    if (a.cols == 0) return 0;
    return (int)(a.ngroups * a.G == 1 ? run_backward<1>(a, status, (cudaStream_t)stream)
                                      : run_backward<SHMM_MAX_RANKS>(a, status, (cudaStream_t)stream));
}

}  // namespace shmm
