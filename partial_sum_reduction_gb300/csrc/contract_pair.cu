// The products of the gated MLP block and of 8-bit operands on the tensor
// cores: CTA pairs (cta_group::2, M = 256), operands by TMA from the ranks'
// shards in place, accumulators in TMEM, results by bulk tensor stores to every
// rank that holds them.
//
// One kernel, six forms (X: the first operand, Y: the second):
//   kGated  X [M,Kd] . Y0, Y1 [Kd,N] bf16: both projections of a gated MLP
//           block.  A 256-column accumulator is 128 columns of the gate's and the
//           same 128 of the up projection's: the pair's even CTA loads Y0's
//           columns, the odd one Y1's, so one MMA computes both and the product
//           of the two needs no exchange.
//   kGated8 the same where the projections are kept in 8 bits
//   kNT     X [M,Kd] . Y [N,Kd]^T bf16, summed over terms: dA = dG . gate^T +
//           dU . up^T is one contraction over both.
//   kTN     X [Kd,M]^T . Y [Kd,N] bf16: a weight gradient.  With two Y (dG, dU),
//           one in each half of the tile, X is loaded once for both.
//   kNN8    X [M,Kd] . Y [Kd,N] in 8 bits with block scales (the forward call)
//   kNT8    X [M,Kd] . Y [N,Kd]^T in 8 bits (dA)
// Nothing is transposed in memory: the MMA reads either operand K-major or
// MN-major from 128-byte-swizzled tiles.
//
// kGated, kNT, kTN: 256 x 512 accumulators (two MMAs of N = 256 per K step, sharing
// X: the tile that moves fewest operand bytes per FLOP), all of TMEM.  The
// contraction stays in one fp32 accumulator; results are bf16.  The epilogue
// takes half a tile's accumulator into registers at once and hands the TMEM
// back before it computes and stores, so the next tile's MMAs wait for a TMEM
// read and not for the stores.  8192 x 4096 by 2 x 4096 x 16384: kGated 1.05 to
// 1.08 ms, 2.04 to 2.10 PFLOP/s (1.06 to 1.09 of the measured bf16 rate; 1.11 to
// 1.16 ms where it keeps the projections in bf16), kNT and kTN 1.11 to 1.18 ms;
// the tensor cores are busy for 93 to 96 % of the cycles, and the power cap sets
// the clock of calls in a row.
//
// kNN8, kNT8: a k-block is 128 values, the scales' block.  Its four MMAs (K =
// 32) fill one of two 256 x 256 accumulators; the epilogue warps read it and
// add it times the two scales to fp32 sums in their registers (128 per thread)
// while the next k-block fills the other.  No sum is longer than 128 products
// in the tensor cores' adders, whose additions truncate.  Measured: 8192 x 8192
// x 28672 in 1.84 ms, 2.09 PFLOP/s, 1.08 of the measured bf16 rate; 965 cycles
// per k-block, where its MMAs take 512.  What bounds it is the way round one
// accumulator, which two k-blocks share: 750 cycles from the issue of the MMAs to
// the signal, some 900 until the last warp has read its part, 260 until the next
// MMAs are issued.  TMEM has no room for a third; reading two or four pieces at a
// time, packed FMAs and other splits of the reads changed nothing (1.84 to 1.87
// ms).  16 epilogue warps with half the columns each lose (1.97 ms; 8192 x 8192 x
// 4096 285 us, with 8 warps 276), and so do four accumulators of 128 columns and
// MMAs half as wide (2.30 ms; 355).
//
// kGated8: 256 x 128 of either projection at a time, summed over several k-blocks
// in TMEM and then in registers, as the 8-bit forms do (see Cfg::LEAD): 1.22 ms.
//
// Every wait is bounded; on expiry the kernel records SHMM_ERR_TIMEOUT, drains
// its own loads and MMAs, frees TMEM and returns.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

#include "checked.cuh"
#include "contract_tc.cuh"
#include "device_wait.cuh"
#include "e4m3.cuh"
#include "gated_act.cuh"
#include "pair.cuh"
#include "pdl.cuh"
#include "shmm_internal.h"
#include "tensor_map.h"

namespace {

using namespace shmm_dev;
using namespace shmm_pair;
using namespace shmm_tcn;

constexpr int kStagingBytes = 32 * 1024;  // epilogue boxes, 4 KB per warp
// Warps 0-3: TMA, MMA, and for the 8-bit forms a second MMA issuer and one that
// fetches the scales; warps 4-11: the epilogue.
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
// 8-bit forms: registers that the first warpgroup hands to the other two, whose
// threads hold 128 sums each.  A launch gives every thread 168 (65536 / 384,
// rounded down to a multiple of 8): 128 * 72 + 256 * 216 = 384 * 168.
constexpr int kFewRegs = 72, kManyRegs = 216;
static_assert(128 * kFewRegs + 256 * kManyRegs <= kThreads * 168, "no more registers than the launch has");
// 8-bit forms: k-blocks whose scales wait in shared memory (1 KB each: the
// product of the row's and the 128 columns' scale, for both column halves).
constexpr int kScaleSlots = 8;

template <int FORM>
struct Cfg {
    static constexpr bool F8 = FORM == kNN8 || FORM == kNT8;
    static constexpr bool X_MN = FORM == kTN;                                       // X stored [Kd, M]
    static constexpr bool GATED = FORM == kGated || FORM == kGated8;
    static constexpr bool Y_MN = GATED || FORM == kTN || FORM == kNN8;              // Y stored [Kd, N]
    static constexpr bool REGS = F8 || FORM == kGated8;  // long sums in registers
    // k-blocks of an accumulator, with REGS: of a tile's first two, and of the others.
    // The first two are filled while the epilogue still works on the last tile.
    // (kGated8, 8192 x 4096 x 16384: 1282 us with runs of 4, 1186 of 8, 1105 of 16;
    // what is kept then differs from the 64-bit form by 1.1e-4, 2.0e-4 and 2.7 to
    // 3.6e-4, with fp32 products by 1.4 to 2.5e-4.)
    static constexpr int LEAD = F8 ? 1 : 8, RUN = F8 ? 1 : 4;
    static __device__ __forceinline__ int run(int r, int left) {
        const int n = r < 2 ? LEAD : RUN;
        return left < n ? left : n;
    }
    static constexpr int ISSUERS = F8 ? 2 : 1;
    static constexpr int NH = REGS ? 1 : 2;    // 256-column halves of a tile
    static constexpr int BK = F8 ? 128 : 64;   // values of a k-block: 128 bytes
    static constexpr int BOX = 16384;          // 128 rows or columns of a k-block
    static constexpr int STAGE = BOX * (1 + NH);
    static constexpr int S = REGS ? 5 : 4;
    static constexpr int SMEM = S * STAGE + kStagingBytes + (REGS ? kScaleSlots * 1024 : 0) + 1024 /*align*/ + 1024 /*barriers*/;
};

// MMA of the pair: M = 256, N = 256, fp32 accumulator.
template <int FORM>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, bool add) {
    using C = Cfg<FORM>;
    constexpr uint32_t idesc = (1u << 4) | (C::F8 ? 0u : (1u << 7) | (1u << 10)) | (C::X_MN ? 1u << 15 : 0u) |
                               (C::Y_MN ? 1u << 16 : 0u) | ((256u >> 3) << 17) | ((256u >> 4) << 24);
    if (C::F8) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
    }
}

// Work item t -> its tile, and *hh: the 256-column half that a half-tile item
// covers, or -1.  Tiles run in bands of 8 m-tiles, m fastest, so the pairs at
// work at one time cover a roughly square part of the result.
__device__ __forceinline__ void item_coords(const ContractK &k, int t, int *mt, int *nt, int *hh) {
    *hh = -1;
    if (t >= k.half_from) {
        const int i = t - k.half_from;
        *hh = i & 1;
        t = k.half_from + (i >> 1);
    }
    constexpr int kBand = 8;
    const int band = t / (kBand * k.n_tiles);
    const int m0 = band * kBand;
    const int bm = k.m_tiles - m0 < kBand ? k.m_tiles - m0 : kBand;
    const int q = t - band * kBand * k.n_tiles;
    *mt = m0 + q % bm;
    *nt = q / bm;
}

// First result column of half h of the n-tile.
template <int FORM>
__device__ __forceinline__ int half_col(const ContractK &k, int nt, int h) {
    if (FORM == kGated) return nt * 256 + h * 128;
    if (FORM == kGated8) return nt * 128;
    if (Cfg<FORM>::F8 || k.two) return nt * 256;
    return nt * 512 + h * 256;
}

// The epilogue's view of a finished 32 x 32 box of bf16 or fp32 values, or of a
// 32 x 64 box of bytes: staged in the warp's next shared-memory box and stored
// to every holder.
struct Stager {
    const ContractK *k;
    uint32_t buf;    // the warp's 4 KB
    uint32_t boxes;  // handed to the copy engine
    int lane;

    __device__ __forceinline__ uint32_t next(uint32_t box_bytes) {
        const uint32_t n = 4096u / box_bytes;
        const uint32_t at = buf + (boxes % n) * box_bytes;
        if (lane == 0) bulk_wait_read((int)n - 1);  // the store n boxes back has read this box
        __syncwarp();
        ++boxes;
        return at;
    }
    __device__ __forceinline__ void send(const ResK &d, int map0, uint32_t at, int row0, int col0) {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            int32_t r, c;
            const int p = block_of(d, row0, col0, &r, &c);
            for (int q = d.first[p]; q < d.first[p + 1]; ++q) tma_store_2d(&k->maps[map0 + q], at, c, r);
            bulk_commit();
        }
    }
    __device__ __forceinline__ void bf16(const ResK &d, int map0, const float *v, int row0, int col0) {
        const uint32_t at = next(2048);
        stage_bf16_row(at, lane, v);
        send(d, map0, at, row0, col0);
    }
    __device__ __forceinline__ void f32(const ResK &d, int map0, const float *v, int row0, int col0) {
        const uint32_t at = next(4096);
        stage_f32_row(at, lane, v);
        send(d, map0, at, row0, col0);
    }
    // 64 values times inv as e4m3; `finite`: no infinity among them
    __device__ __forceinline__ void bytes(const ResK &d, int map0, const float *v, float inv, bool finite, int row0, int col0) {
        const uint32_t at = next(2048);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float *x = v + 16 * j + 4 * i;
                w[i] = finite_to_e4m3x2(x[0] * inv, x[1] * inv) | finite_to_e4m3x2(x[2] * inv, x[3] * inv) << 16;
                if (!finite) w[i] = to_e4m3x2(x[0] * inv, x[1] * inv) | to_e4m3x2(x[2] * inv, x[3] * inv) << 16;
            }
            st_shared_v4(at + (uint32_t)(lane * 64 + ((j ^ ((lane >> 1) & 3)) * 16)), w);
        }
        send(d, map0, at, row0, col0);
    }
};

// act(g) * u of one warp's 32 rows and 64 columns from c0.
template <int ACT>
__device__ __forceinline__ void store_product(const ContractK &k, Stager &st, const float *g, const float *u, int row0, int c0) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (c0 + c * 32 >= k.N) break;
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = gate_act<ACT>(g[c * 32 + i]) * u[c * 32 + i];
        st.bf16(k.D[0], k.D[0].map0, v, row0, c0 + c * 32);
    }
}

// What the two warps of a lane quadrant tell each other of their rows: two
// exponents per row, in turn in two places.  A warp writes a place again only
// after the other has arrived at the next exchange, having read this one.
constexpr int kNoValue = -127;  // a block of zeros, below every exponent
struct Exchange {
    volatile int16_t *at;  // [2][2 warps][32 rows]
    uint32_t bar;          // both warps arrive
    uint32_t turn;
    volatile int *abort_flag;
    int *status;
    __device__ __forceinline__ void give(int set, const int *e, int lane) {
        at[((turn & 1) * 2 + set) * 32 + lane] = (int16_t)((e[0] & 0xFF) | (e[1] << 8));
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);  // releases the warp's writes
    }
    // The larger ones; false: the wait ran out.
    __device__ __forceinline__ bool take(int set, int *e, int lane) {
        int ok = 1;
        if (lane == 0) ok = mbar_wait(bar, turn & 1, abort_flag, status) ? 1 : 0;
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        const int o = at[((turn & 1) * 2 + (set ^ 1)) * 32 + lane];
        e[0] = max(e[0], (int)(int8_t)(o & 0xFF));
        e[1] = max(e[1], o >> 8);
        ++turn;
        return ok != 0;
    }
};

// A finished tile whose pre-activations are kept in 8 bits: this warp's 64 of a
// block's 128 columns, the scales from both warps.
template <int ACT>
__device__ __forceinline__ bool store_kept8(const ContractK &k, Stager &st, Exchange &ex, const float *g, const float *u, int set,
                                            int row0, int col, int lane) {
    const int c0 = col + set * 64;
    bool finite = true;
    int e[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const float *v = y ? u : g;
        float m = 0.0f;  // fmaxf leaves NaN out
#pragma unroll
        for (int i = 0; i < 64; ++i) m = fmaxf(m, fabsf(v[i]));
        const bool inf = m == INFINITY;
        finite = finite && !inf;
        if (__any_sync(0xFFFFFFFFu, inf)) {  // the largest finite one, then
            m = 0.0f;
#pragma unroll
            for (int i = 0; i < 64; ++i) m = fmaxf(m, finite_abs(v[i]));
        }
        e[y] = m == 0.0f ? kNoValue : scale_exp(m);
    }
    ex.give(set, e, lane);
    store_product<ACT>(k, st, g, u, row0, c0);
    if (!ex.take(set, e, lane)) return false;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int ey = e[y] == kNoValue ? 0 : e[y];
        if (c0 < k.N) st.bytes(k.D[0], k.kept_map[y], y ? u : g, pow2(-ey), finite, row0, c0);
        if (y == set && row0 + lane < k.M) {  // one of the two warps writes the gate's scales, the other the up's
            int32_t rl, cl;
            const int p = block_of(k.D[0], row0 + lane, col, &rl, &cl);
            const int64_t at = (int64_t)rl * k.kept_ld + cl / 128;
            if (in_bounds(k.status, at, 1, k.D[0].brows * k.kept_ld))
                for (int q = k.D[0].first[p]; q < k.D[0].first[p + 1]; ++q) k.kept_scale[y][q][at] = pow2(ey);
        }
    }
    return true;
}

// One half of a finished tile of a form that sums in TMEM, for one epilogue warp:
// the half's accumulator (256 columns from `acc`) into registers, `release`,
// then the rest.  The two warps of a lane quadrant (set 0 and 1) share the
// columns.
template <int FORM, int ACT, typename Release>
__device__ __forceinline__ void finish_half(const ContractK &k, Stager &st, uint32_t acc, int set, int row0, int col,
                                            int h, Release release) {
    const bool rows_in = row0 < k.M;
    if (FORM == kGated) {
        uint32_t r[2][64];
#pragma unroll
        for (int y = 0; y < 2; ++y) tmem_read64(acc + (uint32_t)(y * 128 + set * 64), r[y]);
        release();
        if (!rows_in || col >= k.N) return;
        const float *g = reinterpret_cast<float *>(r[0]), *u = reinterpret_cast<float *>(r[1]);
        const int c0 = col + set * 64;
        if (k.keep) {
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (c0 + c * 32 < k.N) st.bf16(k.D[0], k.kept_map[y], (y ? u : g) + c * 32, row0, c0 + c * 32);
        }
        store_product<ACT>(k, st, g, u, row0, c0);
    } else {
        uint32_t r[128];
        tmem_read64(acc + (uint32_t)(set * 128), r);
        tmem_read64(acc + (uint32_t)(set * 128 + 64), r + 64);
        release();
        if (!rows_in) return;
        const ResK &d = k.D[k.two ? h : 0];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int c0 = col + set * 128 + c * 32;
            if (c0 >= k.N) break;
            st.bf16(d, d.map0, reinterpret_cast<float *>(r) + c * 32, row0, c0);
        }
    }
}

template <int FORM, int ACT>
__global__ void __launch_bounds__(kThreads, 1) contract_pair_kernel(const __grid_constant__ ContractK k) {
    using C = Cfg<FORM>;
    constexpr int S = C::S, NH = C::NH;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *tiles = smem;
    uint8_t *staging = smem + S * C::STAGE;
    // 8-bit forms: scales [kScaleSlots][2][128]; kGated8: what pairs of epilogue warps exchange, 256 bytes a pair
    float *scales = reinterpret_cast<float *>(staging + kStagingBytes);
    uint64_t *bars = reinterpret_cast<uint64_t *>(staging + kStagingBytes + (C::REGS ? kScaleSlots * 1024 : 0));
    // bars: full[S], empty[S], acc_full[2], acc_empty[2], drain, hand-off, scales_full[] (kGated8: exchanges), scales_empty[]
    uint32_t *words = reinterpret_cast<uint32_t *>(bars + 2 * S + 6 + 2 * kScaleSlots);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(words + 1);
    volatile uint32_t *peer_issued = words + 2;  // the peer's load count, and its bytes of each of its last S stages
    volatile uint32_t *peer_bytes = words + 4;
    static_assert((2 * S + 6 + 2 * kScaleSlots) * 8 + (4 + S) * 4 <= 1024, "barriers and words");

    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;  // warp: known to be uniform
    const uint32_t cr = cluster_ctarank();  // 0: leader, 1: peer
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    auto full_bar = [&](int s) { return smem_u32(&bars[s]); };
    auto empty_bar = [&](int s) { return smem_u32(&bars[S + s]); };
    auto accf_bar = [&](int s) { return smem_u32(&bars[2 * S + s]); };
    auto acce_bar = [&](int s) { return smem_u32(&bars[2 * S + 2 + s]); };
    const uint32_t drain_bar = smem_u32(&bars[2 * S + 4]), handoff_bar = smem_u32(&bars[2 * S + 5]);
    auto scalesf_bar = [&](int s) { return smem_u32(&bars[2 * S + 6 + s]); };
    auto scalese_bar = [&](int s) { return smem_u32(&bars[2 * S + 6 + kScaleSlots + s]); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(accf_bar(s), 1);
            mbar_init(acce_bar(s), 2 * kEpiWarps);  // both CTAs' epilogue warps
        }
        for (int s = 0; s < kScaleSlots; ++s) {
            mbar_init(scalesf_bar(s), C::F8 ? 1 : 2);  // the warp that fetches them; an exchange's two warps
            mbar_init(scalese_bar(s), kEpiWarps);
        }
        mbar_init(drain_bar, C::ISSUERS);
        mbar_init(handoff_bar, 1);
        *abort_flag = 0;
        *peer_issued = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(words)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers exist before any remote use
    fence_after();
    const uint32_t tmem_base = *words;
    // The prologue above touches no global memory: it may overlap the end of
    // the kernel before in the stream.
    shmm_pdl::pdl_enter(k.beside);

    if (warp < 4) {
        if constexpr (C::REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if (warp == 0) {
            // ---------------- TMA producer (both CTAs) ----------------
            const bool chosen = elect_one();
            uint32_t it = 0;  // stages loaded
            uint32_t stage_bytes[S];
            // One warp feeds the pair: what its loop computes is time between loads.
            const uint32_t full0 = full_bar(0), empty0 = empty_bar(0), leader_full0 = mapa_shared(full0, 0);
            const uint32_t tiles0 = smem_u32(tiles);
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (int t = pair; t < k.total && ok; t += npairs) {
                int mt, nt, hh;
                item_coords(k, t, &mt, &nt, &hh);
                const int nh = hh >= 0 ? 1 : NH;
                const uint32_t bytes = (uint32_t)(C::BOX * (1 + nh));
                for (int term = 0; term < k.terms && ok; ++term) {
                    Cursor x, y[NH];
                    x.template start<!C::X_MN>(k.maps, k.X[term], (int64_t)mt * 256 + (int)cr * 128);
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        const int hc = half_col<FORM>(k, nt, hh >= 0 ? hh : h);
                        if (C::GATED) y[h].template start<!C::Y_MN>(k.maps, k.Y[cr], hc);
                        else y[h].template start<!C::Y_MN>(k.maps, k.Y[k.two ? (hh >= 0 ? hh : h) : term], hc + (int)cr * 128);
                    }
                    for (int kb = 0; kb < k.k_blocks; ++kb, ++it) {
                        if (!warp_wait(empty0 + stage * 8, phase ^ 1, abort_flag, k.status)) {
                            ok = false;
                            break;
                        }
                        stage_bytes[stage] = bytes;
                        const uint32_t bar = leader_full0 + stage * 8, dst = tiles0 + stage * C::STAGE;
                        if (chosen) {
                            if (cr == 0) mbar_expect_tx(full0 + stage * 8, 2 * bytes);
                            load_box<C::X_MN, C::F8>(x, dst, bar);
#pragma unroll
                            for (int h = 0; h < NH; ++h)
                                if (h < nh) load_box<C::Y_MN, C::F8>(y[h], dst + (uint32_t)(C::BOX * (1 + h)), bar);
                        }
                        __syncwarp();
                        x.advance(C::BK);
#pragma unroll
                        for (int h = 0; h < NH; ++h) y[h].advance(C::BK);
                        if (++stage == (uint32_t)S) stage = 0, phase ^= 1;
                    }
                }
            }
            // Both CTAs' loads of a stage complete on the leader's barrier, so the
            // leader waits for all of them; the peer hands over how many stages
            // it loaded, and their bytes.  After an abort the counts may differ by
            // up to S stages: the leader arms the peer's extra stages for the
            // peer's half, and stands in for the half the peer never loaded.
            if (chosen && cr == 1) {
                for (int s = 0; s < S; ++s)
                    if ((uint32_t)s < it) st_cluster_u32(mapa_shared(smem_u32((const void *)(peer_bytes + s)), 0), stage_bytes[s]);
                st_cluster_u32(mapa_shared(smem_u32((const void *)peer_issued), 0), it);
                mbar_arrive_cluster(mapa_shared(handoff_bar, 0));
            } else if (chosen) {
                uint32_t it_peer = it;
                if (mbar_wait_cluster(handoff_bar, 0, k.status)) it_peer = *peer_issued;
                const uint32_t it_max = it_peer > it ? it_peer : it;
                for (uint32_t i = it_peer < it ? it_peer : it; i < it_max; ++i) {
                    const int s = (int)(i % S);
                    if (i >= it) mbar_expect_tx(full_bar(s), peer_bytes[s]);  // the peer's half only
                    else mbar_complete_tx(full_bar(s), stage_bytes[s]);       // the half never loaded
                }
                for (uint32_t i = it_max > (uint32_t)S ? it_max - S : 0; i < it_max; ++i)
                    mbar_wait(full_bar((int)(i % S)), (i / S) & 1, abort_flag, k.status, false);
            }
        } else if (C::REGS && warp <= C::ISSUERS) {
            // ---------------- MMA issuers (leader CTA only) ----------------
            // 8-bit forms: warp 1 fills the even accumulator, warp 2 the odd one; one
            // thread's waits and commits for one would hold up the other's MMAs (1.86
            // ms with one issuer, 1.84 with two).  A stage's barrier tells only the
            // last two fills apart, so nobody may wait for one before the fill before
            // it (S k-blocks back) is complete: with a k-block to an accumulator that
            // one belongs to an accumulator that the epilogue has handed back before.
            // With four it may be the other issuer's present one, so there is one
            // issuer, which takes all in order.
            if (cr == 0) {
                const bool chosen = elect_one();
                const uint32_t mine = pair < k.total ? (uint32_t)((k.total - 1 - pair) / npairs + 1) : 0;  // tiles
                // Descriptors hold addresses in units of 16 bytes.
                const uint64_t a0 = operand_step<C::X_MN, C::F8>(smem_u32(tiles), 0);
                const uint64_t b0 = operand_step<C::Y_MN, C::F8>(smem_u32(tiles) + C::BOX, 0);
                constexpr uint32_t A_STEP = 2, B_STEP = !C::Y_MN ? 2 : C::F8 ? 256 : 128;
                uint32_t stage = 0, phase = 0, it = 0;  // `it`: accumulators filled so far
                bool ok = true;
                for (uint32_t t = 0; t < mine && ok; ++t) {
                    int n = 0;
                    for (int r = 0, kb0 = 0; kb0 < k.k_blocks && ok; ++r, kb0 += n, ++it) {
                        n = C::run(r, k.k_blocks - kb0);
                        const int buf = (int)(it & 1);
                        if (C::ISSUERS == 1 || buf == warp - 1) {
                            const uint32_t d = tmem_base + (uint32_t)(buf * 256);
                            if (!warp_wait(acce_bar(buf), ((it >> 1) & 1) ^ 1, abort_flag, k.status)) {
                                ok = false;
                                break;
                            }
                            uint32_t s = stage, p = phase;
                            for (int kb = 0; kb < n; ++kb) {
                                if (!warp_wait(full_bar((int)s), p, abort_flag, k.status)) {
                                    ok = false;
                                    break;
                                }
                                fence_after();
                                const uint64_t a = a0 + s * (C::STAGE / 16), b = b0 + s * (C::STAGE / 16);
                                if (chosen) {
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk)
                                        pair_mma<FORM>(d, a + kk * A_STEP, b + kk * B_STEP, kb > 0 || kk > 0);
                                    if (kb == n - 1) umma2_commit_both(accf_bar(buf));
                                    umma2_commit_both(empty_bar((int)s));
                                }
                                __syncwarp();
                                if (++s == (uint32_t)S) s = 0, p ^= 1;
                            }
                        }
                        for (stage += (uint32_t)n; stage >= (uint32_t)S; stage -= S) phase ^= 1;
                    }
                }
                if (chosen) {
                    umma2_commit_both(drain_bar);
                    mbar_wait(drain_bar, 0, abort_flag, k.status, false);
                }
                __syncwarp();
            }
        } else if (!C::REGS && warp == 1) {
            // ---------------- MMA issuer (leader CTA only) ----------------
            if (cr == 0) {
                const bool chosen = elect_one();
                const int k_total = k.terms * k.k_blocks;
                uint32_t it = 0, fills0 = 0, fills1 = 0;
                bool ok = true;
                const uint64_t a0 = operand_step<C::X_MN, false>(smem_u32(tiles), 0);
                const uint64_t b0 = operand_step<C::Y_MN, false>(smem_u32(tiles) + C::BOX, 0);
                constexpr uint32_t A_STEP = C::X_MN ? 128 : 2, B_STEP = C::Y_MN ? 128 : 2;
                // The four MMAs of the k-block in stage s, half h of its Y, into buffer
                // h; `done`: and the stage may be filled again.
                auto issue = [&](uint32_t s, int h, bool first, bool done) {
                    const uint64_t a = a0 + s * (C::STAGE / 16), b = b0 + s * (C::STAGE / 16) + (uint32_t)(h * (C::BOX / 16));
                    if (chosen) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            pair_mma<FORM>(tmem_base + (uint32_t)(h * 256), a + kk * A_STEP, b + kk * B_STEP, !first || kk > 0);
                        if (done) umma2_commit_both(empty_bar((int)s));
                    }
                    __syncwarp();
                };
                auto wait_free = [&](int buf, uint32_t fills) -> bool {
                    if (!warp_wait(acce_bar(buf), (fills & 1) ^ 1, abort_flag, k.status)) return false;
                    fence_after();
                    return true;
                };
                auto wait_stage = [&](uint32_t i) -> bool {
                    if (!warp_wait(full_bar((int)(i % S)), (i / S) & 1, abort_flag, k.status)) return false;
                    fence_after();
                    return true;
                };
                for (int t = pair; t < k.total && ok; t += npairs) {
                    // Half 0 runs ahead over the first R loaded stages while the
                    // epilogue still reads half 1 of the previous tile, then half 1
                    // catches up on the same stages.
                    const bool half = t >= k.half_from;
                    const int R = k_total < S ? k_total : S;
                    if (!wait_free(0, fills0)) break;
                    for (int kb = 0; kb < R; ++kb) {
                        if (!wait_stage(it + (uint32_t)kb)) {
                            ok = false;
                            break;
                        }
                        issue((it + (uint32_t)kb) % S, 0, kb == 0, half);
                    }
                    if (!ok) break;
                    if (!half) {
                        if (!wait_free(1, fills1)) break;
                        for (int kb = 0; kb < R; ++kb) issue((it + (uint32_t)kb) % S, NH - 1, kb == 0, true);
                    }
                    it += (uint32_t)R;
                    for (int kb = R; kb < k_total; ++kb, ++it) {
                        if (!wait_stage(it)) {
                            ok = false;
                            break;
                        }
                        issue(it % S, 0, false, half);
                        if (!half) issue(it % S, NH - 1, false, true);
                    }
                    if (!ok) break;
                    if (chosen) {
                        umma2_commit_both(accf_bar(0));
                        if (!half) umma2_commit_both(accf_bar(1));
                    }
                    __syncwarp();
                    ++fills0;
                    if (!half) ++fills1;
                }
                if (chosen) {
                    umma2_commit_both(drain_bar);
                    mbar_wait(drain_bar, 0, abort_flag, k.status, false);
                }
                __syncwarp();
            }
        } else if constexpr (C::F8) {
            // ---------------- scales (both CTAs): a lane has rows lane + 0, 32, 64, 96 ----------------
            if (warp == 3) {
                uint32_t it = 0;
                bool ok = true;
                for (int t = pair; t < k.total && ok; t += npairs) {
                    int mt, nt, hh;
                    item_coords(k, t, &mt, &nt, &hh);
                    const int row = mt * 256 + (int)cr * 128 + lane, col = nt * 256;
                    ScaleCursor x, y;  // the rows of a tile are in one block, and its columns in one or two
                    x.template start<true>(k.X[0], k.x_scale, mt * 256 + (int)cr * 128, 1, true);
                    int64_t at[4];
                    bool in[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        in[q] = row + 32 * q < k.M;
                        at[q] = (int64_t)(lane + 32 * q) * k.x_scale.ld;
                    }
                    // lanes 0-15 fetch the first 128 columns' scale, the others the second's
                    const int yc = col + (lane / 16) * 128;
                    y.template start<!C::Y_MN>(k.Y[0], k.y_scale, yc, 128, yc < k.N);
                    for (int kb = 0; kb < k.k_blocks; ++kb, ++it) {
                        const int s = it % kScaleSlots;
                        float v[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) v[q] = in[q] ? x.peek(at[q], k.status) : 0.0f;
                        x.step_on();
                        const float w = y.next(k.status);
                        const float w0 = __shfl_sync(0xFFFFFFFFu, w, 0), w1 = __shfl_sync(0xFFFFFFFFu, w, 16);
                        ok = mbar_wait(scalese_bar(s), ((it / kScaleSlots) & 1) ^ 1, abort_flag, k.status);
                        if (!__all_sync(0xFFFFFFFFu, ok)) {
                            ok = false;
                            break;
                        }
                        float *to = scales + s * 256 + lane;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            to[32 * q] = v[q] * w0;
                            to[128 + 32 * q] = v[q] * w1;
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(scalesf_bar(s));  // releases the warp's stores, which the sync orders before it
                    }
                }
            }
        }
    } else {
        // ---------------- epilogue (both CTAs) ----------------
        if constexpr (C::REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        const int ew = warp - 4, quad = warp % 4, set = ew / 4;
        const uint32_t lanes = tmem_base + ((uint32_t)(quad * 32) << 16);
        Stager st = {&k, smem_u32(staging) + (uint32_t)ew * 4096u, 0, lane};
        Exchange ex = {reinterpret_cast<volatile int16_t *>(scales) + quad * 128, scalesf_bar(quad), 0, abort_flag, k.status};
        uint32_t used[2] = {0, 0};
        auto wait_full = [&](int b) -> bool {
            int ok = 1;
            if (lane == 0) ok = mbar_wait(accf_bar(b), used[b] & 1, abort_flag, k.status) ? 1 : 0;
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            ++used[b];
            if (ok) fence_after();
            return ok != 0;
        };
        auto release = [&](int b) {
            fence_before();
            __syncwarp();
            if (lane == 31) mbar_arrive_cluster_relaxed(mapa_shared(acce_bar(b), 0));  // the leader's barrier
        };
        bool ok = true;
        uint32_t fill = 0;
        for (int t = pair; t < k.total && ok; t += npairs) {
            int mt, nt, hh;
            item_coords(k, t, &mt, &nt, &hh);
            const int row0 = mt * 256 + (int)cr * 128 + quad * 32;
            if constexpr (!C::REGS) {
                const int nh = hh >= 0 ? 1 : NH;
                for (int h = 0; h < nh; ++h) {
                    if (!wait_full(h)) {
                        ok = false;
                        break;
                    }
                    const int half = hh >= 0 ? hh : h;
                    finish_half<FORM, ACT>(k, st, lanes + (uint32_t)(h * 256), set, row0, half_col<FORM>(k, nt, half), half,
                                           [&] { release(h); });
                }
            } else {
                const int col0 = C::F8 ? nt * 256 + set * 128 : nt * 128;
                // the warp's columns: 128 in a row, or 64 of the gate and the same 64 of the up projection
                const uint32_t first = C::F8 ? set * 128 : set * 64, second = C::F8 ? first + 64 : first + 128;
                float acc[128];
#pragma unroll
                for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
                for (int kb = 0, run = 0; kb < k.k_blocks; kb += C::run(run, k.k_blocks), ++run, ++fill) {
                    const int b = fill & 1, s = fill % kScaleSlots;
                    int got = 1;
                    if (lane == 0)
                        got = (!C::F8 || mbar_wait(scalesf_bar(s), (fill / kScaleSlots) & 1, abort_flag, k.status)) &&
                              mbar_wait(accf_bar(b), (fill >> 1) & 1, abort_flag, k.status);
                    if (!__shfl_sync(0xFFFFFFFFu, got, 0)) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const uint32_t at = lanes + (uint32_t)(b * 256);
                    const float sc =
                        C::F8 ? reinterpret_cast<volatile float *>(scales)[s * 256 + set * 128 + quad * 32 + lane] : 1.0f;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t r[64];
                        tmem_read64(at + (c ? second : first), r);
                        if (c == 1) {
                            release(b);
                            if (C::F8 && lane == 0) mbar_arrive(scalese_bar(s));
                        }
#pragma unroll
                        for (int j = 0; j < 64; ++j) acc[c * 64 + j] = fmaf(__uint_as_float(r[j]), sc, acc[c * 64 + j]);
                    }
                }
                if (!ok) break;
                if (row0 >= k.M) continue;
                if constexpr (FORM == kGated8) {
                    ok = store_kept8<ACT>(k, st, ex, acc, acc + 64, set, row0, col0, lane);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int c0 = col0 + c * 32;
                        if (c0 >= k.N) break;
                        if (k.out_f32) st.f32(k.D[0], k.D[0].map0, acc + c * 32, row0, c0);
                        else st.bf16(k.D[0], k.D[0].map0, acc + c * 32, row0, c0);
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_all();  // no store still reads staging at exit
        __syncwarp();
    }

    fence_before();
    __syncthreads();
    cluster_sync_all();  // no CTA leaves while its peer may still signal it
    fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem_base) : "memory");
    shmm_pdl::pdl_end(k.beside);
}

// ---- host side --------------------------------------------------------------

// CTA pairs that can be resident at once (one CTA per SM).  Sets the kernel's
// shared-memory attribute on first use per device.
template <int FORM, int ACT>
cudaError_t pair_capacity(int *pairs) {
    using C = Cfg<FORM>;
    static std::mutex mu;
    static int cap[shmm::kMaxDevices] = {};  // + 1
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= shmm::kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!cap[dev]) {
        e = cudaFuncSetAttribute(contract_pair_kernel<FORM, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        int sms = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t q = {};
        cudaLaunchAttribute qa[1];
        qa[0].id = cudaLaunchAttributeClusterDimension;
        qa[0].val.clusterDim.x = 2;
        qa[0].val.clusterDim.y = 1;
        qa[0].val.clusterDim.z = 1;
        q.gridDim = dim3((unsigned)(sms & ~1));
        q.blockDim = dim3(kThreads);
        q.dynamicSmemBytes = C::SMEM;
        q.attrs = qa;
        q.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, contract_pair_kernel<FORM, ACT>, &q);
        if (e != cudaSuccess) return e;
        cap[dev] = 1 + (n < 0 ? 0 : n);
    }
    *pairs = cap[dev] - 1;
    return cudaSuccess;
}

template <int FORM, int ACT>
int launch_form(ContractK &k, int max_sms, cudaStream_t s) {
    using C = Cfg<FORM>;
    int cap = 0;
    const cudaError_t e = pair_capacity<FORM, ACT>(&cap);
    if (e != cudaSuccess) return (int)e;
    if (cap < 1) return (int)cudaErrorNotSupported;
    if (max_sms > 0 && max_sms / 2 < cap) cap = max_sms / 2 > 0 ? max_sms / 2 : 1;
    const int width = FORM == kGated8 ? 128 : FORM == kGated || C::F8 || k.two ? 256 : 512;
    k.m_tiles = (int)((k.M + 255) / 256);
    k.n_tiles = (int)((k.N + width - 1) / width);
    k.k_blocks = (int)((k.Kd + C::BK - 1) / C::BK);
    k.total = k.half_from = k.m_tiles * k.n_tiles;
    if (!C::REGS) {
        // A last wave that would leave at least half of the pairs idle runs as
        // halves on twice as many.
        const int r = k.total % cap;
        if (r > 0 && 2 * r <= cap) {
            k.half_from = k.total - r;
            k.total += r;
        }
    }
    const int npairs = k.total < cap ? k.total : cap;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    const char *pdl = getenv("SHMM_PDL");
    cfg.gridDim = dim3((unsigned)(2 * npairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = (pdl && pdl[0] == '0') ? 1 : 2;
    shmm::count_launch();
    return (int)cudaLaunchKernelEx(&cfg, contract_pair_kernel<FORM, ACT>, k);
}

}  // namespace

namespace shmm_tcn {

int launch_pair(ContractK &k, int form, int max_sms, cudaStream_t s) {
    switch (form) {
        case kGated:
            return k.act == SHMM_SILU ? launch_form<kGated, SHMM_SILU>(k, max_sms, s)
                                      : launch_form<kGated, SHMM_GELU_TANH>(k, max_sms, s);
        case kGated8:
            return k.act == SHMM_SILU ? launch_form<kGated8, SHMM_SILU>(k, max_sms, s)
                                      : launch_form<kGated8, SHMM_GELU_TANH>(k, max_sms, s);
        case kNT: return launch_form<kNT, SHMM_SILU>(k, max_sms, s);
        case kTN: return launch_form<kTN, SHMM_SILU>(k, max_sms, s);
        case kNN8: return launch_form<kNN8, SHMM_SILU>(k, max_sms, s);
        default: return launch_form<kNT8, SHMM_SILU>(k, max_sms, s);
    }
}

}  // namespace shmm_tcn
