// The same five products as contract_pair.cu for few rows and small shapes: a
// decoding step, a fine-tuning step of a few hundred tokens.  There a 256-row,
// 512-column tile would leave most SMs idle, and what counts is how many SMs
// read the weights and how soon.
//
// A CTA computes 128 rows by 128 accumulator columns (the gated form: 64 of the
// gate and the same 64 of the up projection) over a part of the contracted dim;
// the CTAs of a cluster (1, 2, 4 or 8) have a part each of one tile, add their
// partial sums through distributed shared memory in the order of the parts, and
// store a share of the columns each.  One input gives one result, no workspace.
// With fewer than 128 rows a stage holds only those of X (whole groups of 8):
// the MMA reads 128 rows all the same, and what lies behind only reaches rows of
// the accumulator that nothing reads.
//
// bf16 forms: two CTAs per SM, one accumulator in TMEM over the whole part.
// 8-bit forms: one CTA per SM and four accumulators of a k-block each in turn,
// which the epilogue adds to sums in registers with the two scales, as in
// contract_pair.cu; four, because the way round one takes some 1000 cycles and a
// k-block's MMAs of this width 128.
//
// Bound by HBM for few rows, where each weight is read once: gated, 4 rows, 4096 x
// 2 x 16384 bf16 in 42 us (6.3 TB/s); 8 bits, 16 rows, 4096 x 16384 in 20 (128
// tiles on 152 SMs).  Above that by the latency of a launch, a tile's loads and the
// parts' join.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <string>

#include "checked.cuh"
#include "contract_tc.cuh"
#include "device_wait.cuh"
#include "gated_act.cuh"
#include "pair.cuh"
#include "pdl.cuh"
#include "shmm_internal.h"

namespace {

using namespace shmm_dev;
using namespace shmm_pair;
using namespace shmm_tcn;

constexpr int kPitch = 132;  // floats of a partial sums' row: a row per thread, 16-byte pieces, no bank twice
constexpr int kScaleSlots = 8;

template <int FORM>
struct Cfg {
    static constexpr bool F8 = FORM == kNN8 || FORM == kNT8;
    static constexpr bool X_MN = FORM == kTN;
    static constexpr bool Y_MN = FORM == kGated || FORM == kTN || FORM == kNN8;
    static constexpr int BK = F8 ? 128 : 64;
    static constexpr int BUFS = F8 ? 4 : 1;       // accumulators
    static constexpr int SETS = F8 ? 2 : 1;       // epilogue warpgroups, sharing the columns
    static constexpr int WIDTH = FORM == kGated ? 64 : 128;  // result columns of a tile
    static constexpr int THREADS = 128 + 128 * SETS;
    static constexpr int CTAS = F8 ? 1 : 2;       // per SM
    static constexpr int RING = F8 ? 192 * 1024 : 100 * 1024;
    static constexpr int FIXED = (F8 ? kScaleSlots * 512 : 0) + 1024 /*barriers*/ + 1024 /*align*/;
    static constexpr int MAX_STAGES = 10;
};
static_assert(128 * kPitch * 4 <= 96 * 1024, "the partial sums fit where three whole stages were");

template <int FORM>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, bool add) {
    using C = Cfg<FORM>;
    constexpr uint32_t idesc = (1u << 4) | (C::F8 ? 0u : (1u << 7) | (1u << 10)) | (C::X_MN ? 1u << 15 : 0u) |
                               (C::Y_MN ? 1u << 16 : 0u) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
    if (C::F8) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
    }
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ void add4(float4 &a, const float4 &b) {
    a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
}

// Four values of global row `row`, columns col .. col + 3, to every holder.
__device__ __forceinline__ void put4(const ContractK &k, const ResK &d, void *const *out, int row, int col, bool f32,
                                     const float4 &v) {
    int32_t r, c;
    const int p = block_of(d, row, col, &r, &c);
    const int64_t at = (int64_t)r * d.bcols + c;
    if (!in_bounds(k.status, at, 4, d.brows * d.bcols)) return;
    for (int q = d.first[p]; q < d.first[p + 1]; ++q) {
        if (f32) {
            *reinterpret_cast<float4 *>(static_cast<float *>(out[q]) + at) = v;
        } else {
            const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(out[q]) + at) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
        }
    }
}

template <int FORM, int ACT>
__global__ void __launch_bounds__(Cfg<FORM>::THREADS, Cfg<FORM>::CTAS)
    contract_small_kernel(const __grid_constant__ ContractK k) {
    using C = Cfg<FORM>;
    constexpr int MS = C::MAX_STAGES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *tiles = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *scales = reinterpret_cast<float *>(tiles + k.ring_bytes);  // [kScaleSlots][128]
    uint64_t *bars = reinterpret_cast<uint64_t *>(tiles + k.ring_bytes + (C::F8 ? kScaleSlots * 512 : 0));
    // bars: full[MS], empty[MS], acc_full[4], acc_empty[4], scales_full[], scales_empty[], drain
    uint32_t *words = reinterpret_cast<uint32_t *>(bars + 2 * MS + 8 + 2 * kScaleSlots + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(words + 1);
    static_assert((2 * MS + 8 + 2 * kScaleSlots + 1) * 8 + 8 <= 1024, "barriers and words");

    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;  // warp: known to be uniform
    const int parts = k.parts, part = (int)cluster_ctarank(), S = k.stages;
    auto full_bar = [&](int s) { return smem_u32(&bars[s]); };
    auto empty_bar = [&](int s) { return smem_u32(&bars[MS + s]); };
    auto accf_bar = [&](int s) { return smem_u32(&bars[2 * MS + s]); };
    auto acce_bar = [&](int s) { return smem_u32(&bars[2 * MS + 4 + s]); };
    auto scalesf_bar = [&](int s) { return smem_u32(&bars[2 * MS + 8 + s]); };
    auto scalese_bar = [&](int s) { return smem_u32(&bars[2 * MS + 8 + kScaleSlots + s]); };
    const uint32_t drain_bar = smem_u32(&bars[2 * MS + 8 + 2 * kScaleSlots]);

    // The tile: m fastest, so CTAs that share columns of Y run together.
    const int tile = (int)blockIdx.x / parts;
    const int mt = tile % k.m_tiles;
    int nt = tile / k.m_tiles, which = 0;
    if (k.two && nt >= k.n_tiles) nt -= k.n_tiles, which = 1;
    const int row0 = mt * 128, col0 = nt * C::WIDTH;
    const int rows = k.M - row0 < 128 ? (int)(k.M - row0) : 128;
    // this CTA's k-blocks, of all terms
    const int all = k.terms * k.k_blocks;
    const int kb0 = (int)((int64_t)all * part / parts), kb1 = (int)((int64_t)all * (part + 1) / parts);

    const int active = (rows + 31) / 32;  // epilogue warps with rows
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int s = 0; s < C::BUFS; ++s) {
            mbar_init(accf_bar(s), 1);
            mbar_init(acce_bar(s), active * C::SETS);
        }
        for (int s = 0; s < kScaleSlots; ++s) {
            mbar_init(scalesf_bar(s), 1);
            mbar_init(scalese_bar(s), active * C::SETS);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    constexpr uint32_t kCols = 128 * C::BUFS;
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(words)), "r"(kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem_base = *words;
    shmm_pdl::pdl_enter(k.beside);

    const uint32_t x_bytes = (uint32_t)k.x_rows * 128;  // of a stage; the 16 KB of Y follow
    const uint32_t stage_bytes = x_bytes + 16384;
    bool ok = true;  // this thread's waits

    if (warp == 0) {
        // ---------------- TMA ----------------
        const bool chosen = elect_one();
        Cursor x, y[2];
        int term = kb0 / k.k_blocks, kb = kb0 % k.k_blocks;
        auto start = [&](int at) {
            if (term >= k.terms) return;
            x.template start<!C::X_MN>(k.maps, k.X[term], row0);
            x.seek(at * C::BK);
            if (FORM == kGated) {
                y[0].template start<false>(k.maps, k.Y[0], col0);
                y[1].template start<false>(k.maps, k.Y[1], col0);
                y[1].seek(at * C::BK);
            } else {
                y[0].template start<!C::Y_MN>(k.maps, k.Y[k.two ? which : term], col0);
            }
            y[0].seek(at * C::BK);
        };
        start(kb);
        const int n = kb1 - kb0;
        int it = 0;
        uint32_t stage = 0, phase = 0, dst = smem_u32(tiles);
        const uint32_t full0 = full_bar(0), empty0 = empty_bar(0);
        const uint32_t row_bytes = (uint32_t)k.X[0].brows * 128;
        for (; it < n; ++it) {
            if (!warp_wait(empty0 + stage * 8, phase ^ 1, abort_flag, k.status)) break;
            const uint32_t bar = full0 + stage * 8;
            const uint32_t to = dst + x_bytes;
            if (chosen) {
                mbar_expect_tx(bar, stage_bytes);
                if (C::X_MN) {
                    tma_load_2d(dst, x.map, bar, x.fixed, x.at);
                    tma_load_2d(dst + 8192, x.map, bar, x.fixed + 64, x.at);
                } else if (k.x_boxes == 1) {
                    tma_load_2d(dst, x.map, bar, x.at, x.fixed);
                } else {  // few rows, split over the ranks: a box from each
                    for (int b = 0; b < k.x_boxes; ++b)
                        tma_load_2d(dst + (uint32_t)b * row_bytes, x.map + b * k.X[0].b1, bar, x.at, 0);
                }
                if (FORM == kGated) {
                    tma_load_2d(to, y[0].map, bar, y[0].fixed, y[0].at);
                    tma_load_2d(to + 8192, y[1].map, bar, y[1].fixed, y[1].at);
                } else if (!C::Y_MN) {
                    tma_load_2d(to, y[0].map, bar, y[0].at, y[0].fixed);
                } else if (C::F8) {
                    tma_load_2d(to, y[0].map, bar, y[0].fixed, y[0].at);
                } else {
                    tma_load_2d(to, y[0].map, bar, y[0].fixed, y[0].at);
                    tma_load_2d(to + 8192, y[0].map, bar, y[0].fixed + 64, y[0].at);
                }
            }
            __syncwarp();
            x.advance(C::BK);
            y[0].advance(C::BK);
            if (FORM == kGated) y[1].advance(C::BK);
            dst += stage_bytes;
            if (++stage == (uint32_t)S) stage = 0, phase ^= 1, dst = smem_u32(tiles);
            if (++kb == k.k_blocks) {
                kb = 0;
                ++term;
                start(0);
            }
        }
        // never leave with a load in flight
        for (int i = it > S ? it - S : 0; chosen && i < it; ++i)
            mbar_wait(full_bar(i % S), (i / S) & 1, abort_flag, k.status, false);
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA ----------------
        const bool chosen = elect_one();
        const int n = kb1 - kb0;
        uint32_t stage = 0, phase = 0;
        // descriptors hold addresses in units of 16 bytes
        const uint64_t a0 = operand_step<C::X_MN, C::F8>(smem_u32(tiles), 0);
        const uint64_t b0 = operand_step<C::Y_MN, C::F8>(smem_u32(tiles) + x_bytes, 0);
        constexpr uint32_t A_STEP = C::X_MN ? 128 : 2, B_STEP = !C::Y_MN ? 2 : C::F8 ? 256 : 128;
        for (int it = 0; it < n; ++it) {
            const int buf = C::F8 ? it % C::BUFS : 0;
            if (!warp_wait(full_bar((int)stage), phase, abort_flag, k.status)) break;
            if (C::F8 && !warp_wait(acce_bar(buf), ((it / C::BUFS) & 1) ^ 1, abort_flag, k.status)) break;
            fence_after();
            const uint64_t a = a0 + stage * (stage_bytes / 16), b = b0 + stage * (stage_bytes / 16);
            if (chosen) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma<FORM>(tmem_base + (uint32_t)(buf * 128), a + kk * A_STEP, b + kk * B_STEP, kk > 0 || (!C::F8 && it > 0));
                if (C::F8) commit(accf_bar(buf));
                commit(empty_bar((int)stage));
            }
            __syncwarp();
            if (++stage == (uint32_t)S) stage = 0, phase ^= 1;
        }
        if (chosen) {
            if (!C::F8) commit(accf_bar(0));
            commit(drain_bar);
            mbar_wait(drain_bar, 0, abort_flag, k.status, false);
        }
        __syncwarp();
    } else if (C::F8 && warp == 2) {
        // ---------------- scales: a lane has rows lane + 0, 32, 64, 96 ----------------
        ScaleCursor x[4], y;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x[q].template start<true>(k.X[0], k.x_scale, row0 + lane + 32 * q, 1, row0 + lane + 32 * q < k.M);
            x[q].seek(kb0);
        }
        y.template start<!C::Y_MN>(k.Y[0], k.y_scale, col0, 128, true);
        y.seek(kb0);
        // Four k-blocks' scales at a time, the next four asked for before these are
        // waited for a place: one at a time, each k-block would take a read's latency.
        const int n = kb1 - kb0;
        float v[4][4], w[4], nv[4][4], nw[4];
        auto ask = [&](int it) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int q = 0; q < 4; ++q) nv[i][q] = it + i < n ? x[q].next(k.status) : 0.0f;
                nw[i] = it + i < n ? y.next(k.status) : 0.0f;
            }
        };
        ask(0);
        for (int it = 0; it < n && ok; it += 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = nw[i];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[i][q] = nv[i][q];
            }
            if (it + 4 < n) ask(it + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (it + i >= n) break;
                const int s = (it + i) % kScaleSlots;
                ok = mbar_wait(scalese_bar(s), (((it + i) / kScaleSlots) & 1) ^ 1, abort_flag, k.status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
#pragma unroll
                for (int q = 0; q < 4; ++q) scales[s * 128 + lane + 32 * q] = v[i][q] * w[i];
                __syncwarp();
                if (lane == 0) mbar_arrive(scalesf_bar(s));
            }
        }
    } else if (warp >= 4 && (warp % 4) < active) {
        // ---------------- partial sums into shared memory ----------------
        const int quad = warp % 4, set = (warp - 4) / 4, row = quad * 32 + lane;
        const uint32_t lanes = tmem_base + ((uint32_t)(quad * 32) << 16);
        float *to = reinterpret_cast<float *>(tiles) + row * kPitch;
        if constexpr (C::F8) {
            float acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0.0f;
            const int n = kb1 - kb0;
            for (int it = 0; it < n; ++it) {
                const int buf = it % C::BUFS, s = it % kScaleSlots;
                int got = 1;
                if (lane == 0)
                    got = mbar_wait(scalesf_bar(s), (it / kScaleSlots) & 1, abort_flag, k.status) &&
                          mbar_wait(accf_bar(buf), (it / C::BUFS) & 1, abort_flag, k.status);
                if (!__shfl_sync(0xFFFFFFFFu, got, 0)) {
                    ok = false;
                    break;
                }
                fence_after();
                const float sc = reinterpret_cast<volatile float *>(scales)[s * 128 + row];
                uint32_t r[64];
                tmem_read64(lanes + (uint32_t)(buf * 128 + set * 64), r);
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(acce_bar(buf));
                    mbar_arrive(scalese_bar(s));
                }
#pragma unroll
                for (int j = 0; j < 64; ++j) acc[j] = fmaf(__uint_as_float(r[j]), sc, acc[j]);
            }
            // The last accumulator is complete: every MMA has read its stage, and
            // the sums may lie where the stages were.  The other warps may still
            // read theirs from TMEM, not from there.
            if (ok) {
                to += set * 64;
#pragma unroll
                for (int j = 0; j < 64; j += 4)
                    *reinterpret_cast<float4 *>(to + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
            }
        } else {
            int got = 1;
            if (lane == 0) got = mbar_wait(accf_bar(0), 0, abort_flag, k.status);
            ok = __shfl_sync(0xFFFFFFFFu, got, 0);
            if (ok) {
                fence_after();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t r[64];
                    tmem_read64(lanes + (uint32_t)(c * 64), r);
#pragma unroll
                    for (int j = 0; j < 64; j += 4)
                        *reinterpret_cast<float4 *>(to + c * 64 + j) =
                            make_float4(__uint_as_float(r[j]), __uint_as_float(r[j + 1]), __uint_as_float(r[j + 2]),
                                        __uint_as_float(r[j + 3]));
                }
                fence_before();
            }
        }
    }

    // Every part's sums are where they belong; after a wait that ran out they are
    // not, the status says so, and what is stored is undefined.
    __syncthreads();
    cluster_sync_all();

    // This CTA's share of the tile's columns, the parts added in ascending order.
    {
        const int share = C::WIDTH / parts, groups = share / 4;
        const uint32_t base = smem_u32(tiles);
        uint32_t from[8];
        for (int q = 0; q < parts; ++q) from[q & 7] = mapa_shared(base, (uint32_t)q);
        for (int i = (int)threadIdx.x; i < rows * groups; i += C::THREADS) {
            const int r = i / groups, c = part * share + (i % groups) * 4;
            if (col0 + c >= k.N) continue;
            const uint32_t at = (uint32_t)((r * kPitch + c) * 4);
            float4 v = ld_cluster4(from[0] + at), u = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (FORM == kGated) u = ld_cluster4(from[0] + at + 64 * 4);
            for (int q = 1; q < parts; ++q) {
                add4(v, ld_cluster4(from[q & 7] + at));
                if (FORM == kGated) add4(u, ld_cluster4(from[q & 7] + at + 64 * 4));
            }
            if (FORM == kGated) {
                if (k.keep) {
                    put4(k, k.D[0], k.out[2], row0 + r, col0 + c, false, v);
                    put4(k, k.D[0], k.out[3], row0 + r, col0 + c, false, u);
                }
                v.x = gate_act<ACT>(v.x) * u.x;
                v.y = gate_act<ACT>(v.y) * u.y;
                v.z = gate_act<ACT>(v.z) * u.z;
                v.w = gate_act<ACT>(v.w) * u.w;
            }
            put4(k, k.D[which], k.out[which], row0 + r, col0 + c, k.out_f32, v);
        }
    }
    fence_before();
    cluster_sync_all();  // no CTA leaves while another reads its sums
    fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kCols) : "memory");
    shmm_pdl::pdl_end(k.beside);
}

// ---- host side --------------------------------------------------------------

template <int FORM, int ACT>
int launch_form(ContractK &k, int sms, cudaStream_t s) {
    using C = Cfg<FORM>;
    static shmm::PerDevice<int> attr_set;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return (int)e;
    if (dev < 0 || dev >= shmm::kMaxDevices) return (int)cudaErrorInvalidDevice;
    constexpr int kSmem = C::RING + C::FIXED;
    if (!attr_set.get(dev)) {
        e = cudaFuncSetAttribute(contract_small_kernel<FORM, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return (int)e;
        attr_set.set(dev, 1);
    }
    k.k_blocks = (int)((k.Kd + C::BK - 1) / C::BK);
    k.m_tiles = (int)((k.M + 127) / 128);
    k.n_tiles = (int)((k.N + C::WIDTH - 1) / C::WIDTH);
    const int stage = k.x_rows * 128 + 16384;
    k.stages = C::RING / stage < C::MAX_STAGES ? C::RING / stage : C::MAX_STAGES;
    k.ring_bytes = k.stages * stage;
    if (k.ring_bytes < k.x_rows * kPitch * 4) k.ring_bytes = (k.x_rows * kPitch * 4 + 1023) / 1024 * 1024;
    const int64_t tiles = (int64_t)k.m_tiles * k.n_tiles * (k.two ? 2 : 1);
    const int parts = k.parts = small_parts(FORM, k.M, k.N, k.Kd, k.terms, k.two, sms);
    shmm::count_launch();
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    const char *pdl = getenv("SHMM_PDL");
    cfg.gridDim = dim3((unsigned)(tiles * parts));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = (size_t)(k.ring_bytes + C::FIXED);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = (pdl && pdl[0] == '0') ? 1 : 2;
    return (int)cudaLaunchKernelEx(&cfg, contract_small_kernel<FORM, ACT>, k);
}

}  // namespace

namespace shmm_tcn {

// As many parts as there are places for, with four k-blocks each at least.
int small_parts(int form, int64_t M, int64_t N, int64_t Kd, int terms, bool two, int sms) {
    const bool f8 = form == kNN8 || form == kNT8;
    const int64_t width = form == kGated ? 64 : 128, bk = f8 ? 128 : 64;
    const int64_t tiles = (M + 127) / 128 * ((N + width - 1) / width) * (two ? 2 : 1), all = terms * ((Kd + bk - 1) / bk);
    const int64_t places = (int64_t)sms * (f8 ? Cfg<kNN8>::CTAS : Cfg<kGated>::CTAS);
    int parts = 1;
    while (parts < 8 && tiles * parts * 2 <= places && all >= parts * 2 * 4) parts *= 2;
    return parts;
}

int launch_small(ContractK &k, int form, int sms, cudaStream_t s) {
    switch (form) {
        case kGated:
            return k.act == SHMM_SILU ? launch_form<kGated, SHMM_SILU>(k, sms, s) : launch_form<kGated, SHMM_GELU_TANH>(k, sms, s);
        case kNT: return launch_form<kNT, SHMM_SILU>(k, sms, s);
        case kTN: return launch_form<kTN, SHMM_SILU>(k, sms, s);
        case kNN8: return launch_form<kNN8, SHMM_SILU>(k, sms, s);
        default: return launch_form<kNT8, SHMM_SILU>(k, sms, s);
    }
}

}  // namespace shmm_tcn
