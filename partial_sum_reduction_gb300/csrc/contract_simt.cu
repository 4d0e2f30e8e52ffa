// The products of the gated MLP block and of 8-bit operands on the CUDA cores:
// any type, size and sharding, for fp32 operands and for shapes that the tensor
// cores' loads cannot address.
//
// A CTA computes 32 rows by 128 columns of the result, the columns counted from
// a result block's left edge, so a 128-column scale block of a kept 8-bit
// result lies in one warp.  The contracted dim goes through shared memory 64 at
// a time.  Two groups of eight warps take 32 of the 64 each, a warp 4 rows and a
// lane 4 columns (of both projections): 16 warps at 128 registers, where one
// group's 8 warps left FMAs waiting for shared memory.  Two pieces lie in shared
// memory and the loads of a third are in flight, with one barrier per piece.
// Everything is fp32; sums of 64 products are added to a second sum (in shared
// memory), so an element's error grows with the number of pieces and not of
// products.  (Of a million values that are kept in 8 bits, sums of 256 leave 27
// on another side of a rounding border than 64-bit sums do, these 13, and a
// library's fp32 products 34; they cost 3 %.)
//
// Measured (fp32): gated forward 301 x 1000 x 1157 in 78 us (18 TFLOP/s; 87 with
// one group of 8 warps and 32-deep pieces), its backward pass in 213 (248),
// forward 1024 x 1024 x 1500 in 229 (247), 2048 x 2048 x 2048 in 1068 (32
// TFLOP/s; 1115); the one-operand products of 2048 x 2048 x 2048 lose 8 to 9 %
// (dA 1267 -> 1368 us).  A 64-deep piece takes 4.7 us of an SM, 2.2 of them FMAs;
// shared-memory reads (9 to 10 cycles for 8 of FMAs) take half of the cycles and
// issue slots 47 %, and what is left is waits for either and for the loads.
// Packed FMAs (2 % slower), 8 rows to a thread with four groups (16 %; packed 3
// %) gained nothing.

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <vector>

#include "checked.cuh"
#include "e4m3.cuh"
#include "gated_act.cuh"
#include "pdl.cuh"
#include "shmm_internal.h"

namespace {

using namespace shmm_dev;

constexpr int TM = 32, TN = 128, TK = 64;
constexpr int kThreads = 512, kGroups = 2;
constexpr int kFlush = 2;   // pieces in the first sum, each TK / kGroups products of it
constexpr int XS = TM + 4, YS = TN + 4;  // shared rows of the pieces, whole 16-byte vectors

// An operand: at most CAP blocks.
template <int CAP>
struct Op {
    const void *at[CAP];
    const float *scale[CAP];
    int64_t brows, bcols, ld, scale_ld;
    int b0, b1, scale_rows;
};

template <int CAP>
struct Res {
    void *to[CAP];
    float *scale[CAP];
    uint16_t first[CAP + 1];  // block p's holders: to[first[p]] .. to[first[p + 1] - 1]
    int64_t brows, bcols, scale_ld;
    int b0, b1, dt;
};

template <int CAP>
struct SimtK {
    Op<CAP> X[2], Y[2];
    Res<CAP> D, kept[2];
    int64_t M, N, Kd;
    int terms, x_t, y_t, keep, act, beside;
    int n_per;  // column tiles of a result block
    int *status;
};

__device__ __forceinline__ float wide(float v) { return v; }
__device__ __forceinline__ float wide(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float wide(uint8_t v) { return from_e4m3x2(v).x; }

// Stored element (r, c) of an operand of several blocks.  T: uint8_t for 8 bits.
template <typename T, int CAP>
__device__ __forceinline__ float fetch(const Op<CAP> &o, int64_t r, int64_t c, int *status) {
    const int64_t b = r / o.brows, d = c / o.bcols;
    const int p = (int)b * o.b1 + (int)d;
    r -= b * o.brows;
    c -= d * o.bcols;
    const int64_t i = r * o.ld + c;
    if (!in_bounds(status, i, 1, (o.brows - 1) * o.ld + o.bcols)) return 0.0f;
    const float v = wide(static_cast<const T *>(o.at[p])[i]);
    if (sizeof(T) > 1) return v;
    const int64_t s = r / o.scale_rows * o.scale_ld + c / 128;
    if (!in_bounds(status, s, 1, (o.brows + o.scale_rows - 1) / o.scale_rows * o.scale_ld)) return 0.0f;
    return v * o.scale[p][s];
}

// N elements of one thread's part of a piece: element i at result index a0 + i *
// DA, contracted index k0 + i * DK (one of the two is 0; 0 past the ends), stored
// as [result, contracted] or, MAJOR_K, the other way round.  One block: addresses
// a stride apart, so the loads go out together at an add or two each.
template <typename T, int CAP, int N, bool MAJOR_K, int DA, int DK>
__device__ __forceinline__ void fetch_part(const Op<CAP> &o, int64_t a0, int64_t a_end, int64_t k0, int64_t k_end, float *v,
                                           int *status) {
    static_assert((DA == 0) != (DK == 0), "one index moves");
    if (o.b0 * o.b1 == 1) {
        // how many of the N exist
        const int64_t room = DA ? (a_end - a0 + DA - 1) / (DA ? DA : 1) : (k_end - k0 + DK - 1) / (DK ? DK : 1);
        const int count = (DA ? k0 < k_end : a0 < a_end) ? (room < N ? (int)room : N) : 0;
        const int64_t r0 = MAJOR_K ? k0 : a0, c0 = MAJOR_K ? a0 : k0;
        const uint32_t step = (uint32_t)(MAJOR_K ? (DA ? DA : DK * o.ld) : (DA ? DA * o.ld : DK));  // N of them: below 2^31
        const int64_t at0 = r0 * o.ld + c0, n = (o.brows - 1) * o.ld + o.bcols;
        const T *p = static_cast<const T *>(o.at[0]) + at0;
        T raw[N];
        float sc[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool in = i < count && in_bounds(status, at0 + (int64_t)i * step, 1, n);
            raw[i] = T(0);
            sc[i] = 0.0f;
            if (in) raw[i] = p[(uint32_t)i * step];
            if (sizeof(T) == 1 && in) {
                const int64_t r = r0 + i * (MAJOR_K ? DK : DA), c = c0 + i * (MAJOR_K ? DA : DK);
                const int64_t s = (o.scale_rows == 1 ? r : r / 128) * o.scale_ld + c / 128;
                if (in_bounds(status, s, 1, (o.brows + o.scale_rows - 1) / o.scale_rows * o.scale_ld)) sc[i] = o.scale[0][s];
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = sizeof(T) == 1 ? wide(raw[i]) * sc[i] : wide(raw[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t a = a0 + (int64_t)i * DA, kk = k0 + (int64_t)i * DK;
            v[i] = a < a_end && kk < k_end ? fetch<T>(o, MAJOR_K ? kk : a, MAJOR_K ? a : kk, status) : 0.0f;
        }
    }
}

__device__ __forceinline__ void store_as(void *p, int64_t i, int dt, float v) {
    if (dt == SHMM_F32) static_cast<float *>(p)[i] = v;
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// Four values of global row `row`, columns cl .. cl + 3 of block column cb, to
// every holder.
template <int CAP>
__device__ __forceinline__ void put4(const Res<CAP> &d, int64_t row, int cb, int64_t cl, const float *v, int *status) {
    const int64_t br = row / d.brows, at = (row - br * d.brows) * d.bcols + cl;
    const int p = (int)br * d.b1 + cb;
    for (int q = d.first[p]; q < d.first[p + 1]; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (cl + j < d.bcols && in_bounds(status, at + j, 1, d.brows * d.bcols)) store_as(d.to[q], at + j, d.dt, v[j]);
}

// The same in 8 bits: the warp holds the row's block of 128 columns.
template <int CAP>
__device__ __forceinline__ void put4_e4m3(const Res<CAP> &d, int64_t row, bool row_ok, int cb, int64_t cl, const float *v,
                                          int lane, int *status) {
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (cl + j < d.bcols) amax = fmaxf(amax, finite_abs(v[j]));
#pragma unroll
    for (int s = 1; s < 32; s *= 2) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, s));
    if (!row_ok) return;
    const int e = scale_exp(amax);
    const float inv = pow2(-e);
    const int64_t br = row / d.brows, rl = row - br * d.brows, at = rl * d.bcols + cl, s = rl * d.scale_ld + cl / 128;
    const int p = (int)br * d.b1 + cb;
    const uint32_t w = to_e4m3x2(v[0] * inv, v[1] * inv) | to_e4m3x2(v[2] * inv, v[3] * inv) << 16;
    for (int q = d.first[p]; q < d.first[p + 1]; ++q) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (cl + j < d.bcols && in_bounds(status, at + j, 1, d.brows * d.bcols))
                static_cast<uint8_t *>(d.to[q])[at + j] = (uint8_t)(w >> (8 * j));
        if (lane == 0 && in_bounds(status, s, 1, d.brows * d.scale_ld)) d.scale[q][s] = pow2(e);
    }
}

// Shared memory: two pieces of X and Y, then every thread's second sums.
struct __align__(16) XPiece { float v[TK][XS]; };
struct __align__(16) YPiece { float v[TK][YS]; };
constexpr size_t smem_bytes(int ny) { return 2 * (sizeof(XPiece) + ny * sizeof(YPiece)) + (size_t)ny * 4 * kThreads * sizeof(float4); }
static_assert(smem_bytes(2) <= 227 * 1024, "a CTA's shared memory");

template <typename T, int CAP, bool GATED>
__global__ void __launch_bounds__(kThreads, 1) contract_simt_kernel(const __grid_constant__ SimtK<CAP> k) {
    constexpr int NY = GATED ? 2 : 1;
    constexpr int PX = TM * TK / kThreads, PY = TK * TN / kThreads;
    extern __shared__ __align__(16) uint8_t smem[];
    XPiece *xs = reinterpret_cast<XPiece *>(smem);
    YPiece *ys = reinterpret_cast<YPiece *>(xs + 2);  // [2][NY]
    float4 *sums = reinterpret_cast<float4 *>(ys + 2 * NY);  // [NY * 4][kThreads]
    shmm_pdl::pdl_enter(k.beside);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32 % 8, group = tid / 256;
    const int64_t m0 = (int64_t)blockIdx.x * TM;
    const int cb = blockIdx.y / k.n_per;                                    // result block column
    const int64_t n0l = (int64_t)(blockIdx.y % k.n_per) * TN;               // first column in it
    const int64_t n0 = cb * k.D.bcols + n0l, n1 = (cb + 1) * k.D.bcols;     // ... of the whole array, and the block's end
    const int64_t per_term = (k.Kd + TK - 1) / TK, pieces = k.terms * per_term;

    // A thread's elements of a piece.  Stored with the contracted dim last, a warp
    // takes 8 of it in 4 rows, which go to 32 banks of [contracted][row].
    const int at_k = lane % 8 + warp * 8, at_r = lane / 8 + group * 4;
    float xr[PX], yr[NY][PY];
    auto ask = [&](int64_t piece) {
        const int t = piece >= per_term ? 1 : 0;
        const int64_t k0 = (piece - t * per_term) * TK;
        if (k.x_t) fetch_part<T, CAP, PX, true, 0, kThreads / TM>(k.X[t], m0 + lane, k.M, k0 + tid / TM, k.Kd, xr, k.status);
        else fetch_part<T, CAP, PX, false, kThreads / TK, 0>(k.X[t], m0 + at_r, k.M, k0 + at_k, k.Kd, xr, k.status);
#pragma unroll
        for (int y = 0; y < NY; ++y) {
            const Op<CAP> &o = k.Y[GATED ? y : t];
            if (k.y_t) fetch_part<T, CAP, PY, false, kThreads / TK, 0>(o, n0 + at_r, n1, k0 + at_k, k.Kd, yr[y], k.status);
            else fetch_part<T, CAP, PY, true, 0, kThreads / TN>(o, n0 + tid % TN, n1, k0 + tid / TN, k.Kd, yr[y], k.status);
        }
    };
    auto put = [&](int b) {
        float (&x)[TK][XS] = xs[b].v;
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            if (k.x_t) x[tid / TM + i * (kThreads / TM)][tid % TM] = xr[i];
            else x[at_k][at_r + i * (kThreads / TK)] = xr[i];
        }
#pragma unroll
        for (int y = 0; y < NY; ++y) {
            float (&v)[TK][YS] = ys[b * NY + y].v;
#pragma unroll
            for (int i = 0; i < PY; ++i) {
                if (k.y_t) v[at_k][at_r + i * (kThreads / TK)] = yr[y][i];
                else v[tid / TN + i * (kThreads / TN)][tid % TN] = yr[y][i];
            }
        }
    };

    float acc[NY][4][4] = {};
#pragma unroll
    for (int i = 0; i < NY * 4; ++i) sums[i * kThreads + tid] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (pieces) {
        ask(0);
        put(0);
    }
    for (int64_t piece = 0; piece < pieces; ++piece) {
        const int b = (int)(piece & 1);
        __syncthreads();  // this piece is in place, and the one before has been used
        if (piece + 1 < pieces) ask(piece + 1);
        const int kk0 = group * (TK / kGroups);
#pragma unroll 8
        for (int kk = kk0; kk < kk0 + TK / kGroups; ++kk) {
            const float4 x4 = *reinterpret_cast<const float4 *>(&xs[b].v[kk][warp * 4]);
            const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
            for (int y = 0; y < NY; ++y) {
                const float4 y4 = *reinterpret_cast<const float4 *>(&ys[b * NY + y].v[kk][lane * 4]);
                const float v[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[y][i][j] = fmaf(x[i], v[j], acc[y][i][j]);
            }
        }
        if (piece % kFlush == kFlush - 1 || piece + 1 == pieces) {
#pragma unroll
            for (int y = 0; y < NY; ++y)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float4 *p = &sums[(y * 4 + i) * kThreads + tid];
                    float4 v = *p;
                    v.x += acc[y][i][0];
                    v.y += acc[y][i][1];
                    v.z += acc[y][i][2];
                    v.w += acc[y][i][3];
                    *p = v;
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[y][i][j] = 0.0f;
                }
        }
        if (piece + 1 < pieces) put(b ^ 1);
    }
    __syncthreads();

    // The groups' sums together; each group finishes two of a warp's four rows.
    const int64_t cl = n0l + lane * 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = group * 2 + h;
        const int64_t row = m0 + warp * 4 + i;
        const bool row_ok = row < k.M;
        float sum[NY][4];
#pragma unroll
        for (int y = 0; y < NY; ++y) {
            const float4 a = sums[(y * 4 + i) * kThreads + tid % 256], c = sums[(y * 4 + i) * kThreads + tid % 256 + 256];
            sum[y][0] = a.x + c.x;
            sum[y][1] = a.y + c.y;
            sum[y][2] = a.z + c.z;
            sum[y][3] = a.w + c.w;
        }
        if (GATED) {
            if (k.keep) {
#pragma unroll
                for (int y = 0; y < NY; ++y) {
                    if (k.kept[y].dt == SHMM_E4M3) put4_e4m3(k.kept[y], row, row_ok, cb, cl, sum[y], lane, k.status);
                    else if (row_ok) put4(k.kept[y], row, cb, cl, sum[y], k.status);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float g = sum[0][j];
                sum[0][j] = (k.act == SHMM_SILU ? gate_act<SHMM_SILU>(g) : gate_act<SHMM_GELU_TANH>(g)) * sum[NY - 1][j];
            }
        }
        if (row_ok) put4(k.D, row, cb, cl, sum[0], k.status);
    }
    shmm_pdl::pdl_end(k.beside);
}

// ---- host side --------------------------------------------------------------

template <int CAP>
void set_op(Op<CAP> *o, const shmm::GridOperand &g) {
    for (size_t i = 0; i < g.at.size(); ++i) {
        o->at[i] = g.at[i];
        if (!g.scale.empty()) o->scale[i] = g.scale[i];
    }
    o->brows = g.brows;
    o->bcols = g.bcols;
    o->ld = g.ld;
    o->scale_ld = g.scale_ld;
    o->b0 = g.b0;
    o->b1 = g.b1;
    o->scale_rows = g.scale_rows;
}

template <int CAP>
void set_res(Res<CAP> *d, const shmm::GridResult &g) {
    int n = 0;
    for (size_t p = 0; p < g.holders.size(); ++p) {
        d->first[p] = (uint16_t)n;
        for (size_t q = 0; q < g.holders[p].size(); ++q, ++n) {
            d->to[n] = g.holders[p][q];
            if (!g.scale_holders.empty()) d->scale[n] = g.scale_holders[p][q];
        }
    }
    d->first[g.holders.size()] = (uint16_t)n;
    d->brows = g.brows;
    d->bcols = g.bcols;
    d->scale_ld = g.scale_ld;
    d->b0 = g.b0;
    d->b1 = g.b1;
    d->dt = g.dt;
}

// Blocks, and holders, of the largest table.
size_t entries(const shmm::ContractArgs &a) {
    size_t n = 1;
    for (int i = 0; i < 2; ++i) {
        n = n > a.X[i].at.size() ? n : a.X[i].at.size();
        n = n > a.Y[i].at.size() ? n : a.Y[i].at.size();
        for (const shmm::GridResult *d : {&a.D[i], &a.kept[i]}) {
            size_t h = 0;
            for (const auto &b : d->holders) h += b.size();
            n = n > h ? n : h;
        }
    }
    return n;
}

template <typename T, int CAP, bool GATED>
cudaError_t go(const SimtK<CAP> &k, dim3 grid, cudaStream_t s) {
    constexpr size_t kSmem = smem_bytes(GATED ? 2 : 1);
    static shmm::PerDevice<int> attr_set;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= shmm::kMaxDevices) return cudaErrorInvalidDevice;
    if (!attr_set.get(dev)) {
        e = cudaFuncSetAttribute(contract_simt_kernel<T, CAP, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) return e;
        attr_set.set(dev, 1);
    }
    return shmm_pdl::launch_pdl(contract_simt_kernel<T, CAP, GATED>, grid, dim3(kThreads), kSmem, s, k);
}

template <int CAP>
cudaError_t launch(const shmm::ContractArgs &a, int which, int *status, cudaStream_t s) {
    static_assert(sizeof(SimtK<CAP>) <= 32764, "kernel parameters");
    SimtK<CAP> k = {};
    for (int i = 0; i < 2; ++i) {
        set_op(&k.X[i], a.X[i]);
        set_op(&k.Y[i], a.two ? a.Y[which] : a.Y[i]);
        if (a.keep) set_res(&k.kept[i], a.kept[i]);
    }
    set_res(&k.D, a.D[which]);
    k.M = a.M;
    k.N = a.N;
    k.Kd = a.Kd;
    k.terms = a.terms;
    k.x_t = a.x_t;
    k.y_t = a.y_t;
    k.keep = a.keep;
    k.act = a.act;
    k.beside = a.beside || which == 1;  // the second of two products does not need the first
    k.n_per = (int)((k.D.bcols + TN - 1) / TN);
    k.status = status;
    const dim3 grid((unsigned)((a.M + TM - 1) / TM), (unsigned)(k.n_per * k.D.b1));
    shmm::count_launch();
    if (a.X[0].dt == SHMM_E4M3) return go<uint8_t, CAP, false>(k, grid, s);
    if (a.X[0].dt == SHMM_BF16) return a.gated ? go<__nv_bfloat16, CAP, true>(k, grid, s) : go<__nv_bfloat16, CAP, false>(k, grid, s);
    return a.gated ? go<float, CAP, true>(k, grid, s) : go<float, CAP, false>(k, grid, s);
}

}  // namespace

namespace shmm {

int launch_contract_simt(const ContractArgs &a, int *status, void *stream) {
    if (a.M == 0 || a.N == 0) return 0;
    const bool small = entries(a) <= 16;
    for (int w = 0; w < (a.two ? 2 : 1); ++w) {
        const cudaError_t e = small ? launch<16>(a, w, status, (cudaStream_t)stream)
                                    : launch<SHMM_MAX_RANKS>(a, w, status, (cudaStream_t)stream);
        if (e != cudaSuccess) return (int)e;
    }
    return 0;
}

}  // namespace shmm
