// 8-bit blocks (e4m3 values with a power-of-two scale for each 128 columns of
// a row, or each 128 x 128 values) and the element-wise gradient of the gated
// MLP block that reads them.
//
// A block's scale is the smallest 2^e (e >= -126) with 448 * 2^e at or above
// its largest finite magnitude, 1 for a block of zeros.  e4m3's relative step
// is the same in every binade, so a power of two gives up nothing but a part
// of one binade of range, and the arithmetic around it is exact: x * 2^-e is
// exact in fp32, the only rounding is the one to e4m3 (to nearest even), and a
// restored value (four significant bits times 2^e) is exact in bf16 and fp32.
// Infinities and NaN become NaN and leave the rest of the block as it is.
//
// All three kernels are bound by HBM: one read and one write of every value.

#include <cuda_bf16.h>
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

constexpr int kBlock = 128;
// Blocks of a grid, and holders of one, that a kernel's parameters have room for:
// CAP in its structures, kFew or all.  With all, 2 to 14 KB go with each launch.
constexpr int kFew = 16, kAll = SHMM_MAX_RANKS;
constexpr int kThreads = 256;
// A warp takes this many columns of one row, kPieces pieces of 256: enough
// loads in flight per lane to cover the memory's latency.
constexpr int kPieces = 4;
constexpr int kChunk = 256 * kPieces;
constexpr int kBackPieces = 8, kBackChunk = 256 * kBackPieces;  // of 8-byte loads

// Eight consecutive values of a row as they are stored, and widened: loads are
// kept apart from their use, so that all of a warp's are in flight at once.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    static constexpr bool kHalf = true;  // a value's bits are the upper half of an fp32 value's
    uint32_t w[4];
    __device__ __forceinline__ void vec(const __nv_bfloat16 *p) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p);
        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    }
    __device__ __forceinline__ void one(int i, __nv_bfloat16 v) {
        w[i / 2] |= (uint32_t)__bfloat16_as_ushort(v) << (16 * (i % 2));
    }
    __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0; }
    __device__ __forceinline__ void get(float *v) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    // The largest magnitude's bits as fp32 (infinities and NaN above all others).
    __device__ __forceinline__ uint32_t top() const {
        const uint32_t m = 0x7FFF7FFFu;
        const uint32_t both = __vmaxu2(__vmaxu2(w[0] & m, w[1] & m), __vmaxu2(w[2] & m, w[3] & m));
        return max(both & 0xFFFF0000u, both << 16);
    }
};
template <>
struct Raw8<float> {
    static constexpr bool kHalf = false;
    float f[8];
    __device__ __forceinline__ void vec(const float *p) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    __device__ __forceinline__ void one(int i, float v) { f[i] = v; }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.0f;
    }
    __device__ __forceinline__ void get(float *v) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f[i];
    }
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
        return m;
    }
};
template <>
struct Raw8<uint8_t> {
    uint32_t w[2];
    __device__ __forceinline__ void vec(const uint8_t *p) {
        const uint2 q = *reinterpret_cast<const uint2 *>(p);
        w[0] = q.x, w[1] = q.y;
    }
    __device__ __forceinline__ void one(int i, uint8_t v) { w[i / 4] |= (uint32_t)v << (8 * (i % 4)); }
    __device__ __forceinline__ void clear() { w[0] = w[1] = 0; }
    __device__ __forceinline__ void get(float *v) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = from_e4m3x2(w[i / 2] >> (16 * (i % 2)));
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
};
// `left` of the eight exist.
template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T *p, int64_t left, Raw8<T> *r) {
    if (VEC) {
        r->vec(p);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) r->one(i, p[i]);
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *p, int64_t left, const float *v) {
    if (VEC) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = __float2bfloat16_rn(v[i]);
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(float *p, int64_t left, const float *v) {
    if (VEC) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = v[i];
    }
}
// Eight values times `inv` as e4m3; `finite`: the block has no infinity (NaN
// stays NaN either way).
template <bool VEC>
__device__ __forceinline__ void store8_e4m3(uint8_t *p, int64_t left, const float *v, float inv, bool finite) {
    uint32_t w[2];
    if (finite) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = finite_to_e4m3x2(v[4 * i] * inv, v[4 * i + 1] * inv) |
                   finite_to_e4m3x2(v[4 * i + 2] * inv, v[4 * i + 3] * inv) << 16;
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = to_e4m3x2(v[4 * i] * inv, v[4 * i + 1] * inv) | to_e4m3x2(v[4 * i + 2] * inv, v[4 * i + 3] * inv) << 16;
    }
    if (VEC) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
}

// ---- to 8 bits ------------------------------------------------------------

// One block of the source grid per blockIdx.z, read at src[z].
template <int CAP>
struct ToK {
    const void *src[CAP];
    uint8_t *codes;
    float *scale;
    int64_t brows, bcols, src_ld, ld, scale_ld;
    int64_t codes_n, scale_n;  // extents (bounds-checked build)
    int b1;                    // blocks along the columns
    int per;                   // scale blocks along a block's columns
    int *status;
};

// A scale for each 128 columns of a row: a warp takes a row's chunk of
// columns, 16 lanes a block, so the largest magnitude takes four shuffles.
// 8192 x 16384 bf16: 71 us, 5.7 TB/s, 66 % of the issue slots; 16 x 4096: 1.8 us
// replayed from a graph.  Two pieces fewer or four more per lane: 88, 80 us.
template <typename T, bool VEC, int CAP>
__global__ void __launch_bounds__(kThreads) to_rows_kernel(const __grid_constant__ ToK<CAP> k) {
    shmm_pdl::pdl_enter();
    const int lane = threadIdx.x % 32;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    if (row >= k.brows) return;
    const int bi = blockIdx.z / k.b1, bj = blockIdx.z % k.b1;
    const T *src = static_cast<const T *>(k.src[blockIdx.z]) + row * k.src_ld;
    const int64_t at = (bi * k.brows + row) * k.ld + bj * k.bcols;
    const int64_t s_at = (bi * k.brows + row) * k.scale_ld + (int64_t)bj * k.per;
    for (int64_t c0 = (int64_t)blockIdx.y * kChunk; c0 < k.bcols; c0 += (int64_t)gridDim.y * kChunk) {
        Raw8<T> raw[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int64_t c = c0 + i * 256 + lane * 8;
            raw[i].clear();
            if (c < k.bcols && piece_in_bounds<VEC>(k.status, row * k.src_ld + c, k.bcols - c, k.brows * k.src_ld))
                load8<VEC>(src + c, k.bcols - c, &raw[i]);
        }
        // The blocks' largest magnitudes over 16 lanes; those of bf16 values two to a
        // register.
        uint32_t top[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) top[i] = raw[i].top();
        if (Raw8<T>::kHalf) {
#pragma unroll
            for (int i = 0; i < kPieces; i += 2) {
                uint32_t two = top[i] | top[i + 1] >> 16;
#pragma unroll
                for (int d = 1; d < 16; d *= 2) two = __vmaxu2(two, __shfl_xor_sync(0xFFFFFFFFu, two, d));
                top[i] = two & 0xFFFF0000u;
                top[i + 1] = two << 16;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
#pragma unroll
                for (int d = 1; d < 16; d *= 2) top[i] = max(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], d));
        }
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) most = max(most, top[i]);
        const bool all_finite = !__any_sync(0xFFFFFFFFu, most >= 0x7F800000u);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int64_t c = c0 + i * 256 + lane * 8;
            float v[8];
            raw[i].get(v);
            const bool finite = top[i] < 0x7F800000u;
            float amax = __uint_as_float(top[i]);
            if (!all_finite) {  // the largest finite one, where that is another
                float m = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = fmaxf(m, finite_abs(v[j]));
#pragma unroll
                for (int d = 1; d < 16; d *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
                amax = m;
            }
            const int e = scale_exp(amax);
            if (c >= k.bcols) continue;
            if (piece_in_bounds<VEC>(k.status, at + c, k.bcols - c, k.codes_n))
                store8_e4m3<VEC>(k.codes + at + c, k.bcols - c, v, pow2(-e), finite);
            if (lane % 16 == 0 && in_bounds(k.status, s_at + c / kBlock, 1, k.scale_n)) k.scale[s_at + c / kBlock] = pow2(e);
        }
    }
}

// A scale for each 128 x 128 values: a CTA takes a block, which stays in its
// registers between the largest magnitude and the rounding.  8192 x 16384 bf16:
// 70 us, 5.8 TB/s.
template <typename T, bool VEC, int CAP>
__global__ void __launch_bounds__(kThreads) to_squares_kernel(const __grid_constant__ ToK<CAP> k) {
    shmm_pdl::pdl_enter();
    __shared__ uint32_t part[kThreads / 32];
    const int bi = blockIdx.z / k.b1, bj = blockIdx.z % k.b1;
    const int x = threadIdx.x % 16, y = threadIdx.x / 16;
    const T *src = static_cast<const T *>(k.src[blockIdx.z]);
    const int64_t rb = blockIdx.x;
    for (int64_t cb = blockIdx.y; cb < k.per; cb += gridDim.y) {
        const int64_t c = cb * kBlock + x * 8, r0 = rb * kBlock + y;
        Raw8<T> raw[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = r0 + 16 * i;
            raw[i].clear();
            if (r < k.brows && c < k.bcols &&
                piece_in_bounds<VEC>(k.status, r * k.src_ld + c, k.bcols - c, k.brows * k.src_ld))
                load8<VEC>(src + r * k.src_ld + c, k.bcols - c, &raw[i]);
        }
        // The largest magnitude's bits over the CTA; with an infinity or NaN among the
        // values, those of the largest finite one.
        auto over_cta = [&](uint32_t m) -> uint32_t {
#pragma unroll
            for (int d = 1; d < 32; d *= 2) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
            __syncthreads();  // the last values have been read
            if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = m;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kThreads / 32; ++i) m = max(m, part[i]);
            return m;
        };
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, raw[i].top());
        top = over_cta(top);
        const bool finite = top < 0x7F800000u;
        if (!finite) {
            top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float v[8];
                raw[i].get(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(finite_abs(v[j])));
            }
            top = over_cta(top);
        }
        const float amax = __uint_as_float(top);
        const int e = scale_exp(amax);
        const int64_t s_at = (bi * ((k.brows + kBlock - 1) / kBlock) + rb) * k.scale_ld + (int64_t)bj * k.per + cb;
        if (threadIdx.x == 0 && in_bounds(k.status, s_at, 1, k.scale_n)) k.scale[s_at] = pow2(e);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = r0 + 16 * i, at = (bi * k.brows + r) * k.ld + bj * k.bcols + c;
            if (r < k.brows && c < k.bcols && piece_in_bounds<VEC>(k.status, at, k.bcols - c, k.codes_n))
            {
                float v[8];
                raw[i].get(v);
                store8_e4m3<VEC>(k.codes + at, k.bcols - c, v, pow2(-e), finite);
            }
        }
    }
}

// ---- and back -------------------------------------------------------------

template <int CAP>
struct BackK {
    const void *src[CAP];
    const float *scale[CAP];
    void *dst;
    int64_t brows, bcols, src_ld, ld, scale_ld, dst_n;
    int b1, scale_rows, beside;
    int *status;
};

// 8192 x 4096 to bf16: 17 us, 6.0 TB/s.
template <typename T, bool VEC, int CAP>
__global__ void __launch_bounds__(kThreads) back_kernel(const __grid_constant__ BackK<CAP> k) {
    shmm_pdl::pdl_enter(k.beside);
    const int lane = threadIdx.x % 32;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    const int64_t cols = row < k.brows ? k.bcols : 0;
    const int bi = blockIdx.z / k.b1, bj = blockIdx.z % k.b1;
    const uint8_t *src = static_cast<const uint8_t *>(k.src[blockIdx.z]) + row * k.src_ld;
    const int64_t s_row = row / k.scale_rows * k.scale_ld;
    const int64_t s_n = (k.brows + k.scale_rows - 1) / k.scale_rows * k.scale_ld;
    const float *scale = k.scale[blockIdx.z] + s_row;
    const int64_t at = (bi * k.brows + row) * k.ld + bj * k.bcols;
    for (int64_t c0 = (int64_t)blockIdx.y * kBackChunk; c0 < cols; c0 += (int64_t)gridDim.y * kBackChunk) {
        Raw8<uint8_t> raw[kBackPieces];
        float s[kBackPieces];
#pragma unroll
        for (int i = 0; i < kBackPieces; ++i) {
            const int64_t c = c0 + i * 256 + lane * 8;
            s[i] = 0.0f;
            raw[i].clear();
            if (c < k.bcols && piece_in_bounds<VEC>(k.status, row * k.src_ld + c, k.bcols - c, k.brows * k.src_ld) &&
                in_bounds(k.status, s_row + c / kBlock, 1, s_n)) {
                load8<VEC>(src + c, k.bcols - c, &raw[i]);
                s[i] = scale[c / kBlock];
            }
        }
#pragma unroll
        for (int i = 0; i < kBackPieces; ++i) {
            const int64_t c = c0 + i * 256 + lane * 8;
            if (c >= k.bcols || !piece_in_bounds<VEC>(k.status, at + c, k.bcols - c, k.dst_n)) continue;
            float v[8];
            raw[i].get(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= s[i];
            store8<VEC>(static_cast<T *>(k.dst) + at + c, k.bcols - c, v);
        }
    }
    shmm_pdl::pdl_end(k.beside);
}

// ---- the gated block's gradient, element by element ------------------------

template <int CAP>
struct SlopeK {
    const void *dH[CAP], *G[CAP], *U[CAP];
    const float *g_scale[CAP], *u_scale[CAP];
    void *H[CAP];              // holders of every block, block by block
    uint16_t h_first[CAP + 1]; // block z's holders: H[h_first[z]] .. H[h_first[z + 1] - 1]
    void *dG, *dU;
    int64_t brows, bcols, ld, scale_ld, out_n;
    int b1;
    int *status;
};

// T: the gradients' type; S: the kept pre-activations' (uint8_t: 8 bits).
// Pieces of eight values, two in flight per lane.  Everything is fp32 up to dG
// and dU, which are rounded to T: they are the next products' operands, and the
// tensor cores' have no more bits.  (In bf16 half a step on each is 1.7e-3 of
// their 2-norm, and what comes of them is that much less exact.)
//
// 8192 x 16384 bf16 from 8 bits: 184 us, 5.8 TB/s, and 72 % of the issue slots.
template <typename T, typename S, int ACT, bool VEC, int CAP>
__global__ void __launch_bounds__(kThreads) slope_kernel(const __grid_constant__ SlopeK<CAP> k) {
    constexpr bool E8 = sizeof(S) == 1;
    constexpr int PIECES = 2;
    shmm_pdl::pdl_enter();
    const int lane = threadIdx.x % 32;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    if (row >= k.brows) return;
    const int z = blockIdx.z, bi = z / k.b1, bj = z % k.b1;
    const int64_t in = row * k.bcols, n = k.brows * k.bcols;
    const int64_t at = (bi * k.brows + row) * k.ld + bj * k.bcols;
    for (int64_t c0 = (int64_t)blockIdx.y * (256 * PIECES); c0 < k.bcols; c0 += (int64_t)gridDim.y * (256 * PIECES)) {
        Raw8<T> dr[PIECES];
        Raw8<S> gr[PIECES], ur[PIECES];
        float gs[PIECES], us[PIECES];
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int64_t c = c0 + i * 256 + lane * 8, left = k.bcols - c;
            gs[i] = us[i] = 1.0f;
            dr[i].clear(), gr[i].clear(), ur[i].clear();
            if (left <= 0 || !piece_in_bounds<VEC>(k.status, in + c, left, n)) continue;
            load8<VEC>(static_cast<const T *>(k.dH[z]) + in + c, left, &dr[i]);
            load8<VEC>(static_cast<const S *>(k.G[z]) + in + c, left, &gr[i]);
            load8<VEC>(static_cast<const S *>(k.U[z]) + in + c, left, &ur[i]);
            const int64_t s = row * k.scale_ld + c / kBlock;
            if (E8 && in_bounds(k.status, s, 1, k.brows * k.scale_ld)) {
                gs[i] = k.g_scale[z][s];
                us[i] = k.u_scale[z][s];
            }
        }
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int64_t c = c0 + i * 256 + lane * 8, left = k.bcols - c;
            if (left <= 0 || !piece_in_bounds<VEC>(k.status, at + c, left, k.out_n)) continue;
            float d[8], g[8], u[8], h[8];
            dr[i].get(d), gr[i].get(g), ur[i].get(u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float gj = E8 ? g[j] * gs[i] : g[j], uj = E8 ? u[j] * us[i] : u[j];
                float slope;
                const float a = gate_act_slope<ACT>(gj, &slope);
                h[j] = a * uj;
                g[j] = d[j] * uj * slope;
                u[j] = d[j] * a;
            }
            store8<VEC>(static_cast<T *>(k.dG) + at + c, left, g);
            store8<VEC>(static_cast<T *>(k.dU) + at + c, left, u);
            for (int q = k.h_first[z]; q < k.h_first[z + 1]; ++q)
                if (piece_in_bounds<VEC>(k.status, in + c, left, n)) store8<VEC>(static_cast<T *>(k.H[q]) + in + c, left, h);
        }
    }
}

// ---- host side --------------------------------------------------------------

bool aligned(const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

// Whole 8-value pieces of rows `ld` apart (and blocks bcols wide) start on
// their own boundaries.
bool pieces_fit(int64_t bcols, int64_t ld) { return bcols % 8 == 0 && ld % 8 == 0; }

dim3 rows_grid(int64_t brows, int64_t bcols, int64_t chunk, int blocks) {
    const int64_t y = (bcols + chunk - 1) / chunk;
    return dim3((unsigned)((brows + kThreads / 32 - 1) / (kThreads / 32)), (unsigned)(y < 65535 ? y : 65535),
                (unsigned)blocks);
}

template <int CAP>
int quantize(const shmm::GridOperand &src, void *codes, int64_t ld, float *scale, int64_t scale_ld, int *status,
             void *stream) {
    const int blocks = src.b0 * src.b1;
    ToK<CAP> k = {};
    for (int i = 0; i < blocks; ++i) k.src[i] = src.at[i];
    k.codes = static_cast<uint8_t *>(codes);
    k.scale = scale;
    k.brows = src.brows;
    k.bcols = src.bcols;
    k.src_ld = src.ld;
    k.ld = ld;
    k.scale_ld = scale_ld;
    k.b1 = src.b1;
    k.per = (int)((src.bcols + kBlock - 1) / kBlock);
    k.codes_n = src.b0 * src.brows * ld;
    k.scale_n = src.b0 * ((src.brows + src.scale_rows - 1) / src.scale_rows) * scale_ld;
    k.status = status;
    bool vec = pieces_fit(src.bcols, src.ld) && ld % 8 == 0 && aligned(codes, 8);
    for (int i = 0; i < blocks; ++i) vec = vec && aligned(src.at[i], 16);
    const bool f32 = src.dt == SHMM_F32, squares = src.scale_rows == kBlock;
    dim3 grid = rows_grid(src.brows, src.bcols, kChunk, blocks);
    if (squares)
        grid = dim3((unsigned)((src.brows + kBlock - 1) / kBlock), (unsigned)(k.per < 65535 ? k.per : 65535), (unsigned)blocks);
    cudaStream_t s = (cudaStream_t)stream;
    shmm::count_launch();
#define GO(KERN, T) (int)(vec ? shmm_pdl::launch_pdl(KERN<T, true, CAP>, grid, dim3(kThreads), 0, s, k) \
                              : shmm_pdl::launch_pdl(KERN<T, false, CAP>, grid, dim3(kThreads), 0, s, k))
    if (squares) return f32 ? GO(to_squares_kernel, float) : GO(to_squares_kernel, __nv_bfloat16);
    return f32 ? GO(to_rows_kernel, float) : GO(to_rows_kernel, __nv_bfloat16);
#undef GO
}

template <int CAP>
int dequantize(const shmm::GridOperand &src, void *dst, int64_t ld, shmm_dtype_t dt, int *status, void *stream,
               bool beside) {
    const int blocks = src.b0 * src.b1;
    BackK<CAP> k = {};
    bool vec = pieces_fit(src.bcols, src.ld) && ld % 8 == 0 && aligned(dst, 16);
    for (int i = 0; i < blocks; ++i) {
        k.src[i] = src.at[i];
        k.scale[i] = src.scale[i];
        vec = vec && aligned(src.at[i], 8);
    }
    k.dst = dst;
    k.brows = src.brows;
    k.bcols = src.bcols;
    k.src_ld = src.ld;
    k.ld = ld;
    k.scale_ld = src.scale_ld;
    k.dst_n = src.b0 * src.brows * ld;
    k.b1 = src.b1;
    k.scale_rows = src.scale_rows;
    k.beside = beside;
    k.status = status;
    const dim3 grid = rows_grid(src.brows, src.bcols, kBackChunk, blocks);
    cudaStream_t s = (cudaStream_t)stream;
    shmm::count_launch();
    if (dt == SHMM_F32)
        return (int)(vec ? shmm_pdl::launch_pdl(back_kernel<float, true, CAP>, grid, dim3(kThreads), 0, s, k)
                         : shmm_pdl::launch_pdl(back_kernel<float, false, CAP>, grid, dim3(kThreads), 0, s, k));
    return (int)(vec ? shmm_pdl::launch_pdl(back_kernel<__nv_bfloat16, true, CAP>, grid, dim3(kThreads), 0, s, k)
                     : shmm_pdl::launch_pdl(back_kernel<__nv_bfloat16, false, CAP>, grid, dim3(kThreads), 0, s, k));
}

template <int CAP>
int gated_slopes(const shmm::GatedSlopeArgs &a, int *status, void *stream) {
    const int blocks = a.dH.b0 * a.dH.b1;
    const bool e8 = a.G.dt == SHMM_E4M3;
    SlopeK<CAP> k = {};
    bool vec = pieces_fit(a.dH.bcols, a.cols) && aligned(a.dG, 16) && aligned(a.dU, 16);
    int h = 0;
    for (int i = 0; i < blocks; ++i) {
        k.dH[i] = a.dH.at[i];
        k.G[i] = a.G.at[i];
        k.U[i] = a.U.at[i];
        vec = vec && aligned(k.dH[i], 16) && aligned(k.G[i], e8 ? 8 : 16) && aligned(k.U[i], e8 ? 8 : 16);
        if (e8) {
            k.g_scale[i] = a.G.scale[i];
            k.u_scale[i] = a.U.scale[i];
        }
        k.h_first[i] = (uint16_t)h;
        if (a.want_H)
            for (void *p : a.H.holders[i]) {
                k.H[h++] = p;
                vec = vec && aligned(p, 16);
            }
    }
    k.h_first[blocks] = (uint16_t)h;
    k.dG = a.dG;
    k.dU = a.dU;
    k.brows = a.dH.brows;
    k.bcols = a.dH.bcols;
    k.ld = a.cols;
    k.scale_ld = a.G.scale_ld;
    k.out_n = a.rows * a.cols;
    k.b1 = a.dH.b1;
    k.status = status;
    const dim3 grid = rows_grid(k.brows, k.bcols, 512, blocks);
    cudaStream_t s = (cudaStream_t)stream;
    shmm::count_launch();
#define GO(T, S, ACT) (int)(vec ? shmm_pdl::launch_pdl(slope_kernel<T, S, ACT, true, CAP>, grid, dim3(kThreads), 0, s, k) \
                                : shmm_pdl::launch_pdl(slope_kernel<T, S, ACT, false, CAP>, grid, dim3(kThreads), 0, s, k))
#define GO_ACT(T, S) (a.act == SHMM_SILU ? GO(T, S, SHMM_SILU) : GO(T, S, SHMM_GELU_TANH))
    if (a.dt == SHMM_F32) return e8 ? GO_ACT(float, uint8_t) : GO_ACT(float, float);
    return e8 ? GO_ACT(__nv_bfloat16, uint8_t) : GO_ACT(__nv_bfloat16, __nv_bfloat16);
#undef GO_ACT
#undef GO
}

}  // namespace

namespace shmm {

int launch_quantize(const GridOperand &src, void *codes, int64_t ld, float *scale, int64_t scale_ld, int *status,
                    void *stream) {
    if (src.brows == 0 || src.bcols == 0) return 0;
    return src.b0 * src.b1 <= kFew ? quantize<kFew>(src, codes, ld, scale, scale_ld, status, stream)
                                   : quantize<kAll>(src, codes, ld, scale, scale_ld, status, stream);
}

int launch_dequantize(const GridOperand &src, void *dst, int64_t ld, shmm_dtype_t dt, int *status, void *stream,
                      bool beside) {
    if (src.brows == 0 || src.bcols == 0) return 0;
    return src.b0 * src.b1 <= kFew ? dequantize<kFew>(src, dst, ld, dt, status, stream, beside)
                                   : dequantize<kAll>(src, dst, ld, dt, status, stream, beside);
}

int launch_gated_slopes(const GatedSlopeArgs &a, int *status, void *stream) {
    if (a.dH.brows == 0 || a.dH.bcols == 0) return 0;
    size_t n = (size_t)a.dH.b0 * a.dH.b1, h = 0;
    if (a.want_H)
        for (const auto &b : a.H.holders) h += b.size();
    return (n > h ? n : h) <= kFew ? gated_slopes<kFew>(a, status, stream) : gated_slopes<kAll>(a, status, stream);
}

}  // namespace shmm
