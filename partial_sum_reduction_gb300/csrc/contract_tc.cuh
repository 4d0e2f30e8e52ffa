// What the tensor-core kernels of the gated block's and the 8-bit products
// share: the launch's tables, operands walked along the contracted dim over the
// ranks' shards, operand tiles and result boxes in shared memory.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "checked.cuh"
#include "pair.cuh"

namespace shmm_tcn {

using shmm_dev::in_bounds;

enum Form { kGated, kNT, kTN, kNN8, kNT8, kGated8 };  // kGated8: the pre-activations kept in 8 bits

constexpr int kSlots = 16;  // blocks of an operand, holders of a result
constexpr int kMaps = 96;

// An operand: block p of its b0 x b1 grid is maps[map0 + p].
struct OpK {
    int map0, b0, b1;
    int64_t brows, bcols;
};
// A result: holder q is maps[map0 + q]; block p's are first[p] .. first[p + 1] - 1.
struct ResK {
    int map0, b0, b1;
    int64_t brows, bcols;
    uint8_t first[kSlots + 1];
};
// Scales of an 8-bit operand's blocks: rows ld apart, n values each.
struct ScalesK {
    const float *at[kSlots];
    int64_t ld, n;
};

struct ContractK {
    CUtensorMap maps[kMaps];
    OpK X[2], Y[2];
    ResK D[2];
    ScalesK x_scale, y_scale;
    float *kept_scale[2][kSlots];
    int64_t kept_ld;
    int kept_map[2];
    int keep;  // 0 nothing, 1 in the plan's type, 2 in 8 bits
    int64_t M, N, Kd;
    int m_tiles, n_tiles, k_blocks, terms;
    int total, half_from;  // work items; from half_from on they are half tiles
    int two, act, out_f32, beside;
    int *status;
    // the kernel for few rows: buffers of the results (D[0], D[1], kept), rows of X
    // in a stage, its boxes there, stages, their bytes, parts of the contracted dim
    void *out[4][kSlots];
    int x_rows, x_boxes, stages, ring_bytes, parts;
};

// Which block of `blocks` along a dim holds coordinate x, and the coordinate in
// it.  Past the array's end it stays past the last block's end, where TMA reads
// zeros.  Tiles never straddle a block: where a dim is split, blocks are
// multiples of 128.
__device__ __forceinline__ int split(int blocks, int64_t extent, int64_t x, int32_t *local) {
    if (blocks == 1) {
        *local = (int32_t)x;
        return 0;
    }
    int p = (int)((uint32_t)x / (uint32_t)extent);
    if (p > blocks - 1) p = blocks - 1;
    *local = (int32_t)(x - (int64_t)p * extent);
    return p;
}

__device__ __forceinline__ int block_of(const ResK &d, int row, int col, int32_t *r, int32_t *c) {
    const int p = split(d.b0, d.brows, row, r);
    return p * d.b1 + split(d.b1, d.bcols, col, c);
}

// An operand's tile as it walks the contracted dim: `map` the shard's, `fixed`
// the tile's row or column in it, `at` the contracted coordinate in it.
// K_MAJOR: stored [rows or columns of the result, contracted].
struct Cursor {
    const CUtensorMap *map;
    int step, left;  // from shard to shard, and those still to come
    int32_t fixed, at, extent;
    template <bool K_MAJOR>
    __device__ __forceinline__ void start(const CUtensorMap *maps, const OpK &o, int64_t fixed_at) {
        if (K_MAJOR) {
            map = maps + o.map0 + split(o.b0, o.brows, fixed_at, &fixed) * o.b1;
            step = 1, left = o.b1 - 1, extent = (int32_t)o.bcols;
        } else {
            map = maps + o.map0 + split(o.b1, o.bcols, fixed_at, &fixed);
            step = o.b1, left = o.b0 - 1, extent = (int32_t)o.brows;
        }
        at = 0;
    }
    // From the start to contracted coordinate `to`.
    __device__ __forceinline__ void seek(int32_t to) {
        while (left > 0 && to >= extent) {
            to -= extent;
            map += step;
            --left;
        }
        at = to;
    }
    __device__ __forceinline__ void advance(int by) {
        at += by;
        if (at >= extent && left > 0) {
            at -= extent;
            map += step;
            --left;
        }
    }
};

// The scale of a row (or of 128 columns) for one k-block after another.  With
// `in` false nothing is read and every scale is 0.
struct ScaleCursor {
    const ScalesK *t;
    const float *p;         // the shard's scales
    int64_t first, inc;     // index of the shard's first k-block, and from one to the next
    int i, n;               // k-block in the shard, of n
    int blk, step, left;
    bool in;
    // K_MAJOR: the operand is stored [result dim, contracted]; `per` values of
    // the result dim share a scale.
    template <bool K_MAJOR>
    __device__ __forceinline__ void start(const OpK &o, const ScalesK &s, int64_t fixed_at, int per, bool inside) {
        t = &s;
        in = inside;
        int32_t local;
        if (K_MAJOR) {
            blk = split(o.b0, o.brows, fixed_at, &local) * o.b1;
            step = 1, left = o.b1 - 1, inc = 1;
            first = (int64_t)(local / per) * s.ld;
            n = (int)((o.bcols + 127) / 128);
        } else {
            blk = split(o.b1, o.bcols, fixed_at, &local);
            step = o.b1, left = o.b0 - 1, inc = s.ld;
            first = local / per;
            n = (int)((o.brows + 127) / 128);
        }
        i = 0;
        p = s.at[blk];
    }
    // The scale `off` places from the next one (another row's), and on to the
    // next k-block.
    __device__ __forceinline__ float peek(int64_t off, int *status) const {
        const int64_t at = first + i * inc + off;
        return in && in_bounds(status, at, 1, t->n) ? __ldg(p + at) : 0.0f;
    }
    // From the start to k-block kb.
    __device__ __forceinline__ void seek(int kb) {
        while (left > 0 && kb >= n) {
            kb -= n;
            blk += step;
            --left;
        }
        p = t->at[blk];
        i = kb;
    }
    __device__ __forceinline__ void step_on() {
        if (++i == n && left > 0) {
            i = 0;
            blk += step;
            --left;
            p = t->at[blk];
        }
    }
    __device__ __forceinline__ float next(int *status) {
        const float v = peek(0, status);
        step_on();
        return v;
    }
};

// One k-block of an operand tile (128 rows or columns of the result, 16 KB)
// into shared memory.  K-major: one box, a row of 128 bytes per row of the
// result.  MN-major: a row per contracted index, 128 bytes of the result's dim
// per box (two boxes of 64 bf16 values, one of 128 bytes).
template <bool MN, bool F8>
__device__ __forceinline__ void load_box(const Cursor &c, uint32_t dst, uint32_t bar) {
    if (!MN) {
        shmm_pair::tma_load_2d_pair(dst, c.map, bar, c.at, c.fixed);
    } else if (F8) {
        shmm_pair::tma_load_2d_pair(dst, c.map, bar, c.fixed, c.at);
    } else {
        shmm_pair::tma_load_2d_pair(dst, c.map, bar, c.fixed, c.at);
        shmm_pair::tma_load_2d_pair(dst + 8192, c.map, bar, c.fixed + 64, c.at);
    }
}

// Matrix descriptor of MMA step kk (32 bytes of the contracted dim) of such a
// tile.  K-major: 32 bytes along the swizzled row, 8-row groups 1024 bytes
// apart.  MN-major: 16 (bf16) or 32 (8 bits) contracted rows, 128 bytes each,
// 8-row groups 1024 bytes apart, the second 64 bf16 columns 8192 bytes on.
template <bool MN, bool F8>
__device__ __forceinline__ uint64_t operand_step(uint32_t addr, int kk) {
    if (!MN) return shmm_pair::smem_desc(addr + (uint32_t)(kk * 32), 16, 1024);
    if (F8) return shmm_pair::smem_desc(addr + (uint32_t)(kk * 4096), 16384, 1024);
    return shmm_pair::smem_desc(addr + (uint32_t)(kk * 2048), 8192, 1024);
}

// TMEM columns of this warp's 32 lanes, read and waited for in one statement:
// nothing that uses the registers can move before the wait.
__device__ __forceinline__ void tmem_read64(uint32_t at, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
        " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31,"
        " %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47,"
        " %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
        "\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(at)
        : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// A wait by a whole warp, with an answer that is the same for all its lanes (and
// known to be): an MMA issuer's loop stays uniform, its descriptors in uniform
// registers, where tcgen05.mma takes them from.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *status) {
    return __all_sync(0xFFFFFFFFu, shmm_dev::mbar_wait(bar, parity, abort_flag, status));
}

__device__ __forceinline__ void st_shared_v4(uint32_t at, const uint32_t *w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

// Row r of a 32 x 32 result box into shared memory, as the result's tensor maps
// declare it: bf16 rows are 64 bytes, 64-byte swizzle; fp32 rows 128 bytes,
// 128-byte swizzle.
__device__ __forceinline__ void stage_bf16_row(uint32_t at, int r, const float *v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        st_shared_v4(at + (uint32_t)(r * 64 + ((j ^ ((r >> 1) & 3)) * 16)), w);
    }
}
__device__ __forceinline__ void stage_f32_row(uint32_t at, int r, const float *v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t w[4] = {__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                               __float_as_uint(v[4 * j + 3])};
        st_shared_v4(at + (uint32_t)(r * 128 + ((j ^ (r & 7)) * 16)), w);
    }
}

int launch_pair(ContractK &k, int form, int max_sms, cudaStream_t s);
int launch_small(ContractK &k, int form, int sms, cudaStream_t s);
int small_parts(int form, int64_t M, int64_t N, int64_t Kd, int terms, bool two, int sms);

}  // namespace shmm_tcn
