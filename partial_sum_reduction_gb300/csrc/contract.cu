// Which kernel takes a contraction of the gated MLP block or of 8-bit operands,
// and the tensor-core kernels' tables.

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>
#include <string>
#include <vector>

#include "contract_tc.cuh"
#include "shmm_internal.h"
#include "tensor_map.h"

namespace {

using namespace shmm_tcn;
using shmm::ContractArgs;
using shmm::GridOperand;
using shmm::GridResult;

bool on16(int64_t n, shmm_dtype_t dt) { return n * shmm::elem_bytes(dt) % 16 == 0; }

// Tiles cross no block's edge: where a dim is split, blocks are whole tiles of
// 128; rows are whole 16-byte pieces for TMA.
bool edges_fit(int b0, int b1, int64_t brows, int64_t bcols) {
    return (b0 == 1 || brows % 128 == 0) && (b1 == 1 || bcols % 128 == 0);
}
bool operand_fits(const GridOperand &o, bool few_rows = false) {
    if (o.at.size() > (size_t)kSlots || !on16(o.ld, o.dt)) return false;
    if (!edges_fit(few_rows ? 1 : o.b0, o.b1, o.brows, o.bcols)) return false;
    for (const void *p : o.at)
        if (reinterpret_cast<uintptr_t>(p) % 16) return false;
    return true;
}
size_t holders_of(const GridResult &d) {
    size_t n = 0;
    for (const auto &b : d.holders) n += b.size();
    return n;
}
bool result_fits(const GridResult &d, bool few_rows = false) {
    return d.holders.size() <= (size_t)kSlots && holders_of(d) <= (size_t)kSlots &&
           edges_fit(few_rows ? 1 : d.b0, d.b1, d.brows, d.bcols) && on16(d.bcols, d.dt);
}

int num_sms() {
    static shmm::PerDevice<int> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= shmm::kMaxDevices) return 148;
    int n = cache.get(dev);
    if (n) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    cache.set(dev, n);
    return n;
}

// Up to 128 rows, split over the ranks in whole groups of 8: the kernel for few
// rows puts the ranks' rows below one another (groups of 8 are what the
// swizzle of a tile repeats over).
bool rows_stack(const ContractArgs &a) {
    return !a.x_t && a.M <= 128 && a.X[0].b0 > 1 && a.X[0].brows % 8 == 0 && a.terms == 1;
}

// The tensor-core form of a contraction, or -1.
int form_of(const ContractArgs &a) {
    if (!a.tensor_core || a.M <= 0 || a.N <= 0 || a.Kd <= 0) return -1;
    if (a.M > (int64_t)1 << 30 || a.Kd > (int64_t)1 << 30) return -1;  // coordinates are 32-bit
    const int ny = a.gated || a.two || a.terms == 2 ? 2 : 1, nx = a.terms;
    const bool stack = rows_stack(a) && !(a.keep && a.kept[0].dt == SHMM_E4M3);
    for (int i = 0; i < nx; ++i)
        if (!operand_fits(a.X[i], stack)) return -1;
    for (int i = 0; i < ny; ++i)
        if (!operand_fits(a.Y[i])) return -1;
    for (int i = 0; i < (a.two ? 2 : 1); ++i)
        if (!result_fits(a.D[i], stack)) return -1;
    for (int i = 0; a.keep && i < 2; ++i)
        if (!result_fits(a.kept[i], stack)) return -1;
    const shmm_dtype_t in = a.X[0].dt;
    if (in == SHMM_BF16 && a.D[0].dt == SHMM_BF16) {
        if (a.gated) return a.keep && a.kept[0].dt == SHMM_E4M3 ? kGated8 : kGated;
        if (!a.x_t && a.y_t) return kNT;
        if (a.x_t && !a.y_t) return kTN;
    }
    if (in == SHMM_E4M3 && !a.x_t && a.terms == 1) return a.y_t ? kNT8 : kNN8;
    return -1;
}

// The kernel for few rows and small shapes, or CTA pairs.  (Kept 8-bit blocks of
// 128 columns need the pairs' tiles.)  Up to 128 rows would fill half a pair's
// tile at most.  Above, the small kernel's 128 x 128 tiles win where they leave
// at least half of its places free, so that two or more CTAs share a tile's
// contracted dim.  Measured, us, pairs / small: 515 x 1024 rows by 2 x 2816
// products (dA) 32 / 19 in four parts; 512 x 4096 by 2 x 4096 51 / 42 in two;
// 1024 x 4096 by 2 x 4096 54 / 71 in one; 8 bits, 256 x 4096 x 4096 23 / 17 in
// two, 512 x 4096 x 4096 23 / 25 in one.
bool use_small(const ContractArgs &a, int form, int sms) {
    if (form == kGated8) return false;
    return a.M <= 128 || small_parts(form, a.M, a.N, a.Kd, a.terms, a.two, sms) > 1;
}

struct Maps {
    ContractK *k;
    shmm::EncodeTiledFn fn;
    int n = 0;
    bool ok = true;
    void add(const void *base, int64_t rows, int64_t cols, int64_t ld, shmm_dtype_t dt, uint32_t bx, uint32_t by,
             CUtensorMapSwizzle sw) {
        if (n >= kMaps) ok = false;
        if (!ok) return;
        const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
        const cuuint64_t strides[1] = {(cuuint64_t)(ld * shmm::elem_bytes(dt))};
        const cuuint32_t box[2] = {bx, by}, estr[2] = {1, 1};
        const CUtensorMapDataType type = dt == SHMM_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                         : dt == SHMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                           : CU_TENSOR_MAP_DATA_TYPE_UINT8;
        ok = fn(&k->maps[n++], type, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    }
    // mn: the contracted dim runs along the rows.
    void operand(OpK *o, const GridOperand &g, bool mn, uint32_t rows = 128) {
        *o = {n, g.b0, g.b1, g.brows, g.bcols};
        const uint32_t row = 128 / (uint32_t)shmm::elem_bytes(g.dt);  // values of a 128-byte swizzled row
        for (const void *p : g.at)
            add(p, g.brows, g.bcols, g.ld, g.dt, row, mn ? row : rows, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    // Result boxes: 32 x 32 (fp32: 128-byte rows, bf16: 64), bytes 32 x 64.
    int holders(const GridResult &d) {
        const int at = n;
        const bool e8 = d.dt == SHMM_E4M3;
        for (const auto &b : d.holders)
            for (void *p : b)
                add(p, d.brows, d.bcols, d.bcols, d.dt, e8 ? 64 : 32, 32,
                    d.dt == SHMM_F32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
        return at;
    }
    void result(ResK *o, const GridResult &d, bool maps) {
        o->b0 = d.b0;
        o->b1 = d.b1;
        o->brows = d.brows;
        o->bcols = d.bcols;
        int h = 0;
        for (size_t p = 0; p < d.holders.size(); ++p) {
            o->first[p] = (uint8_t)h;
            h += (int)d.holders[p].size();
        }
        o->first[d.holders.size()] = (uint8_t)h;
        if (maps) o->map0 = holders(d);
    }
};

void set_scales(ScalesK *t, const GridOperand &g) {
    for (size_t i = 0; i < g.scale.size(); ++i) t->at[i] = g.scale[i];
    t->ld = g.scale_ld;
    t->n = (g.brows + g.scale_rows - 1) / g.scale_rows * g.scale_ld;
}

}  // namespace

namespace shmm {

int launch_contract(const ContractArgs &a, int *status, void *stream, std::string *msg) {
    const int form = form_of(a);
    if (form < 0) return launch_contract_simt(a, status, stream);
    const EncodeTiledFn fn = encode_fn(msg);
    if (!fn) return (int)cudaErrorNotSupported;
    static_assert(sizeof(ContractK) <= 32764, "kernel parameters");
    ContractK k;
    memset(&k, 0, sizeof k);
    Maps m = {&k, fn};
    const bool x_mn = form == kTN, y_mn = form == kGated || form == kGated8 || form == kTN || form == kNN8;
    const int sms = num_sms();  // whatever the plan's limit: which kernel and how many parts set the sums' order
    const bool small = use_small(a, form, sms);
    k.x_boxes = 1;
    k.x_rows = 128;
    if (small && !x_mn && a.M < 128) k.x_rows = (int)((a.M + 7) / 8 * 8);
    uint32_t box_rows = (uint32_t)k.x_rows;
    if (small && rows_stack(a)) {
        k.x_boxes = a.X[0].b0;
        box_rows = (uint32_t)a.X[0].brows;
    }
    for (int i = 0; i < a.terms; ++i) m.operand(&k.X[i], a.X[i], x_mn, box_rows);
    for (int i = 0; i < (a.gated || a.two ? 2 : a.terms); ++i) m.operand(&k.Y[i], a.Y[i], y_mn);
    auto buffers = [&](int at, const GridResult &d) {
        int h = 0;
        for (const auto &b : d.holders)
            for (void *p : b) k.out[at][h++] = p;
    };
    for (int i = 0; i < (a.two ? 2 : 1); ++i) {
        m.result(&k.D[i], a.D[i], !small);
        buffers(i, a.D[i]);
    }
    if (a.keep) {
        k.keep = a.kept[0].dt == SHMM_E4M3 ? 2 : 1;
        k.kept_ld = a.kept[0].scale_ld;
        for (int y = 0; y < 2; ++y) {
            if (!small) k.kept_map[y] = m.holders(a.kept[y]);
            buffers(2 + y, a.kept[y]);
            int h = 0;
            for (const auto &b : a.kept[y].scale_holders)
                for (float *p : b) k.kept_scale[y][h++] = p;
        }
    }
    if (!m.ok) {
        *msg = "cuTensorMapEncodeTiled rejected an operand or a result";
        return (int)cudaErrorInvalidValue;
    }
    if (form == kNN8 || form == kNT8) {
        set_scales(&k.x_scale, a.X[0]);
        set_scales(&k.y_scale, a.Y[0]);
    }
    k.M = a.M;
    k.N = a.N;
    k.Kd = a.Kd;
    k.terms = a.terms;
    k.two = a.two;
    k.act = a.act;
    k.out_f32 = a.D[0].dt == SHMM_F32;
    k.beside = a.beside;
    k.status = status;
    return small ? launch_small(k, form, sms, (cudaStream_t)stream) : launch_pair(k, form, a.max_sms, (cudaStream_t)stream);
}

}  // namespace shmm
