// dgc_layers.hip -- host side of the layer operators: argument checks, the
// split of each product, workspace carving and launch order.  See
// include/dgc.h for the contract of every function.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "layers.hpp"

using namespace dgc::layers;

namespace dgc {
namespace layers {

namespace {

constexpr size_t kPad = 256;

size_t round_up(size_t x) { return (x + kPad - 1) / kPad * kPad; }

}  // namespace

namespace {

// What a kernel takes, measured on bf16 products of 64 to 8192 rows and
// columns: a start, and so many microseconds per step of 64 of k for a round
// of at most `round` workgroups, of which `light` or fewer have a compute unit
// each to themselves.
//   e.g. 333 x 1152 x 3456: kMid32 11.6, kMid64 13.6, kMid128 26.9 us;
//   777 x 1000 x 2048: kMid32 14.5, kMid64 9.1, kMid128 17.0;
//   2048 x 2048 x 2048: kMid64 34.3, kMid128 21.3, kPair128 28.5, kBig 46.5;
//   2048 x 4096 x 2048: kMid128 41.5, kPair128 36.0, kBig 48.1;
//   4096 x 4096 x 4096: kPair128 149, kBig 99
struct Cost {
    int tile;
    int64_t round, light;
    double start, full_step, light_step;
};
constexpr Cost kCosts[] = {{kGuarded, 512, 256, 3.0, 0.85, 0.66}, {kMid32, 256, 256, 2.5, 0.17, 0.17},
                           {kMid64, 256, 256, 2.5, 0.24, 0.24},   {kMid128, 256, 256, 3.0, 0.62, 0.62},
                           {kPair128, 512, 256, 3.0, 1.08, 0.80}, {kBig, 256, 256, 5.0, 1.50, 1.50}};

// A second launch that adds the splits' sums, and its traffic.
double join_us(double bytes) { return 6.0 + bytes / 3e6; }

}  // namespace

Cut plan_product(int form, int64_t m, int64_t n, int64_t k, int parts, bool direct) {
    const int64_t outs = form == kDw ? parts : 1;
    const int64_t steps = std::max<int64_t>(cdiv64(k, 64) * (form == kDx ? parts : 1), 1);
    const int64_t wide = form == kPair ? 2 * n : n;
    Cut best;
    best.us = 1e30;
    // few rows: reading the weight is all there is to it (1 x 4096 x 4096: kThin
    // 7.2, kMid32 10.7 us; 30 rows 13.0 and 11.8, 64 rows 20.8 and 12.2).  Where
    // rows do not lie on 16 bytes it is worth twice the time.
    if ((form == kRows || form == kPair) && m <= (direct ? 16 : 64)) {
        best.tile = kThin;
        best.per = steps;
        best.us = 0;
        return best;
    }
    for (const Cost& c : kCosts) {
        if ((c.tile == kGuarded) == direct) continue;
        const TileSize t = kTileSize[c.tile];
        const int64_t tiles = cdiv64(m, t.m) * cdiv64(wide, t.n) * outs;
        for (int64_t splits = 1; splits <= 8; splits *= 2) {
            // a split keeps 8 steps, and only fills up a round
            if (splits > 1 && (steps < 8 * splits || tiles * splits > c.round)) break;
            const int64_t per = cdiv64(steps, splits), work = tiles * splits;
            const int64_t rest = work % c.round;
            double us = double(work / c.round) * c.full_step;
            if (rest > 0) us += rest <= c.light ? c.light_step : c.full_step;
            us = c.start + us * double(per);
            if (splits > 1)
                us += join_us(8.0 * double(splits) * double(m) * double(wide) * double(outs));
            if (us < best.us) {
                best.tile = c.tile;
                best.per = per;
                best.splits = int(cdiv64(steps, per));
                best.us = us;
            }
        }
    }
    return best;
}

namespace {

// Sizes whose products of two stay far from 2^63 bytes.
constexpr int64_t kMostSide = int64_t(1) << 40;
constexpr int64_t kMostArea = int64_t(1) << 52;

bool sizes_ok(int64_t m, int64_t n, int64_t k) {
    for (int64_t v : {m, n, k})
        if (v < 0 || v > kMostSide) return false;
    const auto fits = [](int64_t a, int64_t b) { return b == 0 || a <= kMostArea / b; };
    return fits(m, n) && fits(m, k) && fits(n, k);
}

bool half(int64_t type) { return type == DGC_BF16 || type == DGC_FP16; }

bool act_ok(int64_t act) { return act >= DGC_ACT_NONE && act <= DGC_ACT_GELU_TANH; }

// A matrix of rows x cols: present where it has elements, aligned to its
// elements, its rows not overlapping.
bool mat_ok(const void* p, int64_t ld, int64_t rows, int64_t cols, int size) {
    if (rows == 0 || cols == 0) return true;
    return p && reinterpret_cast<uintptr_t>(p) % size == 0 && ld >= cols &&
           ld <= kMostArea / rows;
}

bool optional_ok(const void* p, int64_t ld, int64_t rows, int64_t cols, int size) {
    return !p || mat_ok(p, ld, rows, cols, size);
}

int space_ok(const void* ws, size_t have, size_t need) {
    if (need == 0) return DGC_OK;
    if (!ws || reinterpret_cast<uintptr_t>(ws) % kPad != 0) return DGC_EINVAL;
    return have < need ? DGC_ECAPACITY : DGC_OK;
}

int64_t pad8(int64_t x) { return (x + 7) / 8 * 8; }

// A product's splits, in the workspace.
size_t part_bytes(int form, int64_t m, int64_t n, int64_t k, int parts) {
    const int64_t planes = form == kPair ? 2 : form == kDw ? parts : 1;
    size_t most = 0;
    for (const bool d : {false, true}) {
        const Cut c = plan_product(form, m, n, k, parts, d);
        if (c.splits > 1)
            most = std::max(most, size_t(c.splits) * size_t(planes) * size_t(m) * size_t(n) * 4);
    }
    return round_up(most);
}

// Whether a product whose operands (`elements` of them) do not lie on 16 bytes
// gains from laying them out anew first: a launch and twice their bytes.
bool worth_repacking(int form, int64_t m, int64_t n, int64_t k, int parts, int64_t elements) {
    const Cut as_is = plan_product(form, m, n, k, parts, false);
    if (as_is.tile == kThin) return false;
    return plan_product(form, m, n, k, parts, true).us + 3.0 + 4.0 * double(elements) / 3e6 <
           as_is.us;
}

size_t row_bytes(int64_t rows, int64_t cols) {
    return round_up(size_t(rows) * size_t(pad8(cols)) * 2);
}

// Where a call keeps what it lays out: dz (da, db), column sums, operands that
// are repacked, and splits.  From the sizes alone.
struct Space {
    bool pack = false;
    size_t dz = 0, sums = 0, x = 0, w = 0, w2 = 0, part = 0, total = 0;
};

Space space(bool gated, bool backward, int64_t m, int64_t n, int64_t k) {
    const int two = gated ? 2 : 1;
    const int64_t weights = two * n * k;
    Space s;
    size_t at = 0, part = 0;
    const auto take = [&](size_t bytes) {
        const size_t was = at;
        at += bytes;
        return was;
    };
    if (backward) {
        s.dz = take(two * row_bytes(m, n));
        s.sums = take(gated ? 0 : round_up(size_t(cdiv64(m, sum_rows(m, n))) * size_t(n) * 4));
        s.pack = worth_repacking(kDx, m, k, n, two, weights) ||
                 worth_repacking(kDw, n, k, m, two, m * k);
        part = std::max(part_bytes(kDx, m, k, n, two), part_bytes(kDw, n, k, m, two));
    } else {
        s.pack = worth_repacking(gated ? kPair : kRows, m, n, k, 1, weights + m * k);
        part = part_bytes(gated ? kPair : kRows, m, n, k, 1);
    }
    if (s.pack) {
        s.x = take(row_bytes(m, k));
        s.w = take(row_bytes(n, k));
        s.w2 = take(gated ? row_bytes(n, k) : 0);
    }
    s.part = take(part);
    s.total = at;
    return s;
}

// Notes a matrix that is to be laid out anew at `to`, and returns what to use.
Mat packed(Repack& r, bool pack, Mat a, int64_t rows, int64_t cols, void* to) {
    if (!pack || rows == 0 || cols == 0 || direct(a, cols)) return a;
    r.from[r.count] = a.p;
    r.to[r.count] = to;
    r.ld[r.count] = a.ld;
    r.rows[r.count] = rows;
    r.cols[r.count] = cols;
    ++r.count;
    return {to, pad8(cols), true};
}

// Rows at any even address to rows on 16 bytes, zeros up to their ends; one
// thread per 8 elements.
__global__ __launch_bounds__(256) void k_repack(Repack r) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    typedef u32x4 u32x4_any __attribute__((aligned(2), may_alias));
    int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (i >= r.count) return;
        const int64_t per = (r.cols[i] + 7) / 8, have = per * r.rows[i];
        if (id < have) {
            const int64_t row = id / per, col = (id - row * per) * 8;
            const uint16_t* p = static_cast<const uint16_t*>(r.from[i]) + row * r.ld[i] + col;
            u32x4 v;
            if (col + 8 <= r.cols[i]) {
                v = *reinterpret_cast<const u32x4_any*>(p);
            } else {
                uint16_t t[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = col + e < r.cols[i] ? p[e] : uint16_t(0);
                __builtin_memcpy(&v, t, 16);
            }
            reinterpret_cast<u32x4*>(r.to[i])[id] = v;
            return;
        }
        id -= have;
    }
}

int run_product(int64_t type, const Product& p, void* ws, hipStream_t s) {
    return type == DGC_BF16 ? Launch<__bf16>::product(p, ws, s)
                            : Launch<_Float16>::product(p, ws, s);
}

}  // namespace

int repack(const Repack& r, hipStream_t s) {
    if (r.count == 0) return DGC_OK;
    int64_t pieces = 0;
    for (int i = 0; i < r.count; ++i) pieces += r.rows[i] * ((r.cols[i] + 7) / 8);
    const int64_t blocks = cdiv64(pieces, 256);
    if (blocks > 0x7FFFFFFF) return DGC_EINVAL;
    k_repack<<<dim3(unsigned(blocks)), 256, 0, s>>>(r);
    return hipGetLastError() == hipSuccess ? DGC_OK : DGC_EHIP;
}

}  // namespace layers
}  // namespace dgc

extern "C" {

int dgc_linear_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t backward, size_t* bytes) {
    if (!bytes || !sizes_ok(m, n, k)) return DGC_EINVAL;
    *bytes = space(false, backward != 0, m, n, k).total;
    return DGC_OK;
}

int dgc_gated_ffn_workspace_bytes(int64_t m, int64_t d, int64_t f, int32_t backward,
                                  size_t* bytes) {
    if (!bytes || !sizes_ok(m, d, f)) return DGC_EINVAL;
    *bytes = space(true, backward != 0, m, f, d).total;
    return DGC_OK;
}

int dgc_linear(const dgc_linear_args* a, void* workspace, size_t workspace_bytes,
               hipStream_t stream) {
    if (!a || !half(a->type) || !act_ok(a->act) || !sizes_ok(a->m, a->n, a->k)) return DGC_EINVAL;
    if (!mat_ok(a->x, a->ldx, a->m, a->k, 2) || !mat_ok(a->w, a->ldw, a->n, a->k, 2) ||
        !optional_ok(a->bias, a->n, 1, a->n, 2) ||
        !optional_ok(a->residual, a->ldr, a->m, a->n, 2) ||
        !mat_ok(a->y, a->ldy, a->m, a->n, 2) || !optional_ok(a->pre, a->ldpre, a->m, a->n, 2))
        return DGC_EINVAL;
    const int64_t m = a->m, n = a->n, k = a->k;
    const Space sp = space(false, false, m, n, k);
    int rc = space_ok(workspace, workspace_bytes, sp.total);
    if (rc != DGC_OK) return rc;
    char* ws = static_cast<char*>(workspace);
    Repack r;
    Product p;
    p.form = kRows;
    p.m = m;
    p.n = n;
    p.k = k;
    p.a[0] = packed(r, sp.pack, {a->x, a->ldx}, m, k, ws + sp.x);
    p.b[0] = packed(r, sp.pack, {a->w, a->ldw}, n, k, ws + sp.w);
    rc = repack(r, stream);
    if (rc != DGC_OK) return rc;
    p.fin.out[0] = a->y;
    p.fin.ldo = a->ldy;
    p.fin.bias = a->bias;
    p.fin.residual = a->residual;
    p.fin.ldr = a->ldr;
    p.fin.pre[0] = a->pre;
    p.fin.ldp[0] = a->ldpre;
    p.fin.act = int32_t(a->act);
    return run_product(a->type, p, ws + sp.part, stream);
}

int dgc_linear_backward(const dgc_linear_backward_args* a, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
    if (!a || !half(a->type) || !act_ok(a->act) || !sizes_ok(a->m, a->n, a->k) ||
        (a->grad_type != a->type && a->grad_type != DGC_FP32))
        return DGC_EINVAL;
    const int64_t m = a->m, n = a->n, k = a->k;
    const int wide = a->grad_type == DGC_FP32;
    const bool sloped = a->act != DGC_ACT_NONE;
    if (!mat_ok(a->dy, a->lddy, m, n, 2) || !mat_ok(a->x, a->ldx, m, k, 2) ||
        !mat_ok(a->w, a->ldw, n, k, 2) || (sloped && !mat_ok(a->pre, a->ldpre, m, n, 2)) ||
        !optional_ok(a->dx, a->lddx, m, k, 2) ||
        !optional_ok(a->dw, a->lddw, n, k, wide ? 4 : 2) ||
        !optional_ok(a->dbias, n, 1, n, wide ? 4 : 2))
        return DGC_EINVAL;
    const Space sp = space(false, true, m, n, k);
    int rc = space_ok(workspace, workspace_bytes, sp.total);
    if (rc != DGC_OK) return rc;
    char* ws = static_cast<char*>(workspace);
    Repack r;
    Mat x{a->x, a->ldx}, w{a->w, a->ldw}, dz{a->dy, a->lddy};
    if (a->dw) x = packed(r, sp.pack, x, m, k, ws + sp.x);
    if (a->dx) w = packed(r, sp.pack, w, n, k, ws + sp.w);
    rc = repack(r, stream);
    if (rc != DGC_OK) return rc;
    // without an activation dz is dy, copied only where its rows do not lie on 16 bytes
    const bool copied = (a->dx || a->dw) && (sloped || (sp.pack && !direct(dz, n)));
    if (copied) dz = {ws + sp.dz, pad8(n), true};
    rc = (a->type == DGC_BF16 ? Launch<__bf16>::slope : Launch<_Float16>::slope)(
        m, n, {a->dy, a->lddy}, {sloped ? a->pre : nullptr, a->ldpre}, int(a->act),
        copied ? ws + sp.dz : nullptr, pad8(n), a->dbias, wide,
        reinterpret_cast<float*>(ws + sp.sums), stream);
    if (rc != DGC_OK) return rc;
    Product p;
    if (a->dx) {
        p.form = kDx;
        p.m = m;
        p.n = k;
        p.k = n;
        p.a[0] = dz;
        p.b[0] = w;
        p.fin.out[0] = a->dx;
        p.fin.ldo = a->lddx;
        rc = run_product(a->type, p, ws + sp.part, stream);
        if (rc != DGC_OK) return rc;
    }
    if (a->dw) {
        p.form = kDw;
        p.m = n;
        p.n = k;
        p.k = m;
        p.a[0] = dz;
        p.b[0] = x;
        p.fin.out[0] = a->dw;
        p.fin.ldo = a->lddw;
        p.fin.wide = wide;
        rc = run_product(a->type, p, ws + sp.part, stream);
    }
    return rc;
}

int dgc_gated_ffn(const dgc_gated_ffn_args* a, void* workspace, size_t workspace_bytes,
                  hipStream_t stream) {
    if (!a || !half(a->type) || !act_ok(a->act) || !sizes_ok(a->m, a->d, a->f)) return DGC_EINVAL;
    const int64_t m = a->m, d = a->d, f = a->f;
    if (!mat_ok(a->x, a->ldx, m, d, 2) || !mat_ok(a->w_gate, a->ldw_gate, f, d, 2) ||
        !mat_ok(a->w_up, a->ldw_up, f, d, 2) || !mat_ok(a->h, a->ldh, m, f, 2) ||
        !optional_ok(a->gate, a->ldgate, m, f, 2) || !optional_ok(a->up, a->ldup, m, f, 2))
        return DGC_EINVAL;
    const Space sp = space(true, false, m, f, d);
    int rc = space_ok(workspace, workspace_bytes, sp.total);
    if (rc != DGC_OK) return rc;
    char* ws = static_cast<char*>(workspace);
    Repack r;
    Product p;
    p.form = kPair;
    p.m = m;
    p.n = f;
    p.k = d;
    p.a[0] = packed(r, sp.pack, {a->x, a->ldx}, m, d, ws + sp.x);
    p.b[0] = packed(r, sp.pack, {a->w_gate, a->ldw_gate}, f, d, ws + sp.w);
    p.b[1] = packed(r, sp.pack, {a->w_up, a->ldw_up}, f, d, ws + sp.w2);
    rc = repack(r, stream);
    if (rc != DGC_OK) return rc;
    p.fin.out[0] = a->h;
    p.fin.ldo = a->ldh;
    p.fin.pre[0] = a->gate;
    p.fin.ldp[0] = a->ldgate;
    p.fin.pre[1] = a->up;
    p.fin.ldp[1] = a->ldup;
    p.fin.act = int32_t(a->act);
    return run_product(a->type, p, ws + sp.part, stream);
}

int dgc_gated_ffn_backward(const dgc_gated_ffn_backward_args* a, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
    if (!a || !half(a->type) || !act_ok(a->act) || !sizes_ok(a->m, a->d, a->f) ||
        (a->grad_type != a->type && a->grad_type != DGC_FP32))
        return DGC_EINVAL;
    const int64_t m = a->m, d = a->d, f = a->f;
    const int wide = a->grad_type == DGC_FP32, size = wide ? 4 : 2;
    if (!mat_ok(a->dh, a->lddh, m, f, 2) || !mat_ok(a->x, a->ldx, m, d, 2) ||
        !mat_ok(a->w_gate, a->ldw_gate, f, d, 2) || !mat_ok(a->w_up, a->ldw_up, f, d, 2) ||
        !mat_ok(a->gate, a->ldgate, m, f, 2) || !mat_ok(a->up, a->ldup, m, f, 2) ||
        !optional_ok(a->dx, a->lddx, m, d, 2) ||
        !optional_ok(a->dw_gate, a->lddw_gate, f, d, size) ||
        !optional_ok(a->dw_up, a->lddw_up, f, d, size) || !a->dw_gate != !a->dw_up)
        return DGC_EINVAL;
    const Space sp = space(true, true, m, f, d);
    int rc = space_ok(workspace, workspace_bytes, sp.total);
    if (rc != DGC_OK) return rc;
    if (!a->dx && !a->dw_gate) return DGC_OK;
    char* ws = static_cast<char*>(workspace);
    const int64_t ld = pad8(f);
    void *da = ws + sp.dz, *db = ws + sp.dz + row_bytes(m, f);
    Repack r;
    Mat x{a->x, a->ldx}, wg{a->w_gate, a->ldw_gate}, wu{a->w_up, a->ldw_up};
    if (a->dw_gate) x = packed(r, sp.pack, x, m, d, ws + sp.x);
    if (a->dx) {
        wg = packed(r, sp.pack, wg, f, d, ws + sp.w);
        wu = packed(r, sp.pack, wu, f, d, ws + sp.w2);
    }
    rc = repack(r, stream);
    if (rc != DGC_OK) return rc;
    rc = (a->type == DGC_BF16 ? Launch<__bf16>::gate_slope : Launch<_Float16>::gate_slope)(
        m, f, {a->dh, a->lddh}, {a->gate, a->ldgate}, {a->up, a->ldup}, int(a->act), da, db, ld,
        stream);
    if (rc != DGC_OK) return rc;
    Product p;
    p.parts = 2;
    p.a[0] = {da, ld, true};
    p.a[1] = {db, ld, true};
    if (a->dx) {
        p.form = kDx;
        p.m = m;
        p.n = d;
        p.k = f;
        p.b[0] = wg;
        p.b[1] = wu;
        p.fin.out[0] = a->dx;
        p.fin.ldo = a->lddx;
        rc = run_product(a->type, p, ws + sp.part, stream);
        if (rc != DGC_OK) return rc;
    }
    if (a->dw_gate) {
        p.form = kDw;
        p.m = f;
        p.n = d;
        p.k = m;
        p.b[0] = x;
        p.fin.out[0] = a->dw_gate;
        p.fin.ldo = a->lddw_gate;
        p.fin.out[1] = a->dw_up;
        p.fin.ldo2 = a->lddw_up;
        p.fin.wide = wide;
        rc = run_product(a->type, p, ws + sp.part, stream);
    }
    return rc;
}

}  // extern "C"
