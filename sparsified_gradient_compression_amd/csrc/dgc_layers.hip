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

constexpr int64_t kCUs = 256;  // compute units of an MI355X
constexpr size_t kPad = 256;

size_t round_up(size_t x) { return (x + kPad - 1) / kPad * kPad; }

}  // namespace

Cut plan_product(int form, int64_t m, int64_t n, int64_t k, int parts, bool direct) {
    Cut c;
    const int64_t outs = form == kDw ? parts : 1;
    const int64_t steps = cdiv64(k, 64) * (form == kDx ? parts : 1);
    const int64_t wide = form == kPair ? 2 * n : n;
    const auto tiles = [&](int tile) {
        const TileSize t = tile_size(tile);
        return cdiv64(m, t.m) * cdiv64(wide, t.n) * outs;
    };
    if (direct && tiles(kBig256) >= kCUs / 2)
        c.tile = kBig256;
    else if (tiles(kGuarded128) >= kCUs)
        c.tile = direct ? kT128w8 : kGuarded128;
    else
        c.tile = direct ? (steps >= 8 ? kMid64x2 : kMid64) : kGuarded64;
    // too few tiles for the chip: cut the long axis, at least 4 steps each
    const int64_t have = tiles(c.tile);
    int64_t splits = 1;
    if (have > 0 && have < kCUs && c.tile != kBig256)
        splits = std::min(cdiv64(2 * kCUs, have), steps / 4);
    splits = std::max<int64_t>(splits, 1);
    c.per = std::max<int64_t>(cdiv64(steps, splits), 1);
    c.splits = int(std::max<int64_t>(cdiv64(steps, c.per), 1));
    return c;
}

size_t product_bytes(int form, int64_t m, int64_t n, int64_t k, int parts) {
    const int64_t planes = form == kPair ? 2 : form == kDw ? parts : 1;
    int64_t splits = 1;
    for (const bool direct : {false, true})
        splits = std::max<int64_t>(splits, plan_product(form, m, n, k, parts, direct).splits);
    if (splits == 1) return 0;
    return round_up(size_t(splits) * size_t(planes) * size_t(m) * size_t(n) * 4);
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

// Workspace of a gradient call: [slope outputs][column sums][a product's sums].
struct Space {
    size_t dz = 0, sums = 0, part = 0, total = 0;
};

Space linear_backward_space(int64_t m, int64_t n, int64_t k) {
    Space s;
    s.sums = round_up(size_t(m) * size_t(pad8(n)) * 2);
    s.part = s.sums + round_up(size_t(cdiv64(m, kSumRows)) * size_t(n) * 4);
    s.total = s.part + std::max(product_bytes(kDx, m, k, n, 1), product_bytes(kDw, n, k, m, 1));
    return s;
}

Space ffn_backward_space(int64_t m, int64_t d, int64_t f) {
    Space s;
    s.part = 2 * round_up(size_t(m) * size_t(pad8(f)) * 2);
    s.total = s.part + std::max(product_bytes(kDx, m, d, f, 2), product_bytes(kDw, f, d, m, 2));
    return s;
}

int run_product(int64_t type, const Product& p, void* ws, hipStream_t s) {
    return type == DGC_BF16 ? Launch<__bf16>::product(p, ws, s)
                            : Launch<_Float16>::product(p, ws, s);
}

}  // namespace
}  // namespace layers
}  // namespace dgc

extern "C" {

int dgc_linear_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t backward, size_t* bytes) {
    if (!bytes || !sizes_ok(m, n, k)) return DGC_EINVAL;
    *bytes = backward ? linear_backward_space(m, n, k).total : product_bytes(kRows, m, n, k, 1);
    return DGC_OK;
}

int dgc_gated_ffn_workspace_bytes(int64_t m, int64_t d, int64_t f, int32_t backward,
                                  size_t* bytes) {
    if (!bytes || !sizes_ok(m, d, f)) return DGC_EINVAL;
    *bytes = backward ? ffn_backward_space(m, d, f).total : product_bytes(kPair, m, f, d, 1);
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
    const int rc = space_ok(workspace, workspace_bytes, product_bytes(kRows, a->m, a->n, a->k, 1));
    if (rc != DGC_OK) return rc;
    Product p;
    p.form = kRows;
    p.m = a->m;
    p.n = a->n;
    p.k = a->k;
    p.a[0] = {a->x, a->ldx};
    p.b[0] = {a->w, a->ldw};
    p.fin.out[0] = a->y;
    p.fin.ldo = a->ldy;
    p.fin.bias = a->bias;
    p.fin.residual = a->residual;
    p.fin.ldr = a->ldr;
    p.fin.pre[0] = a->pre;
    p.fin.ldp[0] = a->ldpre;
    p.fin.act = int32_t(a->act);
    return run_product(a->type, p, workspace, stream);
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
    const Space sp = linear_backward_space(m, n, k);
    int rc = space_ok(workspace, workspace_bytes, sp.total);
    if (rc != DGC_OK) return rc;
    char* ws = static_cast<char*>(workspace);
    Mat dz{a->dy, a->lddy};
    if (sloped) dz = {ws, pad8(n)};
    const bool half_type = a->type == DGC_BF16;
    rc = (half_type ? Launch<__bf16>::slope : Launch<_Float16>::slope)(
        m, n, {a->dy, a->lddy}, {sloped ? a->pre : nullptr, a->ldpre}, int(a->act),
        sloped && (a->dx || a->dw) ? ws : nullptr, pad8(n), a->dbias, wide,
        reinterpret_cast<float*>(ws + sp.sums), stream);
    if (rc != DGC_OK) return rc;
    Product p;
    if (a->dx) {
        p.form = kDx;
        p.m = m;
        p.n = k;
        p.k = n;
        p.a[0] = dz;
        p.b[0] = {a->w, a->ldw};
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
        p.b[0] = {a->x, a->ldx};
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
    const int rc = space_ok(workspace, workspace_bytes, product_bytes(kPair, m, f, d, 1));
    if (rc != DGC_OK) return rc;
    Product p;
    p.form = kPair;
    p.m = m;
    p.n = f;
    p.k = d;
    p.a[0] = {a->x, a->ldx};
    p.b[0] = {a->w_gate, a->ldw_gate};
    p.b[1] = {a->w_up, a->ldw_up};
    p.fin.out[0] = a->h;
    p.fin.ldo = a->ldh;
    p.fin.pre[0] = a->gate;
    p.fin.ldp[0] = a->ldgate;
    p.fin.pre[1] = a->up;
    p.fin.ldp[1] = a->ldup;
    p.fin.act = int32_t(a->act);
    return run_product(a->type, p, workspace, stream);
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
    const Space sp = ffn_backward_space(m, d, f);
    int rc = space_ok(workspace, workspace_bytes, sp.total);
    if (rc != DGC_OK) return rc;
    if (!a->dx && !a->dw_gate) return DGC_OK;
    char* ws = static_cast<char*>(workspace);
    const int64_t ld = pad8(f);
    void *da = ws, *db = ws + sp.part / 2;
    rc = (a->type == DGC_BF16 ? Launch<__bf16>::gate_slope : Launch<_Float16>::gate_slope)(
        m, f, {a->dh, a->lddh}, {a->gate, a->ldgate}, {a->up, a->ldup}, int(a->act), da, db, ld,
        stream);
    if (rc != DGC_OK) return rc;
    Product p;
    p.parts = 2;
    p.a[0] = {da, ld};
    p.a[1] = {db, ld};
    if (a->dx) {
        p.form = kDx;
        p.m = m;
        p.n = d;
        p.k = f;
        p.b[0] = {a->w_gate, a->ldw_gate};
        p.b[1] = {a->w_up, a->ldw_up};
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
        p.b[0] = {a->x, a->ldx};
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
