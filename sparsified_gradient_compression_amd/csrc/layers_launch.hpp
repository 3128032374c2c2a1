// layers_launch.hpp -- how a product of the layer operators is launched; the
// element type's source file instantiates it.
#pragma once

#include "layers_big.hpp"
#include "layers_elem.hpp"
#include "layers_mid.hpp"
#include "layers_thin.hpp"
#include "layers_tile.hpp"

namespace dgc {
namespace layers {

#define DGC_LAYERS_CHECK() \
    if (hipGetLastError() != hipSuccess) return DGC_EHIP

inline bool direct(const Product& p) {
    const int64_t ca = p.form == kDw ? p.m : p.k, cb = p.form == kRows || p.form == kPair ? p.k : p.n;
    const bool two_a = p.form != kRows && p.form != kPair && p.parts == 2;
    const bool two_b = p.form == kPair || (p.form == kDx && p.parts == 2);
    if (!direct(p.a[0], ca) || !direct(p.b[0], cb)) return false;
    if (two_a && (!direct(p.a[1], ca) || p.a[1].ld != p.a[0].ld)) return false;
    return !two_b || (direct(p.b[1], cb) && p.b[1].ld == p.b[0].ld);
}

template <class T, int FORM>
int launch_tiles(const TileArgs& a, const Cut& c, hipStream_t s) {
    const int64_t blocks = a.mt * a.nt * (FORM == kDw ? a.parts : 1) * c.splits;
    if (blocks > 0x7FFFFFFF) return DGC_EINVAL;
    const dim3 grid(static_cast<unsigned>(blocks));
    switch (c.tile) {
        case kGuarded: k_tile<T, FORM, 64, 64, 2, 2><<<grid, 256, 0, s>>>(a); break;
        case kMid32: k_mid<T, FORM, 32, 64, 2, 2, 4, 3><<<grid, 1024, 0, s>>>(a); break;
        case kMid64: k_mid<T, FORM, 64, 64, 2, 2, 2, 4><<<grid, 512, 0, s>>>(a); break;
        case kMid128: k_mid<T, FORM, 128, 128, 2, 4, 1, 4><<<grid, 512, 0, s>>>(a); break;
        case kPair128: k_mid<T, FORM, 128, 128, 2, 4, 1, 2><<<grid, 512, 0, s>>>(a); break;
        case kBig: k_big<T, FORM><<<grid, 512, 0, s>>>(a); break;
        default:
            if constexpr (FORM == kRows || FORM == kPair) {
                const dim3 rows(static_cast<unsigned>(cdiv64(a.N, 16)));
                if (a.M <= 16)
                    k_thin<T, FORM == kPair, 1><<<rows, 512, 0, s>>>(a);
                else if (a.M <= 32)
                    k_thin<T, FORM == kPair, 2><<<rows, 512, 0, s>>>(a);
                else
                    k_thin<T, FORM == kPair, 4><<<rows, 512, 0, s>>>(a);
            }
    }
    DGC_LAYERS_CHECK();
    return DGC_OK;
}

template <class T>
int Launch<T>::product(const Product& p, void* ws, hipStream_t s) {
    if (p.m == 0 || p.n == 0) return DGC_OK;
    const Cut c = plan_product(p.form, p.m, p.n, p.k, p.parts, direct(p));
    const TileSize side = kTileSize[c.tile];
    TileArgs a{};
    for (int i = 0; i < 2; ++i) {
        a.a[i] = p.a[i].p;
        a.lda[i] = p.a[i].ld;
        a.b[i] = p.b[i].p;
        a.ldb[i] = p.b[i].ld;
    }
    a.M = p.m;
    a.N = p.n;
    a.K = p.k;
    a.mt = cdiv64(p.m, side.m);
    a.nt = cdiv64(p.n, p.form == kPair ? side.n / 2 : side.n);
    a.per = c.per;
    a.splits = c.splits;
    a.parts = p.parts;
    a.outs = p.form == kDw ? p.parts : 1;
    a.part = c.splits > 1 ? static_cast<float*>(ws) : nullptr;
    a.fin = p.fin;
    int rc = DGC_EINVAL;
    switch (p.form) {
        case kRows: rc = launch_tiles<T, kRows>(a, c, s); break;
        case kPair: rc = launch_tiles<T, kPair>(a, c, s); break;
        case kDx: rc = launch_tiles<T, kDx>(a, c, s); break;
        case kDw: rc = launch_tiles<T, kDw>(a, c, s); break;
    }
    if (rc != DGC_OK || c.splits == 1) return rc;
    const int64_t blocks = cdiv64(cdiv64(p.n, 4) * p.m * a.outs, 256);
    if (blocks > 0x7FFFFFFF) return DGC_EINVAL;
    if (p.form == kPair)
        k_join<T, true><<<dim3(unsigned(blocks)), 256, 0, s>>>(a);
    else
        k_join<T, false><<<dim3(unsigned(blocks)), 256, 0, s>>>(a);
    DGC_LAYERS_CHECK();
    return DGC_OK;
}

template <class T>
int Launch<T>::slope(int64_t m, int64_t n, Mat dy, Mat pre, int act, void* dz, int64_t ldz,
                     void* dbias, int wide, float* part, hipStream_t s) {
    if (n == 0 || (!dz && !dbias)) return DGC_OK;
    const int64_t per = sum_rows(m, n), rows = cdiv64(m, per);
    if (m > 0) {
        // grid.y holds at most 65535 blocks of rows
        const int64_t kMost = 65535;
        for (int64_t r = 0; r < rows; r += kMost) {
            const int64_t now = rows - r < kMost ? rows - r : kMost;
            const int64_t m0 = r * per;
            const int64_t left = m - m0 < now * per ? m - m0 : now * per;
            k_slope<T><<<dim3(unsigned(cdiv64(n, 512)), unsigned(now)), 256, 0, s>>>(
                left, n, per, static_cast<const T*>(dy.p) + m0 * dy.ld, dy.ld,
                pre.p ? static_cast<const T*>(pre.p) + m0 * pre.ld : nullptr, pre.ld, act,
                dz ? static_cast<T*>(dz) + m0 * ldz : nullptr, ldz,
                dbias ? part + r * n : nullptr);
            DGC_LAYERS_CHECK();
        }
    }
    if (dbias) {
        const dim3 grid(unsigned(cdiv64(n, 32)));
        if (wide)
            k_sum_columns<float><<<grid, 256, 0, s>>>(rows, n, part, static_cast<float*>(dbias));
        else
            k_sum_columns<T><<<grid, 256, 0, s>>>(rows, n, part, static_cast<T*>(dbias));
        DGC_LAYERS_CHECK();
    }
    return DGC_OK;
}

template <class T>
int Launch<T>::gate_slope(int64_t m, int64_t f, Mat dh, Mat gate, Mat up, int act, void* da,
                          void* db, int64_t ld, hipStream_t s) {
    const int64_t blocks = cdiv64(cdiv64(f, 8) * m, 256);
    if (blocks == 0) return DGC_OK;
    if (blocks > 0x7FFFFFFF) return DGC_EINVAL;
    k_gate_slope<T><<<dim3(unsigned(blocks)), 256, 0, s>>>(
        m, f, static_cast<const T*>(dh.p), dh.ld, static_cast<const T*>(gate.p), gate.ld,
        static_cast<const T*>(up.p), up.ld, act, static_cast<T*>(da), static_cast<T*>(db), ld);
    DGC_LAYERS_CHECK();
    return DGC_OK;
}

}  // namespace layers
}  // namespace dgc
