// layers_launch.hpp -- how a product of the layer operators is launched; the
// element type's source file instantiates it.
#pragma once

#include <algorithm>
#include <type_traits>

#include "layers_big.hpp"
#include "layers_guarded.hpp"
#include "layers_mid.hpp"
#include "layers_thin.hpp"
#include "layers_tile.hpp"

namespace dgc {
namespace layers {

#define DGC_LAYERS_CHECK() \
    if (hipGetLastError() != hipSuccess) return DGC_EHIP

template <class T, int FORM, bool SPLIT>
int launch_tiles(const TileArgs& a, const Cut& c, hipStream_t s) {
    const int64_t blocks = a.mt * a.nt * (FORM == kDw ? a.parts : 1) * c.splits;
    if (blocks > 0x7FFFFFFF) return DGC_EINVAL;
    const auto grid = [=](int threads) { return grid_of(blocks, threads); };
    switch (c.tile) {
        case kGuarded: k_guarded<T, FORM, SPLIT><<<grid(kGuardedThreads), kGuardedThreads, 0, s>>>(a); break;
        case kMid32: k_mid<T, FORM, Shape32, SPLIT><<<grid(1024), 1024, 0, s>>>(a); break;
        case kMid64: k_mid<T, FORM, Shape64, SPLIT><<<grid(512), 512, 0, s>>>(a); break;
        case kLight: k_mid<T, FORM, ShapeLight, SPLIT><<<grid(256), 256, 0, s>>>(a); break;
        case kMid128: k_mid<T, FORM, Shape128, SPLIT><<<grid(512), 512, 0, s>>>(a); break;
        case kPair128: k_mid<T, FORM, ShapePair, SPLIT><<<grid(512), 512, 0, s>>>(a); break;
        case kBig: k_big<T, FORM, SPLIT><<<grid(512), 512, 0, s>>>(a); break;
        default:
            if constexpr (FORM == kRows || FORM == kPair) {
                const dim3 rows = grid_of(cdiv64(a.N, 16), 512);
                if (a.M <= 16)
                    k_thin<T, FORM == kPair, 1><<<rows, 512, 0, s>>>(a);
                else
                    k_thin<T, FORM == kPair, 2><<<rows, 512, 0, s>>>(a);
            }
    }
    DGC_LAYERS_CHECK();
    return DGC_OK;
}

inline TileArgs tile_args(const Product& p, const Cut& c, void* ws) {
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
    a.pieces = p.pieces;
    a.inverse = uint32_t((0x80000000u + uint32_t(p.pieces) - 1) / uint32_t(p.pieces));
    a.low = p.low;
    a.fold = p.fold;
    a.part = c.splits > 1 ? static_cast<float*>(ws) : nullptr;
    a.fin = p.fin;
    return a;
}

template <class T>
int Launch<T>::product(const Product& p, const Cut& c, void* ws, hipStream_t s) {
    if (p.m == 0 || p.n == 0) return DGC_OK;
    const TileArgs a = tile_args(p, c, ws);
    int rc = DGC_EINVAL;
    switch (p.form) {
        case kRows: rc = launch_tiles<T, kRows, false>(a, c, s); break;
        case kPair: rc = launch_tiles<T, kPair, false>(a, c, s); break;
        case kDx:
            rc = a.pieces > 1 ? launch_tiles<T, kDx, true>(a, c, s)
                              : launch_tiles<T, kDx, false>(a, c, s);
            break;
        case kDw:
            rc = a.pieces > 1 ? launch_tiles<T, kDw, true>(a, c, s)
                              : launch_tiles<T, kDw, false>(a, c, s);
            break;
    }
    if (rc != DGC_OK || c.splits == 1) return rc;
    const int64_t blocks = cdiv64(cdiv64(p.n, 4) * p.m * a.outs, 64);
    if (blocks > 0x7FFFFFFF) return DGC_EINVAL;
    if (p.form == kPair)
        k_join<T, true><<<grid_of(blocks, 64), 64, 0, s>>>(a);
    else
        k_join<T, false><<<grid_of(blocks, 64), 64, 0, s>>>(a);
    DGC_LAYERS_CHECK();
    return DGC_OK;
}

template <class T, bool SPLIT>
int launch_both(const TileArgs& x, const TileArgs& w, int tile, const Sums& sums, hipStream_t s) {
    const int64_t nx = x.mt * x.nt, nw = w.mt * w.nt * w.parts;
    const int64_t blocks = (nx + 7) / 8 * 8 + nw + (sums.out ? cdiv64(sums.N, 32) : 0);
    if (blocks > 0x7FFFFFFF) return DGC_EINVAL;
    if (blocks == 0) return DGC_OK;
    const auto grid = [=](int threads) { return grid_of(blocks, threads); };
    switch (tile) {
        case kGuarded:
            k_guarded_both<T, SPLIT><<<grid(kGuardedThreads), kGuardedThreads, 0, s>>>(x, w, int(nx), int(nw), sums);
            break;
        case kMid32: k_mid_both<T, Shape32, SPLIT><<<grid(1024), 1024, 0, s>>>(x, w, int(nx), int(nw), sums); break;
        case kMid64: k_mid_both<T, Shape64, SPLIT><<<grid(512), 512, 0, s>>>(x, w, int(nx), int(nw), sums); break;
        case kLight: k_mid_both<T, ShapeLight, SPLIT><<<grid(256), 256, 0, s>>>(x, w, int(nx), int(nw), sums); break;
        case kMid128: k_mid_both<T, Shape128, SPLIT><<<grid(512), 512, 0, s>>>(x, w, int(nx), int(nw), sums); break;
        case kPair128: k_mid_both<T, ShapePair, SPLIT><<<grid(512), 512, 0, s>>>(x, w, int(nx), int(nw), sums); break;
        default: return DGC_EINVAL;
    }
    DGC_LAYERS_CHECK();
    return DGC_OK;
}

template <class T>
int Launch<T>::both(const Product& dx, const Product& dw, int tile, const Sums& sums,
                    hipStream_t s) {
    Cut c;
    c.tile = tile;
    c.per = cdiv64(dx.k, kStep) * dx.parts * dx.pieces;
    const TileArgs x = tile_args(dx, c, nullptr);
    c.per = cdiv64(dw.k, kStep) * dw.pieces;
    const TileArgs w = tile_args(dw, c, nullptr);
    return x.pieces > 1 || w.pieces > 1 ? launch_both<T, true>(x, w, tile, sums, s)
                                        : launch_both<T, false>(x, w, tile, sums, s);
}

template <class T>
int Launch<T>::prepare(SlopeArgs a, const Repack& r, hipStream_t s) {
    int64_t slopes = 0, pieces = 0;
    if (a.M > 0 && a.N > 0)
        slopes = a.up ? cdiv64(a.ldz / a.per * a.M, 256) : cdiv64(a.N, 512) * cdiv64(a.M, a.per);
    for (int i = 0; i < r.count; ++i) pieces += r.rows[i] * cdiv64(r.cols[i], 8);
    const int64_t blocks = slopes + cdiv64(pieces, 256);
    if (blocks > 0x7FFFFFFF) return DGC_EINVAL;
    if (blocks == 0) return DGC_OK;
    if constexpr (std::is_same_v<T, _Float16>) {
        if (a.most && slopes > 0) {
            int across = 1;
            while (across < 256 && across * 8 < a.N) across *= 2;
            a.parts = int32_t(std::min<int64_t>(kMostParts, cdiv64(a.M, 256 / across)));
            k_most<T><<<dim3(unsigned(a.parts)), 256, 0, s>>>(a, across);
            DGC_LAYERS_CHECK();
        }
    }
    auto kernel = a.pieces == 1 ? k_prepare<T, 1> : k_prepare<T, 2>;
    if constexpr (!std::is_same_v<T, _Float16>)
        if (a.pieces == 3) kernel = k_prepare<T, 3>;
    kernel<<<grid_of(blocks, 256), 256, 0, s>>>(a, slopes, r);
    DGC_LAYERS_CHECK();
    return DGC_OK;
}

template <class T>
int Launch<T>::sum(const Sums& a, hipStream_t s) {
    if (!a.out || a.N == 0) return DGC_OK;
    k_sum_columns<T><<<grid_of(cdiv64(a.N, 32), 256), 256, 0, s>>>(a);
    DGC_LAYERS_CHECK();
    return DGC_OK;
}

}  // namespace layers
}  // namespace dgc
