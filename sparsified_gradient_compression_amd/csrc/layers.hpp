// layers.hpp -- what the host side of the layer operators and their kernels
// share: operand and epilogue descriptions and the launchers' declarations.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "dgc.h"

namespace dgc {
namespace layers {

// A matrix in device memory: rows of `ld` elements, the columns contiguous.
struct Mat {
    const void* p = nullptr;
    int64_t ld = 0;
};

// How an output is finished from the 32-bit sums of its product.
struct Finish {
    void* out[2] = {nullptr, nullptr};  // y | h | dx | dw (the second of two products)
    int64_t ldo = 0, ldo2 = 0;          // ldo2: the second product's output
    const void* bias = nullptr;         // [n] or null
    const void* residual = nullptr;     // [m][n] or null
    int64_t ldr = 0;
    void* pre[2] = {nullptr, nullptr};  // z | gate, up; or null
    int64_t ldp[2] = {0, 0};
    int32_t act = 0;
    int32_t wide = 0;  // outputs in binary32
};

// What a product's operands look like.
//   kRows:  out[m][n] = sum_k a[m][k] b[n][k]               (a layer's output)
//   kPair:  the same for two b at once, joined in the finish (the gated block)
//   kDx:    out[m][n] = sum_s sum_k a_s[m][k] b_s[k][n]     (one or two terms)
//   kDw:    out_s[m][n] = sum_k a_s[k][m] b[k][n]           (one or two outputs)
enum Form { kRows = 0, kPair = 1, kDx = 2, kDw = 3 };

struct Product {
    int form = kRows;
    int64_t m = 0, n = 0, k = 0;
    int parts = 1;  // terms of kDx, outputs of kDw
    Mat a[2], b[2];
    Finish fin;
};

// The kernels: guarded and thin ones take any strides and alignment, the
// others rows on 16 bytes.
enum Tile {
    kGuarded64, kGuarded128, kThin,
    kMid64, kMid64x2, kBig256,
    kT64k2s2, kT64k4, kT128s2, kT128w8, kT128x64, kT32x64, kT64x128, kT128w8s2, kT64x32
};

struct TileSize { int m, n; };
inline TileSize tile_size(int t) {
    switch (t) {
        case kBig256: return {256, 256};
        case kGuarded128: case kT128s2: case kT128w8: case kT128w8s2: return {128, 128};
        case kThin: return {64, 16};
        case kT128x64: return {128, 64};
        case kT64x128: return {64, 128};
        case kT32x64: return {32, 64};
        case kT64x32: return {64, 32};
        default: return {64, 64};
    }
}

// Which kernel, and the split of a product over its long axis: `splits`
// workgroups per tile, each over `per` steps of 64; their 32-bit sums meet in
// the workspace.
struct Cut {
    int tile = kGuarded64;
    int splits = 1;
    int64_t per = 0;
};

// From the sizes, and whether the operands' rows lie on 16 bytes.
Cut plan_product(int form, int64_t m, int64_t n, int64_t k, int parts, bool direct);
// The workspace of either, from the sizes alone.
size_t product_bytes(int form, int64_t m, int64_t n, int64_t k, int parts);

// The launchers, for DGC_BF16 and DGC_FP16 elements.  Each returns a DGC_* code.
template <class T>
struct Launch {
    static int product(const Product& p, void* ws, hipStream_t s);
    // dz = dy * act'(pre) (dz null: not written), and the column sums of dz
    // into dbias (null: none) through `part`.
    static int slope(int64_t m, int64_t n, Mat dy, Mat pre, int act, void* dz, int64_t ldz,
                     void* dbias, int wide, float* part, hipStream_t s);
    // da = dh * up * act'(gate), db = dh * act(gate)
    static int gate_slope(int64_t m, int64_t f, Mat dh, Mat gate, Mat up, int act, void* da,
                          void* db, int64_t ld, hipStream_t s);
};

constexpr int64_t kSumRows = 128;  // rows per block of a column sum

inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace layers
}  // namespace dgc
