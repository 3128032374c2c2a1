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
// padded: its rows go on with zeros up to a multiple of 8 columns.
struct Mat {
    const void* p = nullptr;
    int64_t ld = 0;
    bool padded = false;
};

// Whether a matrix's rows lie on 16 bytes and end there too, with offsets
// within 128 rows (64 of k) inside 2^31 bytes: what loads from memory
// straight to LDS need.
inline bool direct(const Mat& a, int64_t cols) {
    return reinterpret_cast<uintptr_t>(a.p) % 16 == 0 && a.ld % 8 == 0 &&
           (a.padded || cols % 8 == 0) && a.ld <= (int64_t(1) << 22);
}

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
    const float* unscale = nullptr;  // dx, dw: of dz times a power of two, its reciprocal; or null
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
    // kDx, kDw: a comes as the sum of so many matrices, `low` elements apart.
    int32_t pieces = 1;
    int64_t low = 0;
    // Not 0: so many rows of dz, at most 32, come in two pieces, all first pieces
    // before all second ones.  kDx: m = fold, a has 2 fold rows (those of a tile),
    // and sums `fold` rows apart are added.  kDw: k = 2 fold (one step of 64), and
    // b's fold rows are taken for either piece.
    int32_t fold = 0;
    Finish fin;
};

// The kernels.  Guarded and thin ones take any strides and alignment, the
// others rows on 16 bytes.  Outputs per workgroup:
//   kGuarded  64 x 64, four groups; kMid32  32 x 64, four groups of waves over k
//   kThin     32 x 16; kMid64  64 x 64, two groups
//   kBig      256 x 256   kMid128 128 x 128 with a ring of four tiles, one
//                         workgroup per compute unit; kPair128 with two, and two
enum Tile { kGuarded, kThin, kMid32, kMid64, kMid128, kPair128, kBig, kLight };

struct TileSize {
    int64_t m, n;
};
constexpr TileSize kTileSize[] = {{64, 64},   {32, 16},   {32, 64},  {64, 64},
                                  {128, 128}, {128, 128}, {256, 256}, {64, 64}};

// Which kernel, and the split of a product over its long axis: `splits`
// workgroups per tile, each over `per` steps of 64; their 32-bit sums meet in
// the workspace.
struct Cut {
    int tile = kGuarded;
    int splits = 1;
    int64_t per = 0;
    double us = 0;  // what it is expected to take
};

// Whether the kernels that take rows on 16 bytes can take this product.
bool direct(const Product& p);

// From the sizes, and whether the operands' rows lie on 16 bytes.
Cut plan_product(int form, int64_t m, int64_t n, int64_t k, int parts, bool direct,
                 int fold = 0, int pieces = 1);

constexpr int kMostParts = 512;

// dz = dy * act'(pre), its rows padded with zeros to ldz, and the sums of its
// columns over `per` rows each into `part` (either null: not wanted); with
// `up`, dz = dy * up * act'(pre) and dz2 = dy * act(pre) and no sums, `per` (4
// or 8) elements per thread.  dz and dz2 are stored as the sum of `pieces`
// matrices, `low` elements apart.  most (fp16; or null): space for kMostParts partial maxima
// of |dz| and |dz2|; they are then stored times the power of two that brings
// the largest into [2^14, 2^15), and its reciprocal goes to `unscale`.
struct SlopeArgs {
    int64_t M = 0, N = 0, per = 0, low = 0;
    const void *dy = nullptr, *pre = nullptr, *up = nullptr;
    int64_t lddy = 0, ldp = 0, ldu = 0, ldz = 0;
    void *dz = nullptr, *dz2 = nullptr;
    float* part = nullptr;
    float *most = nullptr, *unscale = nullptr;
    int32_t act = 0, pieces = 1;
    int32_t parts = 0;  // how many of `most` there are
};

// The partial column sums, to be added up into `out` (null: none).
struct Sums {
    int64_t rows = 0, N = 0;
    const float* part = nullptr;
    void* out = nullptr;
    int32_t wide = 0;
};

// Rows that are laid out anew, on 16 bytes and padded with zeros.
struct Repack {
    const void* from[3];
    void* to[3];
    int64_t ld[3], rows[3], cols[3];
    int count = 0;
};

// Rows per workgroup of a column sum over 512 columns: enough workgroups for
// the chip (8 waves on each SIMD), then as few as that.
inline int64_t sum_rows(int64_t m, int64_t n) {
    int64_t r = 8;
    while (r < 128 && (n + 511) / 512 * (m / r) > 2048) r *= 2;
    return r;
}

// The launchers, for DGC_BF16 and DGC_FP16 elements.  Each returns a DGC_* code.
template <class T>
struct Launch {
    static int product(const Product& p, const Cut& c, void* ws, hipStream_t s);
    // dx and dw of one layer (neither split, the same kernel for both) and the
    // column sums in one launch
    static int both(const Product& dx, const Product& dw, int tile, const Sums& sums,
                    hipStream_t s);
    // slopes (none if a.N is 0) and rows laid out anew in one launch; the largest
    // |dz| in one before, where it is asked for
    static int prepare(SlopeArgs a, const Repack& r, hipStream_t s);
    static int sum(const Sums& a, hipStream_t s);
};

inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace layers
}  // namespace dgc
