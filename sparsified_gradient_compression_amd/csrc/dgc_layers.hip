// dgc_layers.hip -- host side of the layer operators: argument checks, the
// split of each product, workspace carving and launch order.  See
// include/dgc.h for the contract of every function.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "layers.hpp"

using namespace dgc::layers;

namespace dgc {
namespace layers {

namespace {

constexpr size_t kPad = 256;

size_t round_up(size_t x) { return (x + kPad - 1) / kPad * kPad; }

}  // namespace

namespace {

// What a round of workgroups takes: a start (the first loads, the outputs'
// way out) and so many microseconds per step of 64 of k, for `round`
// workgroups at once and for `light` or fewer of them.  Measured on bf16
// products of 64 to 8192 rows and columns, in microseconds:
//                        kMid32 kMid64 kLight kMid128 kPair128 kBig  kGuarded
//   64 x 704, k 704         5.6    5.5     6.4     8.0      8.6    19       7.2
//   1024 x 1024, k 64        10    5.0     4.2     6.2      4.9    15       6.4
//   1024 x 1024, k 1024      12    6.9     8.5      11       14    27       9.2
//   2048 x 2048, k 2048      57     35      26      20       26    42        47
//   3000 x 1500, k 3000      97     78      70      62       46    65
//   858 x 696, k 14336       89     54     119     100      175   279
//     split in 4 and joined  72     51      44      35       50    84
//   4096 x 4096, k 64       120     51      18      20       13    17        67
//   4096 x 4096, k 2048     221    132      95      75       64    53
// Off 16 bytes a step of kGuarded takes half as long again.
struct Cost {
    int tile;
    int64_t round, light;
    double start, step, light_start, light_step;
};
constexpr Cost kCosts[] = {
    {kGuarded, 256, 256, 2.6, 0.40, 2.6, 0.40}, {kMid32, 256, 256, 3.4, 0.13, 3.4, 0.13},
    {kMid64, 256, 256, 2.2, 0.21, 2.2, 0.21},   {kMid128, 256, 256, 3.8, 0.45, 3.8, 0.45},
    {kPair128, 512, 256, 5.0, 0.80, 3.5, 0.62}, {kBig, 256, 128, 11.0, 1.28, 9.0, 1.05},
    {kLight, 1280, 640, 4.0, 1.25, 2.5, 0.45}};
constexpr double kLaunchUs = 2.5;  // of a launch, or between two

double rounds_us(const Cost& c, int64_t blocks, double steps) {
    const int64_t rest = blocks % c.round;
    double us = double(blocks / c.round) * (c.start + c.step * steps);
    if (rest > c.light)
        us += c.start + c.step * steps;
    else if (rest > 0)
        us += c.light_start + c.light_step * steps;
    return us;
}

// A second launch that adds the splits' sums, and its traffic.
double join_us(double bytes) { return kLaunchUs + bytes / 5e6; }

// Up to 32 rows, kThin and the tiles.  kThin's waves read every row of x for
// their 16 columns; a tile of 32 or 64 rows reads x once for 64 columns, and
// the weight no faster than the memory gives it.  Microseconds per call, in a
// row of calls on six sets of inputs:
//                            kThin  kMid32  kMid32 in 4
//   4 x 4096, k 4096          10.0    11.6    12.1
//   32 x 704, k 704            5.0     6.0     8.6
//   16 x 1024, k 4096         10.4    11.6    10.1
//   32 x 4096, k 4096         14.0    12.6    12.6
//   32 x 512, k 8192          24.1    19.1    11.8
//   16 x 8192, k 2048         11.3     9.4    15.0
//   32 x 16384, k 4096        54.7    32.3    40.2
// The tiles are taken where they are expected to need 15% less, which of 90
// products measured so is never the slower choice.
constexpr int64_t kFewRows = 32;
constexpr double kTilesGain = 0.85, kWeightRate = 5e6;  // bytes per microsecond

double thin_us(int64_t m, int64_t n, int64_t k, int products) {
    const double rounds = double(cdiv64(cdiv64(n, 16), 256)), steps = double(k) / 512;
    const double us = rounds * (3.3 + steps * (0.52 * products + 0.0245 * double(m)));
    return std::max(us, 3.3 + 2.0 * double(n) * double(k) * products / kWeightRate);
}

}  // namespace

bool direct(const Product& p) {
    const int64_t ca = p.form == kDw ? p.m : p.k, cb = p.form == kRows || p.form == kPair ? p.k : p.n;
    const bool two_a = p.form != kRows && p.form != kPair && p.parts == 2;
    const bool two_b = p.form == kPair || (p.form == kDx && p.parts == 2);
    if (!direct(p.a[0], ca) || !direct(p.b[0], cb)) return false;
    if (two_a && (!direct(p.a[1], ca) || p.a[1].ld != p.a[0].ld)) return false;
    return !two_b || (direct(p.b[1], cb) && p.b[1].ld == p.b[0].ld);
}

// The rows that a kernel's tile has have to take both pieces of a folded dz.
bool takes(const TileSize& t, int form, int fold) { return form != kDx || t.m >= 2 * fold; }

Cut plan_product(int form, int64_t m, int64_t n, int64_t k, int parts, bool direct, int fold,
                 int pieces) {
    const int64_t outs = form == kDw ? parts : 1;
    const int64_t steps = std::max<int64_t>(cdiv64(k, 64) * (form == kDx ? parts : 1) * pieces, 1);
    const int64_t wide = form == kPair ? 2 * n : n;
    Cut best;
    best.us = 1e30;
    const bool few = (form == kRows || form == kPair) && m <= kFewRows;
    const double weight_us = few ? 2.0 * double(wide) * double(k) / kWeightRate : 0.0;
    if (few) {
        best.tile = kThin;
        best.per = steps;
        best.us = kTilesGain * thin_us(m, n, k, form == kPair ? 2 : 1);
        if (!direct) return best;  // no tile reads rows off 16 bytes as fast
    }
    for (const Cost& c : kCosts) {
        if ((c.tile == kGuarded) == direct) continue;
        const TileSize t = kTileSize[c.tile];
        if (!takes(t, form, fold)) continue;
        const int64_t tiles = cdiv64(m, t.m) * cdiv64(wide, t.n) * outs;
        for (int64_t splits = 1; splits <= 8; splits *= 2) {
            // a split keeps 8 steps, and only fills up a round
            if (splits > 1 && (steps < 8 * splits || tiles * splits > c.round)) break;
            const int64_t per = cdiv64(steps, splits), work = tiles * splits;
            double us = rounds_us(c, work, double(per));
            if (few) us = std::max(us, c.start + weight_us);
            if (splits > 1)
                us += join_us(8.0 * double(splits) * double(m) * double(wide) * double(outs)) +
                      (few ? 1.0 : 0.0);  // measured where nothing hides it
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

// When the last of nx workgroups of ux microseconds each, and behind them nw of
// uw, ends on `slots` places.
double queue_us(int64_t slots, int64_t nx, double ux, int64_t nw, double uw) {
    const double full = double(nx / slots) * ux;
    const int64_t ex = nx % slots, free = slots - ex;
    double end = full + (ex > 0 ? ux : 0);
    if (nw == 0) return end;
    // the first time by which all nw have ended: a multiple of uw from either
    // moment at which places become free
    const auto ended = [&](double t) {
        const auto each = [&](double from) { return int64_t(std::max(0.0, (t - from) / uw + 1e-6)); };
        return free * each(full) + ex * each(full + ux);
    };
    const auto first = [&](double from, int64_t places) {
        if (places == 0) return 1e30;
        int64_t low = std::max<int64_t>(nw / slots - int64_t(ux / uw) - 1, 0);
        int64_t high = std::max(cdiv64(nw, places), low);
        while (low < high) {
            const int64_t mid = low + (high - low) / 2;
            if (ended(from + double(mid) * uw) >= nw)
                high = mid;
            else
                low = mid + 1;
        }
        return from + double(low) * uw;
    };
    return std::max(end, std::min(first(full, free), first(full + ux, ex)));
}

// Both gradients in one launch, dx's workgroups first: sx and sw steps each.
// Gates' gradients (1531 x 3840 x 1280, 120 and 300 tiles of 128, dz in one piece;
// expected, and measured as what the call takes more than its slopes): kMid128
// 48.6 and 48.2, kPair128 46.5 and 46.7 (traced: 51).
double both_us(const Cost& c, int64_t nx, double sx, int64_t nw, double sw) {
    if (nx + nw <= c.light) return c.light_start + c.light_step * std::max(sx, sw);
    if (nx + nw <= c.round) {  // all at once, and then the longer ones alone
        const int64_t longer = sx > sw ? nx : nw;
        return c.start + c.step * std::min(sx, sw) +
               std::fabs(sx - sw) * (longer <= c.light ? c.light_step : c.step);
    }
    // operands that are turned on their way to the registers: 2048 x 2048, k
    // 8192 takes 73 us with neither, 74-85 as a dx and 81-97 as a dw.  Of 4000
    // drawn layers the factor decides 125; 24 of those take 3% less with it.
    // Products launched apart go without (plan_product): 24 of the 109 that it
    // would decide there take 7% more with it.
    const double step = c.tile == kMid128 ? 1.15 * c.step : c.step;
    return queue_us(c.round, nx, c.start + step * sx, nw, c.start + step * sw);
}

// The kernel that takes both gradients of a layer in the least time, together.
int plan_both(const Product& dx, const Product& dw, bool direct, double& best) {
    int tile = kGuarded;
    best = 1e30;
    const double sx = double(std::max<int64_t>(cdiv64(dx.k, 64) * dx.parts * dx.pieces, 1));
    const double sw = double(std::max<int64_t>(cdiv64(dw.k, 64) * dw.pieces, 1));
    for (const Cost& c : kCosts) {
        if ((c.tile == kGuarded) == direct || c.tile == kBig) continue;
        const TileSize t = kTileSize[c.tile];
        if (!takes(t, kDx, dx.fold)) continue;
        const double us = both_us(c, cdiv64(dx.m, t.m) * cdiv64(dx.n, t.n), sx,
                                  cdiv64(dw.m, t.m) * cdiv64(dw.n, t.n) * dw.parts, sw);
        if (us < best) {
            best = us;
            tile = c.tile;
        }
    }
    return tile;
}

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

// A product's splits, in the workspace: as many as any of its forms has.
size_t part_bytes(int form, int64_t m, int64_t n, int64_t k, int parts, int fold = 0,
                  int most_pieces = 1) {
    const int64_t planes = form == kPair ? 2 : form == kDw ? parts : 1;
    size_t most = 0;
    const auto form_of = [&](bool d, int fo, int pieces) {
        const Cut c = plan_product(form, m, n, k, parts, d, fo, pieces);
        if (c.splits > 1)
            most = std::max(most,
                            size_t(c.splits) * size_t(planes) * size_t(m) * size_t(n) * 4);
    };
    for (const bool d : {false, true}) {
        // folded dz is one piece as far as its steps go; none is folded without an activation
        if (fold) form_of(d, fold, 1);
        for (int pieces = 1; pieces <= most_pieces; ++pieces) form_of(d, 0, pieces);
    }
    return round_up(most);
}

// Whether a product whose operands (`elements` of them) do not lie on 16 bytes
// gains from laying them out anew first: a launch and twice their bytes.
bool worth_repacking(int form, int64_t m, int64_t n, int64_t k, int parts, int64_t elements) {
    const Cut as_is = plan_product(form, m, n, k, parts, false);
    if (as_is.tile == kThin) return false;
    return plan_product(form, m, n, k, parts, true).us + kLaunchUs + 4.0 * double(elements) / 6e6 <
           as_is.us;
}

size_t row_bytes(int64_t rows, int64_t cols) {
    return round_up(size_t(rows) * size_t(pad8(cols)) * 2);
}

// Rows up to which dz is folded: both pieces of as many lie in a tile of 64.
constexpr int64_t kFoldRows = 32;

// Pieces of dz where the caller does not ask for one (layers_elem.hpp).
constexpr int kPieces = 2, kMostPieces = 3;

// Where a call keeps what it lays out: dz (da, db), column sums, dz's partial
// maxima and the factor that its scale is undone by, operands that are
// repacked, and splits.  From the sizes alone.
struct Space {
    bool pack = false;
    int32_t fold = 0;  // rows of dz, where it is folded
    size_t dz = 0, sums = 0, most = 0, x = 0, w = 0, w2 = 0, part = 0, total = 0;
};

Space space(bool gated, int32_t backward, int64_t m, int64_t n, int64_t k) {
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
        const int pieces = backward == DGC_BACKWARD_ROUNDED ? 1 : kMostPieces;
        s.fold = m <= kFoldRows ? int32_t(m) : 0;
        s.dz = take(two * row_bytes(std::max(m + s.fold, pieces * m), n));
        s.sums = take(gated ? 0 : round_up(size_t(cdiv64(m, sum_rows(m, n))) * size_t(n) * 4));
        s.most = take(m > 0 && n > 0 ? round_up((kMostParts + 1) * sizeof(float)) : 0);
        s.pack = worth_repacking(kDx, m, k, n, two, weights) ||
                 worth_repacking(kDw, n, k, m, two, m * k);
        part = std::max(part_bytes(kDx, m, k, n, two, s.fold, pieces),
                        part_bytes(kDw, n, k, m + s.fold, two, 0, pieces));
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
Mat anew(Repack& r, Mat a, int64_t rows, int64_t cols, void* to) {
    r.from[r.count] = a.p;
    r.to[r.count] = to;
    r.ld[r.count] = a.ld;
    r.rows[r.count] = rows;
    r.cols[r.count] = cols;
    ++r.count;
    return {to, pad8(cols), true};
}

// The same for one that does not lie on 16 bytes, if laying out pays.
Mat packed(Repack& r, bool pack, Mat a, int64_t rows, int64_t cols, void* to) {
    const bool as_is = !pack || rows == 0 || cols == 0 || direct(a, cols);
    return as_is ? a : anew(r, a, rows, cols, to);
}

// Both weights of a gated block: the kernels that take rows on 16 bytes take
// them of one length too.  One whose rows are as long as a copy's stays.
void packed_pair(Repack& r, bool pack, Mat& a, Mat& b, int64_t rows, int64_t cols, void* to_a,
                 void* to_b) {
    if (!pack || rows == 0 || cols == 0) return;
    const bool da = direct(a, cols), db = direct(b, cols);
    if (da && db && a.ld == b.ld) return;
    if (!da || a.ld != pad8(cols)) a = anew(r, a, rows, cols, to_a);
    if (!db || b.ld != pad8(cols)) b = anew(r, b, rows, cols, to_b);
}

int run_product(int64_t type, const Product& p, void* ws, hipStream_t s) {
    const Cut c = plan_product(p.form, p.m, p.n, p.k, p.parts, direct(p), p.fold, p.pieces);
    return type == DGC_BF16 ? Launch<__bf16>::product(p, c, ws, s)
                            : Launch<_Float16>::product(p, c, ws, s);
}

// How a dz that 16 bits do not hold is stored, and what its products make of it.
// (dx takes the first two pieces of three, the second of which lies below what
// is left: off by 2^-15, where two of two are off by 2^-16.)
void hold_dz(int64_t type, bool rounded, bool wide, const Space& sp, char* ws, SlopeArgs& a,
             Product& dx, Product& dw) {
    a.low = dx.low = dw.low = a.M * a.ldz;
    const int pieces = rounded ? 1 : kPieces;
    const int dw_pieces = wide && type == DGC_BF16 && !rounded ? kMostPieces : pieces;
    a.pieces = std::max(dw_pieces, sp.fold ? kPieces : 1);
    dx.fold = sp.fold;
    if (!sp.fold) dx.pieces = pieces;
    if (sp.fold && dw_pieces < kMostPieces) {
        dw.fold = sp.fold;
        dw.k += sp.fold;
    } else {
        dw.pieces = dw_pieces;
    }
    // fp16 holds a product of fp16 numbers only after a scale
    if (type != DGC_FP16 || a.M == 0 || a.N == 0) return;
    a.most = reinterpret_cast<float*>(ws + sp.most);
    a.unscale = a.most + kMostParts;
    dx.fin.unscale = dw.fin.unscale = a.unscale;
}

int run_prepare(int64_t type, const SlopeArgs& a, const Repack& r, hipStream_t s) {
    return type == DGC_BF16 ? Launch<__bf16>::prepare(a, r, s)
                            : Launch<_Float16>::prepare(a, r, s);
}

// The gradients' products and the column sums: in one launch where a kernel
// takes both products whole in less time than each its own way and a launch
// more.  Either product's output may be null.
int run_gradients(int64_t type, const Product& dx, const Product& dw, const Sums& sums, void* ws,
                  hipStream_t s) {
    const bool has_dx = dx.fin.out[0] && dx.m > 0 && dx.n > 0;
    const bool has_dw = dw.fin.out[0] && dw.m > 0 && dw.n > 0;
    int rc = DGC_OK;
    if (has_dx && has_dw) {
        const bool d = direct(dx) && direct(dw);
        const Cut cx =
            plan_product(kDx, dx.m, dx.n, dx.k, dx.parts, direct(dx), dx.fold, dx.pieces);
        const Cut cw = plan_product(kDw, dw.m, dw.n, dw.k, dw.parts, direct(dw), 0, dw.pieces);
        const double apart = cx.us + cw.us + (sums.out ? 2 : 1) * kLaunchUs;  // without a first one
        double us = 0;
        const int tile = plan_both(dx, dw, d, us);
        if (us < apart)
            return type == DGC_BF16 ? Launch<__bf16>::both(dx, dw, tile, sums, s)
                                    : Launch<_Float16>::both(dx, dw, tile, sums, s);
    }
    if (has_dx) rc = run_product(type, dx, ws, s);
    if (rc == DGC_OK && has_dw) rc = run_product(type, dw, ws, s);
    if (rc == DGC_OK)
        rc = type == DGC_BF16 ? Launch<__bf16>::sum(sums, s) : Launch<_Float16>::sum(sums, s);
    return rc;
}

}  // namespace
}  // namespace layers
}  // namespace dgc

extern "C" {

int dgc_linear_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t backward, size_t* bytes) {
    if (!bytes || !sizes_ok(m, n, k)) return DGC_EINVAL;
    *bytes = space(false, backward, m, n, k).total;
    return DGC_OK;
}

int dgc_gated_ffn_workspace_bytes(int64_t m, int64_t d, int64_t f, int32_t backward,
                                  size_t* bytes) {
    if (!bytes || !sizes_ok(m, d, f)) return DGC_EINVAL;
    *bytes = space(true, backward, m, f, d).total;
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
    const Space sp = space(false, 0, m, n, k);
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
    rc = run_prepare(a->type, SlopeArgs{}, r, stream);
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
    const bool rounded = a && (a->act & DGC_DZ_ROUNDED);
    const int64_t act = a ? a->act & ~int64_t(DGC_DZ_ROUNDED) : 0;
    if (!a || !half(a->type) || !act_ok(act) || !sizes_ok(a->m, a->n, a->k) ||
        (a->grad_type != a->type && a->grad_type != DGC_FP32))
        return DGC_EINVAL;
    const int64_t m = a->m, n = a->n, k = a->k;
    const int wide = a->grad_type == DGC_FP32;
    const bool sloped = act != DGC_ACT_NONE;
    if (!mat_ok(a->dy, a->lddy, m, n, 2) || !mat_ok(a->x, a->ldx, m, k, 2) ||
        !mat_ok(a->w, a->ldw, n, k, 2) || (sloped && !mat_ok(a->pre, a->ldpre, m, n, 2)) ||
        !optional_ok(a->dx, a->lddx, m, k, 2) ||
        !optional_ok(a->dw, a->lddw, n, k, wide ? 4 : 2) ||
        !optional_ok(a->dbias, n, 1, n, wide ? 4 : 2))
        return DGC_EINVAL;
    const Space sp = space(false, rounded ? DGC_BACKWARD_ROUNDED : 1, m, n, k);
    int rc = space_ok(workspace, workspace_bytes, sp.total);
    if (rc != DGC_OK) return rc;
    char* ws = static_cast<char*>(workspace);
    Repack r;
    Mat x{a->x, a->ldx}, w{a->w, a->ldw}, dz{a->dy, a->lddy};
    if (a->dw) x = packed(r, sp.pack, x, m, k, ws + sp.x);
    if (a->dx) w = packed(r, sp.pack, w, n, k, ws + sp.w);
    // without an activation dz is dy, copied only where its rows do not lie on 16 bytes
    const bool copied = (a->dx || a->dw) && (sloped || (sp.pack && !direct(dz, n)));
    if (copied) dz = {ws + sp.dz, pad8(n), true};
    SlopeArgs sl;
    Sums sums;
    Product dx, dw;
    dw.k = m;
    if (copied || a->dbias) {
        sl.M = m;
        sl.N = n;
        sl.per = sum_rows(m, n);
        sl.dy = a->dy;
        sl.lddy = a->lddy;
        sl.pre = a->pre;
        sl.ldp = a->ldpre;
        sl.act = int32_t(act);
        sl.dz = copied ? ws + sp.dz : nullptr;
        sl.ldz = pad8(n);
        // (relu's slope is 0 or 1: dz is 0 or dy)
        if (sloped && act != DGC_ACT_RELU && copied)
            hold_dz(a->type, rounded, wide, sp, ws, sl, dx, dw);
        sl.part = a->dbias ? reinterpret_cast<float*>(ws + sp.sums) : nullptr;
        sums.rows = cdiv64(m, sl.per);
        sums.N = n;
        sums.part = sl.part;
        sums.out = a->dbias;
        sums.wide = wide;
    }
    rc = run_prepare(a->type, sl, r, stream);
    if (rc != DGC_OK) return rc;
    dx.form = kDx;
    dx.m = m;
    dx.n = k;
    dx.k = n;
    dx.a[0] = dz;
    dx.b[0] = w;
    dx.fin.out[0] = a->dx;
    dx.fin.ldo = a->lddx;
    dw.form = kDw;
    dw.m = n;
    dw.n = k;
    dw.a[0] = dz;
    dw.b[0] = x;
    dw.fin.out[0] = a->dw;
    dw.fin.ldo = a->lddw;
    dw.fin.wide = wide;
    return run_gradients(a->type, dx, dw, sums, ws + sp.part, stream);
}

int dgc_gated_ffn(const dgc_gated_ffn_args* a, void* workspace, size_t workspace_bytes,
                  hipStream_t stream) {
    if (!a || !half(a->type) || !act_ok(a->act) || !sizes_ok(a->m, a->d, a->f)) return DGC_EINVAL;
    const int64_t m = a->m, d = a->d, f = a->f;
    if (!mat_ok(a->x, a->ldx, m, d, 2) || !mat_ok(a->w_gate, a->ldw_gate, f, d, 2) ||
        !mat_ok(a->w_up, a->ldw_up, f, d, 2) || !mat_ok(a->h, a->ldh, m, f, 2) ||
        !optional_ok(a->gate, a->ldgate, m, f, 2) || !optional_ok(a->up, a->ldup, m, f, 2))
        return DGC_EINVAL;
    const Space sp = space(true, 0, m, f, d);
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
    p.b[0] = {a->w_gate, a->ldw_gate};
    p.b[1] = {a->w_up, a->ldw_up};
    packed_pair(r, sp.pack, p.b[0], p.b[1], f, d, ws + sp.w, ws + sp.w2);
    rc = run_prepare(a->type, SlopeArgs{}, r, stream);
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
    const bool rounded = a && (a->act & DGC_DZ_ROUNDED);
    const int64_t act = a ? a->act & ~int64_t(DGC_DZ_ROUNDED) : 0;
    if (!a || !half(a->type) || !act_ok(act) || !sizes_ok(a->m, a->d, a->f) ||
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
    const Space sp = space(true, rounded ? DGC_BACKWARD_ROUNDED : 1, m, f, d);
    int rc = space_ok(workspace, workspace_bytes, sp.total);
    if (rc != DGC_OK) return rc;
    if (!a->dx && !a->dw_gate) return DGC_OK;
    char* ws = static_cast<char*>(workspace);
    const int64_t ld = pad8(f);
    Repack r;
    Mat x{a->x, a->ldx}, wg{a->w_gate, a->ldw_gate}, wu{a->w_up, a->ldw_up};
    if (a->dw_gate) x = packed(r, sp.pack, x, m, d, ws + sp.x);
    if (a->dx) packed_pair(r, sp.pack, wg, wu, f, d, ws + sp.w, ws + sp.w2);
    SlopeArgs sl;
    sl.M = m;
    sl.N = f;
    sl.per = m * f < (int64_t(1) << 21) ? 4 : 8;  // fewer than 8 waves on each SIMD: shorter ones
    sl.dy = a->dh;
    sl.lddy = a->lddh;
    sl.pre = a->gate;
    sl.ldp = a->ldgate;
    sl.up = a->up;
    sl.ldu = a->ldup;
    sl.act = int32_t(act);
    sl.ldz = ld;
    Product dx, dw;
    dw.k = m;
    hold_dz(a->type, rounded, wide, sp, ws, sl, dx, dw);
    sl.dz = ws + sp.dz;
    sl.dz2 = ws + sp.dz + row_bytes(sl.pieces * m, f);
    rc = run_prepare(a->type, sl, r, stream);
    if (rc != DGC_OK) return rc;
    dx.form = kDx;
    dx.parts = 2;
    dx.m = m;
    dx.n = d;
    dx.k = f;
    dx.b[0] = wg;
    dx.b[1] = wu;
    dx.fin.out[0] = a->dx;
    dx.fin.ldo = a->lddx;
    dw.form = kDw;
    dw.parts = 2;
    dw.m = f;
    dw.n = d;
    dw.b[0] = x;
    dw.fin.out[0] = a->dw_gate;
    dw.fin.ldo = a->lddw_gate;
    dw.fin.out[1] = a->dw_up;
    dw.fin.ldo2 = a->lddw_up;
    dw.fin.wide = wide;
    dx.a[0] = dw.a[0] = {sl.dz, ld, true};
    dx.a[1] = dw.a[1] = {sl.dz2, ld, true};
    return run_gradients(a->type, dx, dw, Sums{}, ws + sp.part, stream);
}

}  // extern "C"
