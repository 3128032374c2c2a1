// layers_plan_check.cpp -- what the layer operators' host code hands to its
// launchers, which are replaced here: nothing runs on a GPU, and the addresses
// are never followed.  Built with dgc_layers.hip and run by
// tests/test_layers_plan.py.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "layers.hpp"

#define CHECK(c)                                                             \
    do {                                                                     \
        if (!(c)) {                                                          \
            std::fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__); \
            std::abort();                                                    \
        }                                                                    \
    } while (0)

namespace dgc {
namespace layers {

std::vector<Product> products;
std::vector<int> tiles;
std::vector<Repack> repacks;
uintptr_t space_begin = 0, space_end = 0;  // the call's workspace, where it is checked
std::vector<std::pair<uintptr_t, uintptr_t>> used;

// A range of the workspace that a launch uses; none overlap.
void uses(const void* p, int64_t bytes) {
    if (space_end == 0 || bytes == 0) return;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = a + uintptr_t(bytes);
    CHECK(a >= space_begin && b <= space_end);
    for (const auto& r : used) CHECK(b <= r.first || a >= r.second);
    used.push_back({a, b});
}

template <class T>
int Launch<T>::product(const Product& p, const Cut& c, void* ws, hipStream_t) {
    if (c.splits > 1) {
        const int64_t planes = p.form == kPair ? 2 : p.form == kDw ? p.parts : 1;
        const auto before = used;  // the next product's sums may lie there again
        uses(ws, 4 * c.splits * planes * p.m * p.n);
        used = before;
    }
    CHECK(c.splits * c.per * 64 >= p.k * p.pieces * (p.form == kDx ? p.parts : 1));
    products.push_back(p);
    tiles.push_back(c.tile);
    return DGC_OK;
}

template <class T>
int Launch<T>::both(const Product& dx, const Product& dw, int tile, const Sums&, hipStream_t) {
    products.push_back(dx);
    products.push_back(dw);
    tiles.push_back(tile);
    return DGC_OK;
}

template <class T>
int Launch<T>::prepare(SlopeArgs a, const Repack& r, hipStream_t) {
    if (a.M > 0 && a.N > 0) {
        const int64_t piece = a.M * a.ldz;
        CHECK(a.pieces >= 1 && a.pieces <= 3 && (a.pieces == 1 || a.low == piece));
        if (a.dz) uses(a.dz, 2 * a.pieces * piece);
        if (a.dz2) uses(a.dz2, 2 * a.pieces * piece);
        if (a.part) uses(a.part, 4 * cdiv64(a.M, a.per) * a.N);
        if (a.most) {
            CHECK(sizeof(T) == 2 && (__is_same(T, _Float16)));
            uses(a.most, 4 * kMostParts);
            uses(a.unscale, 4);
        }
    }
    for (int i = 0; i < r.count; ++i) uses(r.to[i], 2 * r.rows[i] * ((r.cols[i] + 7) / 8 * 8));
    repacks.push_back(r);
    return DGC_OK;
}

template <class T>
int Launch<T>::sum(const Sums&, hipStream_t) {
    return DGC_OK;
}

template struct Launch<__bf16>;
template struct Launch<_Float16>;

}  // namespace layers
}  // namespace dgc

using namespace dgc::layers;

namespace {

void* const kSpace = reinterpret_cast<void*>(uintptr_t(1) << 40);

const void* at(int i, int off = 0) {
    return reinterpret_cast<const void*>((uintptr_t(i) << 34) + uintptr_t(off));
}

void* out(int i) { return const_cast<void*>(at(i)); }

void reset() {
    products.clear();
    tiles.clear();
    repacks.clear();
}

// Every product takes rows on 16 bytes, and `copies` matrices were laid out anew for it.
void check_direct(int copies) {
    CHECK(!products.empty() && repacks.size() == 1);
    for (const Product& p : products) CHECK(direct(p));
    for (int t : tiles) CHECK(t != kGuarded);
    CHECK(repacks[0].count == copies);
}

// A gated block of m x d and f x d, its weights' rows ld_g and ld_u elements
// apart and starting off_g and off_u bytes off 16.
void gated(int64_t m, int64_t d, int64_t f, int64_t ld_g, int64_t ld_u, int off_g, int off_u,
           int copies) {
    size_t bytes = 0;
    reset();
    CHECK(dgc_gated_ffn_workspace_bytes(m, d, f, 0, &bytes) == DGC_OK);
    dgc_gated_ffn_args a{DGC_BF16, DGC_ACT_SILU, m, d, f, at(1), d, at(2, off_g), ld_g,
                         at(3, off_u), ld_u, out(4), f, out(5), f, out(6), f};
    CHECK(dgc_gated_ffn(&a, kSpace, bytes, nullptr) == DGC_OK);
    check_direct(copies);
    reset();
    CHECK(dgc_gated_ffn_workspace_bytes(m, d, f, 1, &bytes) == DGC_OK);
    dgc_gated_ffn_backward_args b{DGC_BF16, DGC_BF16, DGC_ACT_SILU, m, d, f, at(7), f, at(1), d,
                                  at(2, off_g), ld_g, at(3, off_u), ld_u, at(5), f, at(6), f,
                                  out(8), d, out(9), d, out(10), d};
    CHECK(dgc_gated_ffn_backward(&b, kSpace, bytes, nullptr) == DGC_OK);
    check_direct(copies);
}

}  // namespace

// Few rows: kThin where it is measured to be faster, tiles where they are.
void few_rows() {
    struct Case {
        int form;
        int64_t m, n, k;
        bool thin;
    };
    for (const Case& c : {Case{kRows, 1, 4096, 4096, true}, Case{kPair, 3, 8192, 2048, true},
                          Case{kRows, 32, 704, 704, true}, Case{kRows, 16, 4096, 1024, true},
                          Case{kRows, 32, 4096, 1024, true}, Case{kRows, 16, 1000, 2048, true},
                          Case{kPair, 4, 16384, 4096, true}, Case{kRows, 4, 4096, 8192, true},
                          Case{kRows, 32, 512, 8192, false}, Case{kPair, 4, 512, 8192, false},
                          Case{kRows, 32, 16384, 4096, false}, Case{kRows, 17, 8192, 2048, false},
                          Case{kPair, 32, 1024, 4096, false}, Case{kRows, 24, 1024, 4096, false}}) {
        const Cut cut = plan_product(c.form, c.m, c.n, c.k, 1, true);
        CHECK((cut.tile == kThin) == c.thin && cut.us > 0);
        CHECK(plan_product(c.form, c.m, c.n, c.k, 1, false).tile == kThin);
    }
}

// Calls of any sizes, types and strides: whatever they launch stays in the
// workspace that their sizes gave.
void workspaces() {
    std::mt19937 rng(5);
    const auto pick = [&](int n) { return int(rng() % unsigned(n)); };
    const auto size = [&] {
        const int64_t v = int64_t(1) << pick(14);
        return v + pick(int(v));
    };
    for (int round = 0; round < 20000; ++round) {
        const int64_t m = pick(3) ? size() : 1 + pick(40), n = size(), k = size();
        const int64_t type = pick(2) ? DGC_BF16 : DGC_FP16, act = pick(5);
        const int64_t grad = pick(2) ? type : int64_t(DGC_FP32);
        const int64_t flag = pick(3) ? 0 : DGC_DZ_ROUNDED;
        const int back = flag ? DGC_BACKWARD_ROUNDED : 1;
        const int64_t pad = pick(2) ? 0 : 1 + pick(16), pad2 = pick(2) ? pad : 8 * pick(3);
        const int off = pick(2) ? 0 : 2 * pick(8);
        const auto call = [&](size_t bytes, auto f) {
            reset();
            used.clear();
            space_begin = reinterpret_cast<uintptr_t>(kSpace);
            space_end = space_begin + bytes;
            CHECK(f(bytes) == DGC_OK);
            space_end = 0;
        };
        size_t bytes = 0;
        CHECK(dgc_linear_workspace_bytes(m, n, k, 0, &bytes) == DGC_OK);
        call(bytes, [&](size_t b) {
            dgc_linear_args a{type, act, m, n, k, at(1, off), k + pad, at(2), k + pad2, at(3),
                              at(4), n, out(5), n, out(6), n};
            return dgc_linear(&a, kSpace, b, nullptr);
        });
        CHECK(dgc_linear_workspace_bytes(m, n, k, back, &bytes) == DGC_OK);
        call(bytes, [&](size_t b) {
            dgc_linear_backward_args a{type, grad, act | flag, m, n, k, at(7, off), n + pad, at(1), k + pad2,
                                       at(2), k + pad, at(6), n, pick(4) ? out(8) : nullptr, k,
                                       pick(4) ? out(9) : nullptr, k, pick(2) ? out(10) : nullptr};
            return dgc_linear_backward(&a, kSpace, b, nullptr);
        });
        CHECK(dgc_gated_ffn_workspace_bytes(m, k, n, 0, &bytes) == DGC_OK);
        call(bytes, [&](size_t b) {
            dgc_gated_ffn_args a{type, act, m, k, n, at(1), k + pad2, at(2, off), k + pad, at(3), k + pad2,
                                 out(4), n, out(5), n, out(6), n};
            return dgc_gated_ffn(&a, kSpace, b, nullptr);
        });
        CHECK(dgc_gated_ffn_workspace_bytes(m, k, n, back, &bytes) == DGC_OK);
        const bool dw = pick(4);
        call(bytes, [&](size_t b) {
            dgc_gated_ffn_backward_args a{type, grad, act | flag, m, k, n, at(7), n, at(1, off), k + pad, at(2),
                                          k + pad2, at(3), k + pad, at(5), n + pad, at(6), n, pick(4) ? out(8) : nullptr,
                                          k, dw ? out(9) : nullptr, k, dw ? out(10) : nullptr, k};
            return dgc_gated_ffn_backward(&a, kSpace, b, nullptr);
        });
    }
}

int main() {
    few_rows();
    workspaces();
    const int64_t m = 2048, d = 1024, f = 4096;
    gated(m, d, f, d, d, 0, 0, 0);
    gated(m, d, f, d + 64, d + 64, 0, 0, 0);
    gated(m, d, f, d + 8, d, 0, 0, 1);    // the one in rows of their own width stays
    gated(m, d, f, d, d + 8, 0, 0, 1);
    gated(m, d, f, d + 8, d + 16, 0, 0, 2);
    gated(m, d, f, d, d, 2, 0, 1);        // one of them off 16 bytes
    gated(m, d, f, d, d + 1, 0, 0, 1);
    gated(m, d, f, d + 64, d + 64, 0, 6, 2);
    gated(m, d, f, d + 3, d + 5, 4, 2, 2);
    std::printf("plan check: ok\n");
    return 0;
}
