// tokens_host_check.cpp -- exercises the host code of the token operators
// (argument checks, workspace sizes; no GPU calls) for a build with
// AddressSanitizer and UndefinedBehaviorSanitizer.  Built and run by
// tests/test_tokens_abi.py.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>

#include "dgc.h"

#define CHECK(c)                                                             \
    do {                                                                     \
        if (!(c)) {                                                          \
            std::fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__); \
            std::abort();                                                    \
        }                                                                    \
    } while (0)

int main() {
    std::mt19937_64 rng(12);
    void* const at = reinterpret_cast<void*>(4096);
    float* const f = static_cast<float*>(at);
    for (int round = 0; round < 20000; ++round) {
        int64_t s[3];
        for (int64_t& v : s) {
            const int bits = int(rng() % 33);
            v = int64_t(rng() % (uint64_t(1) << bits)) + int64_t(rng() % 3) - 1;
        }
        const int64_t m = s[0], d = s[1], n = s[2];
        const bool fine = m >= 0 && d >= 0 && m < (int64_t(1) << 31) && d < (int64_t(1) << 31);
        const bool fits = fine && (d == 0 || m <= (int64_t(1) << 48) / d);
        const bool third = n >= 0 && n < (int64_t(1) << 31);
        for (int back = 0; back < 2; ++back) {
            size_t bytes = 0, more = 0;
            CHECK((dgc_layer_norm_workspace_bytes(m, d, back, &bytes) == DGC_OK) == fits);
            CHECK((dgc_embedding_workspace_bytes(m, n, d, back, &bytes) == DGC_OK) == (fits && third));
            CHECK((dgc_recurrence_workspace_bytes(m, d, n, back, &more) == DGC_OK) == (fits && third));
            if (fits && third && m > 0 && d > 0) {
                CHECK(back ? bytes > 0 : bytes == 0);
                CHECK(n == 0 ? more == 0 : more > 0);
            }
        }
        // refused by a leading dimension that is too small, whatever the sizes are
        if (!(m > 0 && d > 0)) continue;
        const dgc_layer_norm_args a{DGC_BF16, DGC_FP32, m, d, 1e-5, at, d, at, at, at, d - 1, f, f};
        CHECK(dgc_layer_norm(&a, nullptr) == DGC_EINVAL);
        const dgc_layer_norm_backward_args b{DGC_BF16, DGC_BF16, DGC_FP32, m, d, at, d, at, d, f, f,
                                             at,       at,       d - 1,    at, d, at, at};
        CHECK(dgc_layer_norm_backward(&b, at, ~size_t(0), nullptr) == DGC_EINVAL);
        const dgc_dropout_args c{DGC_FP16, m, d, 0.5, rng(), rng(), nullptr, at, d, at, d - 1, at, d};
        CHECK(dgc_dropout(&c, nullptr) == DGC_EINVAL);
        const dgc_embedding_args e{DGC_FP32, DGC_INT64, m, 10, d, at, at, d - 1, 1.0, at, d};
        CHECK(dgc_embedding(&e, nullptr) == DGC_EINVAL);
        const dgc_embedding_backward_args g{DGC_FP32, DGC_FP32, DGC_INT32, m, 10, d, 1, at, d, at, 1.0, at, d - 1};
        CHECK(dgc_embedding_backward(&g, at, ~size_t(0), nullptr) == DGC_EINVAL);
        const dgc_recurrence_args r{DGC_BF16, DGC_INT32, m, d, 1, nullptr, at, d, at, d, f, d, at, d - 1, f, d};
        CHECK(dgc_recurrence(&r, at, ~size_t(0), nullptr) == DGC_EINVAL);
        const dgc_recurrence_backward_args q{DGC_BF16, DGC_INT64, m, d,  1, at, at, d, at, d,     at, d, at, d,
                                             f,        d,         f, d, at, d,  at, d, f,  d - 1};
        CHECK(dgc_recurrence_backward(&q, at, ~size_t(0), nullptr) == DGC_EINVAL);
        // ... or for want of room
        if (!fits) continue;
        size_t need = 0;
        CHECK(dgc_recurrence_workspace_bytes(m, d, 1, 0, &need) == DGC_OK);
        const dgc_recurrence_args p{DGC_BF16, DGC_INT32, m, d, 1, nullptr, at, d, at, d, f, d, at, d, f, d};
        CHECK(dgc_recurrence(&p, at, need - 1, nullptr) == DGC_ECAPACITY);
    }
    std::printf("host check: ok\n");
    return 0;
}
