// layers_host_check.cpp -- exercises the host code of the layer and
// gradient-set operators (planning, argument checks; no GPU calls) for a
// build with AddressSanitizer and UndefinedBehaviorSanitizer.  Built and run
// by tests/test_layers_abi.py.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "dgc.h"

#define CHECK(c)                                                             \
    do {                                                                     \
        if (!(c)) {                                                          \
            std::fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__); \
            std::abort();                                                    \
        }                                                                    \
    } while (0)

int main() {
    std::mt19937_64 rng(11);
    size_t bytes = 0;
    void* at = reinterpret_cast<void*>(4096);
    for (int round = 0; round < 20000; ++round) {
        int64_t s[3];
        for (int64_t& v : s) {
            const int bits = int(rng() % 42);
            v = int64_t(rng() % (uint64_t(1) << bits)) + int64_t(rng() % 3) - 1;
        }
        for (int back = 0; back < 2; ++back) {
            const int a = dgc_linear_workspace_bytes(s[0], s[1], s[2], back, &bytes);
            const int b = dgc_gated_ffn_workspace_bytes(s[0], s[1], s[2], back, &bytes);
            CHECK(a == b && (a == DGC_OK || a == DGC_EINVAL));
        }
        dgc_linear_args l{DGC_BF16, int64_t(rng() % 5), s[0], s[1], s[2], at, s[2], at, s[2],
                          nullptr, nullptr, 0, at, s[1] - 1, nullptr, 0};
        if (s[0] > 0 && s[1] > 0) CHECK(dgc_linear(&l, nullptr, 0, nullptr) == DGC_EINVAL);
        dgc_gated_ffn_args g{DGC_FP16, 2, s[0], s[1], s[2], at, s[1], at, s[1], at, s[1],
                             at, s[2] - 1, nullptr, 0, nullptr, 0};
        if (s[0] > 0 && s[2] > 0) CHECK(dgc_gated_ffn(&g, nullptr, 0, nullptr) == DGC_EINVAL);
    }
    for (int round = 0; round < 200; ++round) {
        const int T = 1 + int(rng() % 3000);
        std::vector<int64_t> sizes(T);
        std::vector<int32_t> types(T);
        for (int t = 0; t < T; ++t) {
            sizes[t] = int64_t(rng() % (rng() % 2 ? 100 : 50000000));
            types[t] = 1 + int(rng() % 3);
        }
        CHECK(dgc_gradset_bytes(T, sizes.data(), types.data(), &bytes) == DGC_OK && bytes > 0);
        dgc_gradset* set = reinterpret_cast<dgc_gradset*>(0x1);
        CHECK(dgc_gradset_init(&set, T, sizes.data(), types.data(), at, bytes - 1, nullptr) ==
              DGC_ECAPACITY);
        CHECK(set == nullptr);
        types[T - 1] = 0;
        CHECK(dgc_gradset_bytes(T, sizes.data(), types.data(), &bytes) == DGC_EINVAL);
    }
    dgc_gradset_destroy(nullptr);
    std::printf("host check: ok\n");
    return 0;
}
