// Host-only checks of the 8-bit integer and grouped products, built together
// with their sources with AddressSanitizer and UndefinedBehaviorSanitizer on the
// host code: strides and workspace sizes over the whole range of sizes, and
// calls that every entry point must refuse before a launch.  Nothing here
// touches a GPU: device pointers are fake addresses that are never followed.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <random>

#include "tlc.h"

static int failures = 0;
#define CHECK(cond)                                                          \
    do {                                                                     \
        if (!(cond)) {                                                       \
            std::fprintf(stderr, "check failed, line %d: %s\n", __LINE__, #cond); \
            ++failures;                                                      \
        }                                                                    \
    } while (0)

int main() {
    const uint64_t top = 0x7FFFFFFFull, big = top + 1;
    CHECK(tlc_q8_code_stride(0) == 0 && tlc_q8_code_stride(131073) == 0 && tlc_q8_code_stride(~0ull) == 0);
    CHECK(tlc_q8_code_stride(131072) == 131072 && tlc_q8_code_stride(1) == 128);
    std::mt19937_64 rng(7);
    auto size = [&](int least) { return 1 + (rng() >> (least + rng() % (63 - least))); };
    for (int k = 0; k < 200000; ++k) {
        const uint64_t rows = size(33) - 1, n = size(34), cols = size(34), experts = size(47);
        const size_t c = tlc_q8_pack_columns_workspace_size(rows, cols);
        CHECK(c % 256 == 0 && (c > 0) == (rows >= 1 && rows <= 131072 && cols <= top));
        const size_t g = tlc_expert_weight_grad_workspace_size(rows, n, cols, experts);
        CHECK(g % 256 == 0 && (g > 0) == (rows <= top && n <= top && cols <= top && experts <= 65536));
        for (int dtype = 0; dtype < 3; ++dtype) {
            const size_t y = tlc_expert_product_workspace_size(rows, cols, n, experts, dtype);
            const size_t dx = tlc_expert_input_grad_workspace_size(rows, cols, n, experts, dtype);
            // the sums of at most 32 slices
            CHECK(y % 256 == 0 && y / 32 <= rows * (n + 7) * 4 + 256);
            CHECK(dx % 256 == 0 && dx / 32 <= rows * (n + 7) * 4 + 256);
        }
        const size_t q = tlc_q8_product_workspace_size(rows, n, cols, experts);
        CHECK(q % 256 == 0 && q / 32 <= rows * (n + 7) * 4 + 256 && (cols <= 131072 || q == 0));
    }
    for (uint64_t v : {uint64_t(0), uint64_t(big), uint64_t(~0ull)}) {
        CHECK(tlc_expert_product_workspace_size(v, v, v, v, 0) == 0);
        CHECK(tlc_expert_input_grad_workspace_size(v, 64, 64, 1, 1) == 0);
        CHECK(tlc_q8_product_workspace_size(64, v, 64, 1) == 0 && tlc_q8_product_workspace_size(64, 64, v, 1) == 0);
        CHECK(tlc_expert_weight_grad_workspace_size(64, v, 64, 1) == 0);
        CHECK(tlc_q8_pack_columns_workspace_size(64, v) == 0);
    }
    CHECK(tlc_expert_product_workspace_size(64, 64, 64, 1, 3) == 0);

    void* const p = reinterpret_cast<void*>(0x10000);
    int8_t* const c = static_cast<int8_t*>(p);
    uint8_t* const u = static_cast<uint8_t*>(p);
    float* const f = static_cast<float*>(p);
    uint64_t* const o = static_cast<uint64_t*>(p);
    const int bad = TLC_ERR_INVALID_ARG;
    CHECK(tlc_q8_pack_rows(p, 64, 2, ~0ull, 40, c, f, nullptr) == bad);
    CHECK(tlc_q8_pack_rows(p, 64, 2, 4, ~0ull, c, f, nullptr) == bad);
    CHECK(tlc_q8_pack_rows(p, ~0ull, 2, 4, 40, c, f, nullptr) == bad);
    CHECK(tlc_q8_pack_rows(nullptr, 64, 2, 0, 40, nullptr, nullptr, nullptr) == TLC_OK);
    CHECK(tlc_q8_pack_columns(p, 64, 2, 0, 40, c, f, p, 1 << 20, nullptr) == bad);
    CHECK(tlc_q8_pack_columns(p, 64, 2, 4, 40, c, f, nullptr, 0, nullptr) == TLC_ERR_WORKSPACE);
    CHECK(tlc_q8_product(c, f, ~0ull, c, f, 24, 40, o, 2, p, 24, 0, 0, p, 1 << 30, nullptr) == bad);
    CHECK(tlc_q8_product(c, f, 4, c, f, ~0ull, 40, o, 2, p, 24, 0, 0, p, 1 << 30, nullptr) == bad);
    CHECK(tlc_q8_product(c, f, 4, c, f, 24, 40, o, ~0ull, p, 24, 0, 0, p, 1 << 30, nullptr) == bad);
    CHECK(tlc_q8_product(c, f, top, c, f, top, 40, nullptr, 1, p, top, 0, 0, p, 1 << 30, nullptr) == bad);
    CHECK(tlc_q8_product(nullptr, nullptr, 0, c, f, 24, 40, o, 2, nullptr, 24, 0, 0, nullptr, 0, nullptr) == TLC_OK);
    CHECK(tlc_expert_product(p, 64, 2, ~0ull, 40, p, 64, 960, 24, o, 2, p, 24, p, 1 << 30, nullptr) == bad);
    CHECK(tlc_expert_product(p, 64, 2, 4, ~0ull, p, 64, 960, 24, o, 2, p, 24, p, 1 << 30, nullptr) == bad);
    CHECK(tlc_expert_product(p, 64, 2, 4, 40, p, 64, ~0ull, 24, o, 2, p, 24, p, 1 << 30, nullptr) == bad);
    CHECK(tlc_expert_product(p, (1 << 22) + 1, 2, 4, 40, p, 64, 960, 24, o, 2, p, 24, p, 1 << 30, nullptr) == bad);
    CHECK(tlc_expert_input_grad(p, 64, 2, 4, 24, p, (1 << 22) + 1, 960, 40, o, 2, p, 40, p, 1 << 30, nullptr) == bad);
    // a reduction in slices without a workspace for them
    const size_t need = tlc_expert_product_workspace_size(128, 4096, 256, 1, 2);
    CHECK(need > 0);
    CHECK(tlc_expert_product(p, 4096, 2, 128, 4096, p, 4096, 0, 256, nullptr, 1, p, 256, nullptr, 0, nullptr) ==
          TLC_ERR_WORKSPACE);
    CHECK(tlc_expert_product(p, 4096, 2, 128, 4096, p, 4096, 0, 256, nullptr, 1, p, 256, p, need - 1, nullptr) ==
          TLC_ERR_WORKSPACE);
    CHECK(tlc_expert_weight_grad(p, 64, 2, 4, ~0ull, 1, u, u, 40, o, 2, nullptr, 0, f, 40, 960, 0, p, 1 << 30,
                                 nullptr) == bad);
    CHECK(tlc_expert_weight_grad(p, 64, 2, 4, 24, 1, u, u, 40, o, 2, nullptr, 0, f, 40, ~0ull, 0, p, 1 << 30,
                                 nullptr) == bad);
    CHECK(tlc_expert_weight_grad(p, 64, 2, 4, 24, 1, u, u, 40, o, 65537, nullptr, 0, f, 40, 960, 0, p, 1 << 30,
                                 nullptr) == bad);
    if (failures) return 1;
    std::printf("product host checks ok\n");
    return 0;
}
