// Host-only checks of the 8-bit checkpoint calls, built together with their
// sources with AddressSanitizer and UndefinedBehaviorSanitizer on the host
// code: strides and workspace sizes over the whole range of sizes, and calls
// that every entry point must refuse before a launch.  Nothing here touches a
// GPU: device pointers are fake addresses that are never followed.
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
    const uint64_t big = 1ull << 31, top = big - 1;
    CHECK(tlc_ckpt8_code_stride(0) == 0 && tlc_ckpt8_code_stride(big) == 0 && tlc_ckpt8_scale_stride(big) == 0);
    CHECK(tlc_ckpt8_code_stride(top) == 1ull << 31 && tlc_ckpt8_scale_stride(top) == 1ull << 26);
    std::mt19937_64 rng(7);
    for (int k = 0; k < 200000; ++k) {
        const uint64_t rows = rng() >> (33 + rng() % 31), n = 1 + (rng() >> (34 + rng() % 30)),
                       cols = 1 + (rng() >> (34 + rng() % 30));
        const size_t w = tlc_ckpt8_weight_grad_workspace_size(rows, n, cols);
        CHECK(w % 256 == 0 && (w > 0) == (rows <= top && n <= top && cols <= top));
        const size_t g = tlc_ckpt8_norm_grad_workspace_size(rows, cols);
        CHECK(g % 256 == 0 && (g > 0) == (rows <= top && cols <= 16384));
    }
    void* const p = reinterpret_cast<void*>(0x10000);
    uint8_t* const b = static_cast<uint8_t*>(p);
    float* const f = static_cast<float*>(p);
    const int bad = TLC_ERR_INVALID_ARG;
    CHECK(tlc_ckpt8_pack(nullptr, 64, 2, 4, 40, 1, b, b, nullptr) == bad);
    CHECK(tlc_ckpt8_pack(p, big, 2, 4, 40, 1, b, b, nullptr) == bad);
    CHECK(tlc_ckpt8_pack(p, 64, 2, ~0ull, 40, 1, b, b, nullptr) == bad);
    CHECK(tlc_ckpt8_pack(p, 64, 2, 4, ~0ull, 1, b, b, nullptr) == bad);
    CHECK(tlc_ckpt8_unpack(b, nullptr, 1, 4, 40, p, 64, 2, nullptr) == bad);
    CHECK(tlc_ckpt8_act(9, p, 64, p, 64, 2, 4, 40, p, 64, 1, b, b, b, b, nullptr) == bad);
    CHECK(tlc_ckpt8_act(1, p, 64, nullptr, 0, 2, 4, 40, p, 64, 1, b, b, b, b, nullptr) == bad);
    CHECK(tlc_ckpt8_act_grad(1, b, b, b, nullptr, 1, p, 64, 2, 4, 40, p, 64, p, 64, b, b, nullptr) == bad);
    CHECK(tlc_ckpt8_norm(p, 64, p, 64, 2, 4, 16385, p, 2, 1e-5f, 0, p, 64, p, 64, 1, b, b, f, nullptr) == bad);
    CHECK(tlc_ckpt8_norm(p, 64, p, 64, 2, 4, 40, p, 1, 1e-5f, 0, p, 64, p, 64, 1, b, b, f, nullptr) == bad);
    CHECK(tlc_ckpt8_norm_grad(p, 64, p, 64, 2, ~0ull, 40, nullptr, 0, 1, b, b, f, p, 2, p, 64, f, 0, p, 1u << 30,
                              nullptr) == bad);
    CHECK(tlc_ckpt8_norm_grad(p, 64, p, 64, 2, 4, 40, nullptr, 0, 1, b, b, f, p, 2, p, 64, f, 0, nullptr, 0, nullptr) ==
          TLC_ERR_WORKSPACE);
    CHECK(tlc_ckpt8_weight_grad(p, 64, 2, 4, top, 1, b, b, top, nullptr, 0, f, top, 0, p, ~size_t{0}, nullptr) == bad);
    CHECK(tlc_ckpt8_weight_grad(p, 64, 2, 4, 50, 1, b, b, 40, p, 2, f, 64, 0, p, 128, nullptr) == TLC_ERR_WORKSPACE);
    // no rows: nothing to write, no pointer asked for
    CHECK(tlc_ckpt8_pack(nullptr, 40, 2, 0, 40, 1, nullptr, nullptr, nullptr) == TLC_OK);
    CHECK(tlc_ckpt8_weight_grad(nullptr, 50, 2, 0, 50, 1, nullptr, nullptr, 40, nullptr, 0, f, 40, 1, p, 256, nullptr) ==
          TLC_OK);
    if (failures) return 1;
    std::puts("ckpt8 host checks ok");
    return 0;
}
