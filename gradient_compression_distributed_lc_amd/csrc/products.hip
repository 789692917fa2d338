// products.hip -- products of rows with a weight, or with the weight of each
// row's expert:
//   y[t][o] = sum over k of a[t][k] * w[o][k]      (both with the reduction as the fast index)
//   y[t][c] = sum over o of a[t][o] * w[o][c]      (the input gradient: the weight's rows are the reduction)
// in bf16, fp16, fp32 and, the first form, in 8-bit integers with a scale per
// row of either side.  16-bit and fp32 sums are the matrix cores' fp32, integer
// sums are exact in 32 bits.
#include <algorithm>
#include <type_traits>

#include "ckpt8.h"
#include "experts.h"
#include "launch.h"

namespace {

using namespace tlc_ckpt8;
using namespace tlc_experts;
using tlc_internal::launch_blocks;

constexpr int kThreads = 256;

typedef int i4 __attribute__((ext_vector_type(4)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef int i16v __attribute__((ext_vector_type(16)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef __bf16 b8v __attribute__((ext_vector_type(8)));
typedef _Float16 h8v __attribute__((ext_vector_type(8)));

struct I8 {
    using Elem = int8_t;
};

struct ProductArgs {
    const void *a, *w;
    uint64_t a_stride, w_stride, w_expert;  // elements
    Experts experts;
    uint32_t n, k;                          // columns of y, length of the reduction
    const float *a_scales, *w_scales;       // 8-bit integers only
    void* y;
    uint64_t y_stride;
    int accumulate;
    uint32_t tiles_n;
    uint32_t first;                         // block of the whole that the launch begins with
};

// 32 rows by 32 rows over 32 bytes of the reduction: a lane holds 16 bytes of
// row lane%32 on each side, the first or the second by lane/32.
template <typename E>
struct Sums {
    using Type = f16v;
};
template <>
struct Sums<I8> {
    using Type = i16v;
};
template <typename E>
__device__ __forceinline__ typename Sums<E>::Type multiply(u4 a, u4 b, typename Sums<E>::Type c) {
    if constexpr (std::is_same<E, I8>::value)
        return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i4, a), __builtin_bit_cast(i4, b), c, 0, 0, 0);
    else if constexpr (std::is_same<E, BF16>::value)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8v, a), __builtin_bit_cast(b8v, b), c, 0, 0,
                                                       0);
    else if constexpr (std::is_same<E, F16>::value)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8v, a), __builtin_bit_cast(h8v, b), c, 0, 0,
                                                      0);
    else {
#pragma unroll
        for (int j = 0; j < 4; ++j)  // the reduction's order inside the 8 does not matter where both sides have it
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(from_bits(a[j]), from_bits(b[j]), c, 0, 0, 0);
        return c;
    }
}

// The first n of the elements in 16 bytes at p, the rest 0.
template <typename E>
__device__ __forceinline__ u4 load16(const typename E::Elem* p, int n) {
    if constexpr (sizeof(typename E::Elem) == 2) {
        return load8<E>(p, n).w[0];
    } else if constexpr (sizeof(typename E::Elem) == 4) {
        if (n >= 4) return *reinterpret_cast<const u4_at4*>(p);
        u4 r = {};
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (j < n) r[j] = reinterpret_cast<const uint32_t*>(p)[j];
        return r;
    } else {
        return *reinterpret_cast<const u4*>(p);  // codes are padded with zeros
    }
}

// The scales' product with a sum: the smaller scale first, so that nothing
// leaves fp32's range on the way that the result does not.  Three roundings.
__device__ __forceinline__ float scaled(int sum, float sa, float sw) {
    const bool below = sa < sw;  // false with a NaN, which then stays in one of the two
    return (float)sum * (below ? sa : sw) * (below ? sw : sa);
}

// Orders a wavefront's own LDS accesses across its lanes.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ s4v read_tr(const void* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4v*)p);
}

// A block computes kTile x kTile values of y, each of its four wavefronts a
// quarter, in steps of 128 bytes of the reduction.
template <typename E, typename Out, bool kInner, int kTile>
__global__ __launch_bounds__(kThreads, 2) void k_product(ProductArgs p) {
    using Elem = typename E::Elem;
    using Acc = typename Sums<E>::Type;
    constexpr int kPer = 16 / sizeof(Elem);     // elements of a 16-byte chunk
    constexpr int kStep = 128 / sizeof(Elem);   // of the reduction in a step
    constexpr int kLoads = kTile * 8 / kThreads;  // chunks a lane, of either operand
    constexpr int kWave = kTile / 2, kTiles = kWave / 32;
    __shared__ u4 stages[2][2][kTile * 8];

    uint32_t b = p.first + blockIdx.x;
    const uint32_t tiles_t = tiles_of(p.experts, kTile), total = tiles_t * p.tiles_n;
    if (b >= total) return;
    b = xcd_place(b, total);
    // bands of 4 tiles of rows
    const uint32_t band = b / (4 * p.tiles_n), in_band = b % (4 * p.tiles_n);
    const uint32_t band_rows = min(4u, tiles_t - band * 4);
    const Span at = tile_rows(p.experts, kTile, band * 4 + in_band % band_rows);
    const uint32_t o0 = in_band / band_rows * kTile;
    if (at.begin >= at.end) return;  // offsets that change meanwhile

    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const Elem* const a = static_cast<const Elem*>(p.a);
    const Elem* const w = static_cast<const Elem*>(p.w) + at.expert * p.w_expert;
    const int steps = (int)((p.k + kStep - 1) / kStep);

    // Rows of 128 bytes: slot c of row r holds chunk c ^ (r/2 % 8).
    const int row = tid / 8, chunk = tid % 8 ^ (row >> 1 & 7);
    u4 ga[kLoads], gw[kLoads];
    auto load = [&](int s) {
        const int left = (int)p.k - s * kStep - chunk * kPer;
        const uint64_t at_k = (uint64_t)s * kStep + (left > 0 ? chunk * kPer : 0);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t r = min(at.begin + row + i * 32, at.end - 1);
            ga[i] = left > 0 ? load16<E>(a + r * p.a_stride + at_k, left) : u4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if constexpr (!kInner) {
                const uint32_t r = min(o0 + row + i * 32, p.n - 1);
                gw[i] = left > 0 ? load16<E>(w + r * p.w_stride + at_k, left) : u4{0, 0, 0, 0};
            } else {
                constexpr int kChunks = kTile / kPer;  // of a row of the weight
                const uint32_t id = i * kThreads + tid, r = id / kChunks;
                const uint32_t c = sizeof(Elem) == 2 ? id % kChunks ^ ((r & 3) << 2 | (r & 1)) : id % kChunks;
                const uint32_t o = s * kStep + r, col = o0 + c * kPer;
                gw[i] = o < p.k && col < p.n ? load16<E>(w + o * p.w_stride + col, (int)(p.n - col)) : u4{0, 0, 0, 0};
            }
        }
    };
    auto store = [&](int s) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            stages[s & 1][0][i * kThreads + tid] = ga[i];
            stages[s & 1][1][i * kThreads + tid] = gw[i];
        }
    };

    const int wi = (wave >> 1) * kWave, wc = (wave & 1) * kWave;
    const int r32 = lane & 31, half = lane >> 5;
    Acc acc[kTiles][kTiles] = {};
    auto operand_rows = [&](const u4* st, int sub, int from) {  // of 32 rows beginning with `from`
        return st[(from + r32) * 8 + ((sub * 2 + half) ^ (r32 >> 1 & 7))];
    };
    auto operand_columns = [&](const u4* st, int sub, int from) {
        if constexpr (sizeof(Elem) == 2) {
            const int r = sub * 16 + half * 8 + (lane >> 2 & 3);
            const int slot = from / 8 + (lane >> 4 & 1) * 2 + (lane >> 1 & 1);
            const char* q = reinterpret_cast<const char*>(st) + r * kTile * 2 +
                            (slot ^ ((r & 3) << 2 | (r & 1))) * 16 + (lane & 1) * 8;
            const s4v lo = read_tr(q), hi = read_tr(q + 4 * kTile * 2);
            return __builtin_bit_cast(u4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(st) + (sub * 8 + half * 4) * kTile + from + r32;
            return u4{q[0], q[kTile], q[2 * kTile], q[3 * kTile]};
        }
    };
    if (steps > 0) {
        load(0);
        store(0);
    }
    __syncthreads();
    for (int s = 0; s < steps; ++s) {
        if (s + 1 < steps) load(s + 1);
#pragma unroll
        for (int sub = 0; sub < 4; ++sub) {
            u4 fa[kTiles], fb[kTiles];
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                fa[i] = operand_rows(stages[s & 1][0], sub, wi + i * 32);
                fb[i] = kInner ? operand_columns(stages[s & 1][1], sub, wc + i * 32)
                               : operand_rows(stages[s & 1][1], sub, wc + i * 32);
            }
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
#pragma unroll
                for (int c = 0; c < kTiles; ++c) acc[i][c] = multiply<E>(fa[i], fb[c], acc[i][c]);
        }
        if (s + 1 < steps) store(s + 1);
        __syncthreads();
    }

    // register j of a lane: row 8*(j/4) + 4*(lane/32) + j%4, column lane%32.
    // 32 rows at a time through LDS, so that a lane has eight values of a row.
    uint32_t* const mine = reinterpret_cast<uint32_t*>(&stages[0][0][0]) + wave * 32 * kWave;
    constexpr int kAcross = kWave / 8, kDown = 64 / kAcross;
    const uint32_t col = o0 + wc + lane % kAcross * 8;
    const int count = (int)min((int64_t)p.n - (int64_t)col, (int64_t)8);
    float sw[8];
    if constexpr (std::is_same<E, I8>::value) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sw[j] = j < count ? p.w_scales[(uint64_t)at.expert * p.n + col + j] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int c = 0; c < kTiles; ++c) {
                const auto v = acc[i][c][j];
                mine[((j >> 2) * 8 + half * 4 + (j & 3)) * kWave + c * 32 + r32] = __builtin_bit_cast(uint32_t, v);
            }
        wave_sync();
#pragma unroll
        for (int q = 0; q < 32; q += kDown) {
            const uint32_t r = q + lane / kAcross, t = at.begin + wi + i * 32 + r;
            if (t < at.end && count > 0) {
                const u4* const in = reinterpret_cast<const u4*>(mine + r * kWave + lane % kAcross * 8);
                const u4 lo = in[0], hi = in[1];
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t u = j < 4 ? lo[j & 3] : hi[j & 3];
                    if constexpr (std::is_same<E, I8>::value)
                        v[j] = scaled((int)u, p.a_scales[t], sw[j]);
                    else
                        v[j] = from_bits(u);
                }
                typename Out::Elem* const o = static_cast<typename Out::Elem*>(p.y) + t * p.y_stride + col;
                if constexpr (std::is_same<Out, F32>::value) {
                    if (p.accumulate) {
                        float old[8];
                        unpack8<Out>(load8<Out>(o, count), old);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += old[j];
                    }
                }
                store8<Out>(o, count, pack8<Out>(v));
            }
        }
        wave_sync();
    }
}

template <typename E, typename Out, bool kInner>
int product(const char* name, ProductArgs p, hipStream_t st) {
    const uint64_t tiles_t = most_tiles(p.experts.rows, p.experts.count, 128, p.experts.offsets != nullptr);
    p.tiles_n = (p.n + 127) / 128;
    return launch_blocks(name, st, tiles_t * p.tiles_n, kThreads, [&](uint64_t first, uint32_t blocks) {
        p.first = (uint32_t)first;
        k_product<E, Out, kInner, 128><<<blocks, kThreads, 0, st>>>(p);
    });
}

constexpr uint64_t kMaxTiles = 1u << 24;  // of 128 x 128

bool valid_product(uint64_t rows, uint64_t n, uint64_t k, const void* offsets, uint64_t experts) {
    if (!valid_shape(rows, n) || k < 1 || k > kMaxDim || experts < 1 || experts > kMaxExperts) return false;
    if (offsets ? !aligned(offsets, 8) : experts != 1) return false;
    return most_tiles(rows, experts, 128, offsets != nullptr) * ((n + 127) / 128) <= kMaxTiles;
}

int expert_call(const char* name, bool inner, const void* a, uint64_t a_stride, int dtype, uint64_t rows,
                uint64_t k, const void* w, uint64_t w_stride, uint64_t w_expert_stride, uint64_t w_cols, uint64_t n,
                const uint64_t* offsets, uint64_t experts, void* y, uint64_t y_stride, void*, size_t,
                tlc_stream_t stream) {
    if (!valid_dtype(dtype) || !valid_product(rows, n, k, offsets, experts) || w_expert_stride >> 48)
        return TLC_ERR_INVALID_ARG;
    if (rows == 0) return TLC_OK;
    if (!valid_matrix(a, dtype, k, a_stride) || !valid_matrix(w, dtype, w_cols, w_stride) ||
        !valid_matrix(y, dtype, n, y_stride))
        return TLC_ERR_INVALID_ARG;
    ProductArgs p = {};
    p.a = a, p.a_stride = a_stride, p.w = w, p.w_stride = w_stride, p.w_expert = w_expert_stride;
    p.experts = {offsets, (uint32_t)experts, (uint32_t)rows};
    p.n = (uint32_t)n, p.k = (uint32_t)k;
    p.y = y, p.y_stride = y_stride;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        return inner ? product<T, T, true>(name, p, st) : product<T, T, false>(name, p, st);
    });
}

}  // namespace

extern "C" {

size_t tlc_q8_product_workspace_size(uint64_t, uint64_t, uint64_t, uint64_t) { return 0; }
size_t tlc_expert_product_workspace_size(uint64_t, uint64_t, uint64_t, uint64_t, int) { return 0; }
size_t tlc_expert_input_grad_workspace_size(uint64_t, uint64_t, uint64_t, uint64_t, int) { return 0; }

int tlc_q8_product(const int8_t* a, const float* a_scales, uint64_t rows, const int8_t* w, const float* w_scales,
                   uint64_t n, uint64_t k, const uint64_t* offsets, uint64_t experts, void* y, uint64_t y_stride,
                   int dtype, int accumulate, void*, size_t, tlc_stream_t stream) {
    const uint64_t stride = tlc_q8_code_stride(k);
    if (!valid_dtype(dtype) || !stride || !valid_product(rows, n, k, offsets, experts) ||
        (accumulate && dtype != TLC_F32))
        return TLC_ERR_INVALID_ARG;
    if (rows == 0) return TLC_OK;
    if (!a || !w || !aligned(a, 16) || !aligned(w, 16) || !a_scales || !w_scales || !aligned(a_scales, 4) ||
        !aligned(w_scales, 4) || !valid_matrix(y, dtype, n, y_stride))
        return TLC_ERR_INVALID_ARG;
    ProductArgs p = {};
    p.a = a, p.a_stride = stride, p.w = w, p.w_stride = stride, p.w_expert = n * stride;
    p.experts = {offsets, (uint32_t)experts, (uint32_t)rows};
    p.n = (uint32_t)n, p.k = (uint32_t)stride;
    p.a_scales = a_scales, p.w_scales = w_scales;
    p.y = y, p.y_stride = y_stride, p.accumulate = accumulate != 0;
    return with_dtype(dtype, [&](auto t) {
        return product<I8, decltype(t), false>("tlc_q8_product", p, static_cast<hipStream_t>(stream));
    });
}

int tlc_expert_product(const void* x, uint64_t x_stride, int dtype, uint64_t rows, uint64_t k, const void* w,
                       uint64_t w_stride, uint64_t w_expert_stride, uint64_t n, const uint64_t* offsets,
                       uint64_t experts, void* y, uint64_t y_stride, void* workspace, size_t workspace_bytes,
                       tlc_stream_t stream) {
    return expert_call("tlc_expert_product", false, x, x_stride, dtype, rows, k, w, w_stride, w_expert_stride, k, n,
                       offsets, experts, y, y_stride, workspace, workspace_bytes, stream);
}

int tlc_expert_input_grad(const void* dy, uint64_t dy_stride, int dtype, uint64_t rows, uint64_t n, const void* w,
                          uint64_t w_stride, uint64_t w_expert_stride, uint64_t k, const uint64_t* offsets,
                          uint64_t experts, void* dx, uint64_t dx_stride, void* workspace, size_t workspace_bytes,
                          tlc_stream_t stream) {
    return expert_call("tlc_expert_input_grad", true, dy, dy_stride, dtype, rows, n, w, w_stride, w_expert_stride, k,
                       k, offsets, experts, dx, dx_stride, workspace, workspace_bytes, stream);
}

}  // extern "C"
