// ckpt8_matrix.hip -- the weight gradient from an 8-bit checkpoint:
//   dw[i][c] (+)= col_scale[c] * sum over rows t of dy[t][i] * x[t][c],
// x the checkpoint's values.  x is a bfloat16 number as it stands, dy is one
// (bf16), the sum of two (fp16) or of three (fp32) of them, so every product is
// exact and the sums are the matrix cores' fp32.

#include <algorithm>

#include "ckpt8.h"
#include "launch.h"

namespace {

using namespace tlc_ckpt8;
using tlc_internal::launch;

constexpr int kThreads = 256;
constexpr int kTile = 128;   // rows and columns of dw a block computes
constexpr int kStep = 32;    // rows of dy and x it takes at a time
constexpr int kLdsRow = 40;  // bfloat16 numbers between columns in LDS: 32 and a pad of 16 bytes

typedef short s8v __attribute__((ext_vector_type(8)));
typedef __bf16 b8v __attribute__((ext_vector_type(8)));

struct MatArgs {
    const void* dy;
    uint64_t dy_stride;
    const uint8_t *codes, *scales;
    uint64_t rows;
    uint32_t n, cols;
    uint32_t code_row, scale_row;
    const void* col_scale;
    int accumulate;
    float* dw;           // with one slice
    uint64_t dw_stride;
    float* partial;      // [slices][n][cols], else nullptr
    uint64_t slice_rows; // rows of one slice, a multiple of kStep
    uint32_t tiles, tiles_c;  // tiles of dw, and of one row of them
};

// v as a sum of bfloat16 numbers, each the leading bits of what is left.
template <int kTerms>
__device__ __forceinline__ void split(float v, uint16_t* t) {
#pragma unroll
    for (int k = 0; k < kTerms; ++k) {
        const uint32_t u = to_bits(v);
        t[k] = (uint16_t)(u >> 16);
        if (k + 1 < kTerms) v = (u & 0x7FFFFFFFu) == 0x7F800000u ? 0.0f : v - from_bits(u & 0xFFFF0000u);
    }
}

template <typename W>
__device__ __forceinline__ float column_scale(const void* p, uint32_t c) {
    if (!p) return 1.0f;
    return (float)static_cast<const typename W::Elem*>(p)[c];
}

template <typename T, typename W, int FMT>
__global__ __launch_bounds__(kThreads) void k_weight_grad(MatArgs p) {
    constexpr int kTerms = T::kTerms;
    __shared__ __align__(16) uint16_t sa[kTerms][kTile][kLdsRow];
    __shared__ __align__(16) uint16_t sb[kTile][kLdsRow];
    const uint32_t slice = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles;
    const uint32_t i0 = tile / p.tiles_c * kTile, c0 = tile % p.tiles_c * kTile;
    const uint64_t t_begin = slice * p.slice_rows, t_end = min(p.rows, t_begin + p.slice_rows);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int wi = (wave >> 1) * 64, wc = (wave & 1) * 64;
    f4 acc[4][4] = {};
    for (uint64_t t0 = t_begin; t0 < t_end; t0 += kStep) {
        // 32 rows of 128 columns of each: 16 lanes of eight columns a row
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = (threadIdx.x >> 4) + 16 * h, q = (threadIdx.x & 15) * 8;
            const uint64_t t = t0 + r;
            const int left = (int)(p.n - i0) - q;
            const int cnt = t < t_end ? min(max(left, 0), 8) : 0;
            float v[8];
            unpack8<T>(load8<T>(static_cast<const typename T::Elem*>(p.dy) + t * p.dy_stride + i0 + q, cnt), v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint16_t term[kTerms];
                split<kTerms>(v[j], term);
#pragma unroll
                for (int k = 0; k < kTerms; ++k) sa[k][q + j][r] = term[k];
            }
            u2 code = {0, 0};
            uint32_t byte = 0;
            if (t < t_end && c0 + q < p.code_row) {
                code = *reinterpret_cast<const u2*>(p.codes + t * p.code_row + c0 + q);
                byte = p.scales[t * p.scale_row + (c0 + q) / 32];
            }
            decode8<FMT>(code, byte, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) sb[q + j][r] = (uint16_t)(to_bits(v[j]) >> 16);
        }
        __syncthreads();
        // lane l of a 16x16x32 product: row (column) l%16, reduction l/16*8 .. +7
        const int fr = lane & 15, fk = (lane >> 4) * 8;
        b8v fb[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) fb[c] = *reinterpret_cast<const b8v*>(&sb[wc + c * 16 + fr][fk]);
#pragma unroll
        for (int k = 0; k < kTerms; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const b8v fa = *reinterpret_cast<const b8v*>(&sa[k][wi + i * 16 + fr][fk]);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    acc[i][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa, fb[c], acc[i][c], 0, 0, 0);
            }
        }
        __syncthreads();
    }
    // lane l holds rows l/16*4 .. +3 of column l%16
    const uint32_t row0 = i0 + wi + (lane >> 4) * 4, col0 = c0 + wc + (lane & 15);
    const bool direct = p.partial == nullptr;
    float* const out = direct ? p.dw : p.partial + (uint64_t)slice * p.n * p.cols;
    const uint64_t stride = direct ? p.dw_stride : p.cols;
    float cs[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) cs[c] = column_scale<W>(direct ? p.col_scale : nullptr, min(col0 + c * 16, p.cols - 1));
    const bool add = direct && p.accumulate;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t row = row0 + i * 16 + j;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t col = col0 + c * 16;
                if (row < p.n && col < p.cols) {
                    float* const o = out + row * stride + col;
                    const float v = acc[i][c][j] * cs[c];
                    *o = add ? *o + v : v;
                }
            }
        }
}

// dw (+)= col_scale * the slices' sums, added in order; no slices: 0.
template <typename W>
__global__ __launch_bounds__(kThreads) void k_weight_sum(MatArgs p, uint32_t slices) {
    const uint64_t per_row = (p.cols + kThreads - 1) / kThreads;
    for (uint64_t b = blockIdx.x; b < per_row * p.n; b += gridDim.x) {
        const uint64_t row = b / per_row;
        const uint32_t c = (uint32_t)(b - row * per_row) * kThreads + threadIdx.x;
        if (c >= p.cols) continue;
        float s = 0.0f;
        for (uint32_t k = 0; k < slices; ++k) s += p.partial[((uint64_t)k * p.n + row) * p.cols + c];
        s *= column_scale<W>(p.col_scale, c);
        float* const o = p.dw + row * p.dw_stride + c;
        *o = p.accumulate ? *o + s : s;
    }
}

// Slices of the rows: enough blocks for the chip, none below 256 rows.
struct Slices {
    uint32_t count;
    uint64_t rows;
};
Slices slices_of(uint64_t rows, uint64_t n, uint64_t cols) {
    const uint64_t tiles = ((n + kTile - 1) / kTile) * ((cols + kTile - 1) / kTile);
    uint64_t want = std::min<uint64_t>((512 + tiles - 1) / tiles, std::max<uint64_t>(rows / 256, 1));
    Slices s;
    s.rows = ((rows + want - 1) / want + kStep - 1) / kStep * kStep;
    s.count = s.rows ? (uint32_t)((rows + s.rows - 1) / s.rows) : 0;
    return s;
}

}  // namespace

extern "C" {

size_t tlc_ckpt8_weight_grad_workspace_size(uint64_t rows, uint64_t n, uint64_t cols) {
    if (!valid_shape(rows, cols) || n < 1 || n > kMaxDim) return 0;
    const Slices s = slices_of(rows, n, cols);
    const uint64_t bytes = s.count > 1 ? (uint64_t)s.count * n * cols * sizeof(float) : 0;
    return std::max<size_t>((bytes + 255) / 256 * 256, 256);
}

int tlc_ckpt8_weight_grad(const void* dy, uint64_t dy_stride, int dtype, uint64_t rows, uint64_t n, int format,
                          const uint8_t* codes, const uint8_t* scales, uint64_t cols, const void* col_scale,
                          int col_scale_dtype, float* dw, uint64_t dw_stride, int accumulate, void* workspace,
                          size_t workspace_bytes, tlc_stream_t stream) {
    if (!valid_dtype(dtype) || !valid_format(format) || !valid_shape(rows, cols) || n < 1 || n > kMaxDim ||
        !valid_matrix(dw, TLC_F32, cols, dw_stride))
        return TLC_ERR_INVALID_ARG;
    if (rows && (!valid_matrix(dy, dtype, n, dy_stride) || !valid_checkpoint(codes, scales)))
        return TLC_ERR_INVALID_ARG;
    if (!valid_weight(col_scale, col_scale_dtype, dtype)) return TLC_ERR_INVALID_ARG;
    const uint64_t ti = (n + kTile - 1) / kTile, tc = (cols + kTile - 1) / kTile;
    if (ti * tc > (1u << 30)) return TLC_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < tlc_ckpt8_weight_grad_workspace_size(rows, n, cols))
        return TLC_ERR_WORKSPACE;
    if (rows == 0 && accumulate) return TLC_OK;
    const Slices s = slices_of(rows, n, cols);
    MatArgs p;
    p.dy = dy, p.dy_stride = dy_stride, p.codes = codes, p.scales = scales, p.rows = rows;
    p.n = (uint32_t)n, p.cols = (uint32_t)cols;
    p.code_row = (uint32_t)code_stride(cols), p.scale_row = (uint32_t)scale_stride(cols);
    p.col_scale = col_scale;
    p.dw = dw, p.dw_stride = dw_stride, p.accumulate = accumulate != 0;
    p.partial = s.count > 1 ? static_cast<float*>(workspace) : nullptr;
    p.slice_rows = s.rows;
    p.tiles = (uint32_t)(ti * tc), p.tiles_c = (uint32_t)tc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (s.count) {
        const uint32_t grid = p.tiles * s.count;
        const int rc = with_dtype(dtype, [&](auto t) {
            return with_weight(t, col_scale, col_scale_dtype, [&](auto w) {
                return with_format(format, [&](auto f) {
                    return launch("tlc_ckpt8_weight_grad", st, [&] {
                        k_weight_grad<decltype(t), decltype(w), decltype(f)::value><<<grid, kThreads, 0, st>>>(p);
                    });
                });
            });
        });
        if (rc || s.count == 1) return rc;
    }
    const uint32_t blocks = (uint32_t)std::min<uint64_t>(n * ((cols + kThreads - 1) / kThreads), 1u << 20);
    return with_dtype(dtype, [&](auto t) {
        return with_weight(t, col_scale, col_scale_dtype, [&](auto w) {
            return launch("tlc_ckpt8_weight_sum", st, [&] {
                k_weight_sum<decltype(w)><<<blocks, kThreads, 0, st>>>(p, s.count);
            });
        });
    });
}

}  // extern "C"
