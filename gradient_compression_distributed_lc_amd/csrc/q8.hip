// q8.hip -- matrices in 8-bit integers with one fp32 scale per row, made from
// the rows or from the columns of a matrix.  Their product is in products.hip.
//
// With amax a row's largest magnitude, its scale is amax/127 and a code is the
// nearest integer to x times 127/amax, both quotients rounded to fp32.  One
// fused multiply-add rounds that exact product once, to an integer:
// 1.5*2^23 + q holds q in its low byte.
#include <algorithm>

#include "ckpt8.h"
#include "launch.h"

namespace {

using namespace tlc_ckpt8;
using tlc_internal::launch_blocks;

constexpr int kThreads = 256;
constexpr uint64_t kMaxCols = 131072;  // 2^17 products of 127*127 stay in 32 bits
inline uint64_t q8_stride(uint64_t cols) { return (cols + 127) / 128 * 128; }

constexpr float kLeast = 0x1p-126f;

// Scale and inverse of a row whose largest magnitude has these bits.  Below
// 127*2^-126 the scale is 2^-126, so that both are normal; a row that is not
// finite has codes 0 and scale NaN.
__device__ __forceinline__ float scale_for(uint32_t amax, float* inverse) {
    const float a = from_bits(amax);
    if (amax >= 0x7F800000u) {
        *inverse = 0.0f;
        return from_bits(0x7FC00000u);
    }
    const bool small = a < 127.0f * kLeast;
    *inverse = small ? 0x1p126f : 127.0f / a;
    return small ? kLeast : a / 127.0f;
}

__device__ __forceinline__ uint32_t code(float v, float inverse) { return to_bits(fmaf(v, inverse, 12582912.0f)); }

__device__ __forceinline__ u2 codes8(const float* v, float inverse) {
    if (inverse == 0.0f) return u2{0, 0};
    uint32_t q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = code(v[j], inverse);
    return u2{low_bytes(q[0], q[1], q[2], q[3]), low_bytes(q[4], q[5], q[6], q[7])};
}

__device__ __forceinline__ uint32_t wave_max(uint32_t m) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    return m;
}

// ---- rows ------------------------------------------------------------------

struct RowArgs {
    const void* x;
    uint64_t x_stride;
    uint64_t rows;
    uint32_t cols, code_row;
    int8_t* codes;
    float* scales;
    uint64_t first;
};

// kWaves wavefronts share a row, U units of eight values a lane and turn.  A
// row of one turn stays in registers (up to 16384 columns); a longer one is read
// twice.  Bound by HBM: 16384x8192 bf16 in 63 to 71 us, 6.4 to 5.7 TB/s.
template <typename T, int kWaves, int U>
__global__ __launch_bounds__(kThreads) void k_pack_rows(RowArgs p) {
    constexpr int kLanes = kWaves * 64, kRows = kThreads / kLanes;
    __shared__ uint32_t box[4];
    const uint64_t row = (p.first + blockIdx.x) * kRows + (kRows > 1 ? threadIdx.x / kLanes : 0);
    if (kRows > 1 && row >= p.rows) return;  // whole wavefronts, and only where no barrier follows
    const uint32_t lane = threadIdx.x % kLanes;
    const typename T::Elem* const x = static_cast<const typename T::Elem*>(p.x) + row * p.x_stride;
    const uint32_t units = p.code_row / 8;
    Raw8<T> raw[U];
    uint32_t m = 0;
    for (uint32_t at = 0; at < units; at += kLanes * U) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const uint32_t u = at + lane + i * kLanes;
            raw[i] = load8<T>(x + (uint64_t)u * 8, (int)min((int64_t)p.cols - (int64_t)u * 8, (int64_t)8));
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float v[8];
            unpack8<T>(raw[i], v);
            m = max(m, amax8(v));
        }
    }
    m = wave_max(m);
    if constexpr (kWaves > 1) {
        if ((threadIdx.x & 63) == 0) box[threadIdx.x / 64] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) m = max(m, box[w]);
    }
    float inverse;
    const float scale = scale_for(m, &inverse);
    if (lane == 0) p.scales[row] = scale;
    int8_t* const out = p.codes + row * p.code_row;
    for (uint32_t at = 0; at < units; at += kLanes * U) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const uint32_t u = at + lane + i * kLanes;
            if (units > kLanes * U)
                raw[i] = load8<T>(x + (uint64_t)u * 8, (int)min((int64_t)p.cols - (int64_t)u * 8, (int64_t)8));
            float v[8];
            unpack8<T>(raw[i], v);
            if (u < units) *reinterpret_cast<u2*>(out + u * 8) = codes8(v, inverse);
        }
    }
}

// ---- columns ---------------------------------------------------------------

struct ColumnArgs {
    const void* x;
    uint64_t x_stride;
    uint32_t rows, cols;
    uint32_t code_row;    // bytes between the codes of two columns
    int8_t* codes;
    float* scales;
    uint32_t* maxima;     // [chunks][cols rounded up to 256]: bits of each chunk's largest magnitudes
    uint32_t chunks, chunk_rows, padded;
    uint32_t blocks_c;    // blocks side by side
    uint32_t row_tiles;   // of 128 rows, for a block of the second kernel
    uint64_t first;
};

// The largest magnitudes of 256 columns over a chunk of rows.  16384x4096 bf16,
// 134 MB, in 34 us.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_column_max(ColumnArgs p) {
    __shared__ uint32_t box[8][256];
    const uint64_t b = p.first + blockIdx.x;
    const uint32_t chunk = (uint32_t)(b / p.blocks_c), c0 = (uint32_t)(b % p.blocks_c) * 256;
    const uint32_t unit = threadIdx.x % 32, r0 = threadIdx.x / 32;
    const uint32_t begin = chunk * p.chunk_rows, end = min(p.rows, begin + p.chunk_rows);
    const int n = (int)min((int64_t)p.cols - (int64_t)(c0 + unit * 8), (int64_t)8);
    const typename T::Elem* const x = static_cast<const typename T::Elem*>(p.x) + (uint64_t)(c0 + unit * 8);
    uint32_t m[8] = {};
    constexpr int kDeep = 8;  // rows under way
    for (uint32_t r = begin + r0; r < end; r += 8 * kDeep) {
        Raw8<T> raw[kDeep];
#pragma unroll
        for (int i = 0; i < kDeep; ++i)  // past the end the last row again
            raw[i] = load8<T>(x + (uint64_t)min(r + i * 8, end - 1) * p.x_stride, n);
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            float v[8];
            unpack8<T>(raw[i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] = max(m[j], to_bits(v[j]) & 0x7FFFFFFFu);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) box[r0][unit * 8 + j] = m[j];
    __syncthreads();
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, box[i][threadIdx.x]);
    p.maxima[(uint64_t)chunk * p.padded + c0 + threadIdx.x] = most;
}

// Codes of 128 columns over row_tiles tiles of 128 rows, transposed through LDS.
// A thread takes 8 columns of 4 neighbouring rows, so that a column's four
// codes are one 32-bit word.  A column's 128 bytes lie as eight 16-byte slots at
// slot ^ (column/8 % 8), which spreads the words that a wavefront writes at once.
// The first values are on their way while the maxima are joined, and each tile's
// while the one before is written (4096x1024 bf16 12.7 -> 7.6 us).  16384x4096
// bf16 in 32 us, 6.3 TB/s; the matrix is read twice in all.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_pack_columns(ColumnArgs p) {
    __shared__ __align__(16) uint8_t box[128 * 128];
    __shared__ uint32_t most[2][128];
    const uint64_t b = p.first + blockIdx.x;
    const uint32_t band = (uint32_t)(b / p.blocks_c), c0 = (uint32_t)(b % p.blocks_c) * 128;
    const uint32_t tid = threadIdx.x;
    const uint32_t unit = tid % 16, quad = tid / 16;
    const int n = (int)min((int64_t)p.cols - (int64_t)(c0 + unit * 8), (int64_t)8);
    const typename T::Elem* const x = static_cast<const typename T::Elem*>(p.x) + (uint64_t)(c0 + unit * 8);
    Raw8<T> raw[2][4];
    auto load = [&](uint32_t r0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t r = r0 + h * 64 + quad * 4 + i;
                raw[h][i] = load8<T>(x + (uint64_t)r * p.x_stride, r < p.rows ? n : 0);
            }
    };
    const uint32_t begin = band * p.row_tiles * 128, end = min(p.code_row, begin + p.row_tiles * 128);
    load(begin);  // on its way while the maxima are joined
    uint32_t m = 0;
#pragma unroll 8
    for (uint32_t k = tid / 128; k < p.chunks; k += 2)
        m = max(m, p.maxima[(uint64_t)k * p.padded + c0 + tid % 128]);
    most[tid / 128][tid % 128] = m;
    __syncthreads();
    float inverse[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t c = unit * 8 + j;
        const float scale = scale_for(max(most[0][c], most[1][c]), &inverse[j]);
        if (band == 0 && quad == 0 && c0 + c < p.cols) p.scales[c0 + c] = scale;
    }
    for (uint32_t r0 = begin; r0 < end; r0 += 128) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t q[4][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v[8];
                unpack8<T>(raw[h][i], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) q[i][j] = inverse[j] == 0.0f ? 0u : code(v[j], inverse[j]);
            }
            const uint32_t slot = h * 4 + quad / 4;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint32_t*>(box + (unit * 8 + j) * 128 + (slot ^ (unit & 7)) * 16 + quad % 4 * 4) =
                    low_bytes(q[0][j], q[1][j], q[2][j], q[3][j]);
        }
        if (r0 + 128 < end) load(r0 + 128);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t c = i * 32 + tid / 8, slot = tid % 8;
            const u4 w = *reinterpret_cast<const u4*>(box + c * 128 + (slot ^ (c >> 3 & 7)) * 16);
            if (c0 + c < p.cols)
                *reinterpret_cast<u4*>(p.codes + (uint64_t)(c0 + c) * p.code_row + r0 + slot * 16) = w;
        }
        __syncthreads();
    }
}

// Chunks of rows for the maxima: about 1024 blocks of 256 columns, and at most
// 32 of them, which the second kernel reads for each of its blocks.
struct Chunks {
    uint64_t count, rows, padded;
};
Chunks chunks_of(uint64_t rows, uint64_t cols) {
    const uint64_t across = (cols + 255) / 256;
    uint64_t k = std::min<uint64_t>({32, std::max<uint64_t>(1, 1024 / across), std::max<uint64_t>(1, rows / 32)});
    const uint64_t each = std::max<uint64_t>(1, (rows + k - 1) / k);
    return {std::max<uint64_t>(1, (rows + each - 1) / each), each, across * 256};
}

bool valid_q8(uint64_t rows, uint64_t cols) { return valid_shape(rows, cols) && cols <= kMaxCols; }

}  // namespace

extern "C" {

uint64_t tlc_q8_code_stride(uint64_t cols) { return cols < 1 || cols > kMaxCols ? 0 : q8_stride(cols); }

int tlc_q8_pack_rows(const void* x, uint64_t x_stride, int dtype, uint64_t rows, uint64_t cols, int8_t* codes,
                     float* scales, tlc_stream_t stream) {
    if (!valid_dtype(dtype) || !valid_q8(rows, cols)) return TLC_ERR_INVALID_ARG;
    if (rows == 0) return TLC_OK;
    if (!valid_matrix(x, dtype, cols, x_stride) || !codes || !aligned(codes, 16) || !scales || !aligned(scales, 4))
        return TLC_ERR_INVALID_ARG;
    RowArgs p;
    p.x = x, p.x_stride = x_stride, p.rows = rows, p.cols = (uint32_t)cols, p.code_row = (uint32_t)q8_stride(cols);
    p.codes = codes, p.scales = scales;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        auto go = [&](auto waves, auto units) {
            constexpr int W = decltype(waves)::value, U = decltype(units)::value;
            return launch_blocks("tlc_q8_pack_rows", st, (rows + 4 / W - 1) / (4 / W), kThreads,
                                 [&](uint64_t first, uint32_t blocks) {
                                     p.first = first;
                                     k_pack_rows<T, W, U><<<blocks, kThreads, 0, st>>>(p);
                                 });
        };
        if (p.code_row <= 512) return go(Int<1>{}, Int<1>{});
        if (p.code_row <= 2048) return go(Int<1>{}, Int<4>{});
        if (p.code_row <= 8192) return go(Int<4>{}, Int<4>{});
        return go(Int<4>{}, Int<8>{});
    });
}

size_t tlc_q8_pack_columns_workspace_size(uint64_t rows, uint64_t cols) {
    if (!valid_q8(cols, rows) || cols < 1) return 0;
    const Chunks k = chunks_of(rows, cols);
    return k.count * k.padded * 4;
}

int tlc_q8_pack_columns(const void* x, uint64_t x_stride, int dtype, uint64_t rows, uint64_t cols, int8_t* codes,
                        float* scales, void* workspace, size_t workspace_bytes, tlc_stream_t stream) {
    if (!valid_dtype(dtype) || !valid_q8(cols, rows) || cols < 1) return TLC_ERR_INVALID_ARG;
    if (!valid_matrix(x, dtype, cols, x_stride) || !codes || !aligned(codes, 16) || !scales || !aligned(scales, 4))
        return TLC_ERR_INVALID_ARG;
    const Chunks k = chunks_of(rows, cols);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < k.count * k.padded * 4) return TLC_ERR_WORKSPACE;
    ColumnArgs p;
    p.x = x, p.x_stride = x_stride, p.rows = (uint32_t)rows, p.cols = (uint32_t)cols;
    p.code_row = (uint32_t)q8_stride(rows);
    p.codes = codes, p.scales = scales;
    p.maxima = static_cast<uint32_t*>(workspace);
    p.chunks = (uint32_t)k.count, p.chunk_rows = (uint32_t)k.rows, p.padded = (uint32_t)k.padded;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        p.blocks_c = (uint32_t)(k.padded / 256);
        const int rc = launch_blocks("tlc_q8_column_max", st, k.count * p.blocks_c, kThreads,
                                     [&](uint64_t first, uint32_t blocks) {
                                         p.first = first;
                                         k_column_max<T><<<blocks, kThreads, 0, st>>>(p);
                                     });
        if (rc) return rc;
        p.blocks_c = (uint32_t)((cols + 127) / 128);
        // several row tiles a block, which reads the maxima once for them, where there are blocks enough
        const uint64_t tiles = p.code_row / 128;
        p.row_tiles = (uint32_t)std::min<uint64_t>(4, std::max<uint64_t>(1, tiles * p.blocks_c / 1024));
        return launch_blocks("tlc_q8_pack_columns", st, (tiles + p.row_tiles - 1) / p.row_tiles * p.blocks_c, kThreads,
                             [&](uint64_t first, uint32_t blocks) {
                                 p.first = first;
                                 k_pack_columns<T><<<blocks, kThreads, 0, st>>>(p);
                             });
    });
}

}  // extern "C"
