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

constexpr int kThreads = 256;  // four wavefronts, two by two
constexpr int kStep = 32;      // rows of dy and x a block takes at a time

typedef short s4v __attribute__((ext_vector_type(4)));
typedef __bf16 b8v __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));

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
    uint32_t tiles, tiles_i, tiles_c;  // tiles of dw, its rows of them, and those of one row
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

// Sixteen codes of one group as bfloat16 numbers.
template <int FMT>
__device__ __forceinline__ void decode16(u4 codes, uint32_t byte, u4* w) {
    if constexpr (FMT == TLC_CKPT8_E4M3) {
        const float s = scale_of(byte);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j / 2][j % 2 * 2] =
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[j], s, false));
            w[j / 2][j % 2 * 2 + 1] =
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[j], s, true));
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
            decode8<FMT>(u2{codes[2 * h], codes[2 * h + 1]}, byte, v);
#pragma unroll
            for (int j = 0; j < 4; ++j)  // exact: the low halves are 0
                w[h][j] = __builtin_amdgcn_perm(to_bits(v[2 * j + 1]), to_bits(v[2 * j]), 0x07060302u);
        }
    }
}

template <typename W>
__device__ __forceinline__ float column_scale(const void* p, uint32_t c) {
    if (!p) return 1.0f;
    return (float)static_cast<const typename W::Elem*>(p)[c];
}

// The product.  A block computes kTile x kTile values of dw, each wavefront a
// quarter, as 32x32x16 products.  Both operands lie with the reduction (the
// rows t) as the slow index, in memory and, unchanged, in LDS: [t][column].
// The transposing LDS read turns them: 16 lanes read 4 rows of 16 columns and
// each gets 4 rows of one column.  Which 8 of the 16 rows a lane holds is the
// same for both operands, so their order does not matter.
//
// LDS: 32-byte segments (16 columns) of row t lie at segment ^ (t & 3), so that
// the 4 rows of one transposing read fall into different banks (measured: 105
// bytes a clock and CU instead of 32).
//
// Two stages.  While one is multiplied, the rows loaded before go to the other
// and the next ones are on their way in registers.  The block meets once a
// step, before the last products, whose operands it has then read; these run
// while the next stage's first operands are read.
template <int kTerms, int kTile>
struct __align__(16) Stage {
    uint16_t a[kTerms][kStep][kTile];
    uint16_t b[kStep][kTile];
};

__device__ __forceinline__ s4v read_tr(const uint16_t* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4v*)p);
}
// Operand of a 32x32x16 product: `p` is the lane's place in rows k .. k+7 of
// its half, with a read of rows +0..3 and one of rows +4..7.
template <int kTile>
__device__ __forceinline__ b8v operand(const uint16_t* p) {
    const s4v lo = read_tr(p), hi = read_tr(p + 4 * kTile);
    return __builtin_bit_cast(b8v, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The order of instructions in a region of kGroups times 16 products: a
// product keeps the matrix core busy for 32 clocks, in which the wavefront can
// issue about seven others.
template <int kGroups>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int i = 0; i < kGroups * 16; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);  // vector arithmetic
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // LDS write
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // global load
    }
}

template <typename T, typename W, int FMT, int kTile>
__global__ __launch_bounds__(kThreads, 1) void k_weight_grad(MatArgs p) {
    using Elem = typename T::Elem;
    constexpr int kTerms = T::kTerms;
    constexpr int kWave = kTile / 2, kTiles = kWave / 32;
    constexpr int kUnits = kTile / 8;                          // 16-byte units of a row of dy in bfloat16
    constexpr int kLoadsA = kStep * kUnits / kThreads;         // of them a lane
    constexpr int kLoadsB = kStep * kTile / 16 / kThreads;     // 16-byte units of codes a lane
    static_assert(kLoadsA >= 1 && kLoadsB >= 1, "too narrow a tile");
    __shared__ Stage<kTerms, kTile> stage0, stage1;

    // neighbouring tiles on one XCD (blocks go round the 8 of them), in bands of 4 rows of tiles
    uint32_t b = blockIdx.x;
    const uint32_t total = gridDim.x, per = total / 8;
    if (b < per * 8) b = b % 8 * per + b / 8;
    const uint32_t slice = b / p.tiles, tile = b % p.tiles;
    const uint32_t band = tile / (4 * p.tiles_c), in_band = tile % (4 * p.tiles_c);
    const uint32_t band_rows = min(4u, p.tiles_i - band * 4);
    const uint32_t i0 = (band * 4 + in_band % band_rows) * kTile, c0 = in_band / band_rows * kTile;
    const uint64_t t_begin = slice * p.slice_rows, t_end = min(p.rows, t_begin + p.slice_rows);
    const int steps = (int)((t_end - t_begin + kStep - 1) / kStep);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;

    // what the lane loads: rows ra + i*(rows between), columns from i0 + 8*ua; codes likewise
    const int ra = threadIdx.x / kUnits, ua = threadIdx.x % kUnits;
    const int rb = threadIdx.x / (kTile / 16), ub = threadIdx.x % (kTile / 16);
    constexpr int kRowsA = kThreads / kUnits, kRowsB = kThreads / (kTile / 16);
    // A lane past the last column loads the row's first ones, and a unit that
    // ends past it runs on into the next row: those columns of the operands
    // only reach values of dw that are not stored.  Only the last row may not
    // be read past its end, and rows past t_end have to be zeros.
    const int count = min(max((int)(p.n - i0) - ua * 8, 0), 8);
    const Elem* const pa =
        static_cast<const Elem*>(p.dy) + (t_begin + ra) * p.dy_stride + (count ? i0 + ua * 8 : 0);
    const uint32_t cb = c0 + ub * 16 < p.code_row ? c0 + ub * 16 : 0;
    const uint8_t* const pb = p.codes + (t_begin + rb) * p.code_row + cb;
    const uint8_t* const ps = p.scales + (t_begin + rb) * p.scale_row + cb / 32;
    const uint64_t here = t_end - t_begin;
    // steps all of whose rows are here and not the matrix's last one
    const int whole = p.dy_stride >= 8 ? (int)((t_end == p.rows ? here - 1 : here) / kStep) : 0;

    // In registers: what was loaded for the two steps after the next (an even
    // and an odd one), and the next step's codes as bfloat16 numbers.
    struct Loaded {
        Raw8<T> a[kLoadsA];
        u4 codes[kLoadsB];
        uint32_t byte[kLoadsB];
    } g0, g1;
    u4 gx[kLoadsB][2];
    auto load_whole = [&](Loaded& g, int s) {
        const uint64_t t = (uint64_t)s * kStep;
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i) g.a[i] = load8<T>(pa + (t + i * kRowsA) * p.dy_stride, 8);
#pragma unroll
        for (int i = 0; i < kLoadsB; ++i) {
            g.codes[i] = *reinterpret_cast<const u4*>(pb + (t + i * kRowsB) * p.code_row);
            g.byte[i] = ps[(t + i * kRowsB) * p.scale_row];
        }
    };
    auto load = [&](Loaded& g, int s) {
        if (s < whole) return load_whole(g, s);
        const uint64_t t = (uint64_t)s * kStep;
        const uint64_t left = here - t;  // rows from this step on
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i) {
            const int r = i * kRowsA;
            g.a[i] = load8<T>(pa + (t + r) * p.dy_stride, (uint64_t)(ra + r) < left ? count : 0);
        }
#pragma unroll
        for (int i = 0; i < kLoadsB; ++i) {
            const int r = i * kRowsB;
            g.codes[i] = u4{0, 0, 0, 0};
            g.byte[i] = 0;
            if ((uint64_t)(rb + r) < left) {
                g.codes[i] = *reinterpret_cast<const u4*>(pb + (t + r) * p.code_row);
                g.byte[i] = ps[(t + r) * p.scale_row];
            }
        }
    };
    auto decode = [&](const Loaded& g) {
#pragma unroll
        for (int i = 0; i < kLoadsB; ++i) decode16<FMT>(g.codes[i], g.byte[i], gx[i]);
    };
    auto store = [&](Stage<kTerms, kTile>& st, const Loaded& g) {
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i) {
            const int r = ra + i * kRowsA, at = ((ua >> 1) ^ (r & 3)) * 16 + (ua & 1) * 8;
            if constexpr (kTerms == 1) {
                *reinterpret_cast<u4*>(&st.a[0][r][at]) = g.a[i].w[0];
            } else {
                float v[8];
                unpack8<T>(g.a[i], v);
                u4 w[kTerms];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint16_t lo[kTerms], hi[kTerms];
                    split<kTerms>(v[2 * j], lo);
                    split<kTerms>(v[2 * j + 1], hi);
#pragma unroll
                    for (int k = 0; k < kTerms; ++k) w[k][j] = (uint32_t)lo[k] | (uint32_t)hi[k] << 16;
                }
#pragma unroll
                for (int k = 0; k < kTerms; ++k) *reinterpret_cast<u4*>(&st.a[k][r][at]) = w[k];
            }
        }
#pragma unroll
        for (int i = 0; i < kLoadsB; ++i) {
            const int r = rb + i * kRowsB, at = (ub ^ (r & 3)) * 16;
            *reinterpret_cast<u4*>(&st.b[r][at]) = gx[i][0];
            *reinterpret_cast<u4*>(&st.b[r][at + 8]) = gx[i][1];
        }
    };

    // the lane's place in an operand: rows lane/32*8 + (lane%16)/4, segment + lane/16%2, 4 columns of lane%4
    const int sub = (lane >> 2) & 3, seg = (lane >> 4) & 1;
    const int wi = (wave >> 1) * kWave, wc = (wave & 1) * kWave;
    const int row = (lane >> 5) * 8 + sub;
    int place[2];  // of an even and an odd 32-column tile: the segments' low bits differ
#pragma unroll
    for (int q = 0; q < 2; ++q) place[q] = row * kTile + (((2 * q + seg) ^ sub) * 16) + (lane & 3) * 4;

    f16v acc[kTiles][kTiles] = {};
    auto operands_b = [&](const Stage<kTerms, kTile>& st, int k, b8v* f) {
#pragma unroll
        for (int c = 0; c < kTiles; ++c)
            f[c] = operand<kTile>(&st.b[0][0] + k * 16 * kTile + place[c & 1] + wc + (c & ~1) * 32);
    };
    auto operands_a = [&](const Stage<kTerms, kTile>& st, int k, int term, b8v* f) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
            f[i] = operand<kTile>(&st.a[term][0][0] + k * 16 * kTile + place[i & 1] + wi + (i & ~1) * 32);
    };
    auto multiply = [&](const b8v* fa, const b8v* fb) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
                acc[i][c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[c], acc[i][c], 0, 0, 0);
    };

    b8v fa[2][kTiles], fb[2][kTiles];
    // Step s: multiplies `now`, stores step s+1 to `next`, loads step s+3 into
    // the registers that frees, and decodes the codes of step s+2.  kMain: all
    // of it without a branch, so that one schedule spans the products and
    // everything else.
    auto step = [&](Stage<kTerms, kTile>& now, Stage<kTerms, kTile>& next, Loaded& here_g, Loaded& next_g, int s,
                    auto main) {
        constexpr bool kMain = decltype(main)::value;
        operands_b(now, 1, fb[1]);
#pragma unroll
        for (int k = 0; k < kTerms; ++k) {
            operands_a(now, k + 1 < kTerms ? 0 : 1, (k + 1) % kTerms, fa[(k + 1) & 1]);
            multiply(fa[k & 1], fb[0]);
        }
        if (kMain || s + 1 < steps) store(next, next_g);
        if constexpr (kMain)
            load_whole(next_g, s + 3);
        else if (s + 3 < steps)
            load(next_g, s + 3);
#pragma unroll
        for (int k = 0; k + 1 < kTerms; ++k) {
            operands_a(now, 1, k + 1, fa[(kTerms + k + 1) & 1]);
            multiply(fa[(kTerms + k) & 1], fb[1]);
        }
        if constexpr (kMain && kTiles == 4) interleave<kTerms * 2 - 1>();
        __syncthreads();
        b8v last[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) last[i] = fa[(2 * kTerms - 1) & 1][i];
        if (kMain || s + 1 < steps) {
            operands_a(next, 0, 0, fa[0]);
            operands_b(next, 0, fb[0]);
        }
        multiply(last, fb[1]);
        if (kMain || s + 2 < steps) decode(here_g);
        if constexpr (kMain && kTiles == 4) interleave<1>();
    };
    if (steps > 0) {
        load(g0, 0);
        decode(g0);
        store(stage0, g0);
        if (steps > 1) {
            load(g1, 1);
            decode(g1);
        }
        if (steps > 2) load(g0, 2);
        __syncthreads();
        operands_a(stage0, 0, 0, fa[0]);
        operands_b(stage0, 0, fb[0]);
        int s = 0;
        for (; s + 4 < whole; s += 2) {
            step(stage0, stage1, g0, g1, s, Int<1>{});
            step(stage1, stage0, g1, g0, s + 1, Int<1>{});
        }
#pragma unroll 1
        for (; s < steps; s += 2) {
            step(stage0, stage1, g0, g1, s, Int<0>{});
            if (s + 1 < steps) step(stage1, stage0, g1, g0, s + 1, Int<0>{});
        }
    }

    // register j of a lane: row 8*(j/4) + 4*(lane/32) + j%4, column lane%32
    const uint32_t row0 = i0 + wi + (lane >> 5) * 4, col0 = c0 + wc + (lane & 31);
    const bool direct = p.partial == nullptr;
    float* const out = direct ? p.dw : p.partial + (uint64_t)slice * p.n * p.cols;
    const uint64_t stride = direct ? p.dw_stride : p.cols;
    float cs[kTiles];
#pragma unroll
    for (int c = 0; c < kTiles; ++c)
        cs[c] = column_scale<W>(direct ? p.col_scale : nullptr, min(col0 + c * 32, p.cols - 1));
    const bool add = direct && p.accumulate;
    auto write = [&](auto edge) {
        constexpr bool kEdge = decltype(edge)::value;
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const uint32_t r = row0 + i * 32 + (j >> 2) * 8 + (j & 3);
                float* const o = out + r * stride + col0;
                if (!kEdge || r < p.n) {
#pragma unroll
                    for (int c = 0; c < kTiles; ++c)
                        if (!kEdge || col0 + c * 32 < p.cols) {
                            const float v = acc[i][c][j] * cs[c];
                            o[c * 32] = kEdge && add ? o[c * 32] + v : v;
                        }
                }
            }
    };
    if (i0 + kTile <= p.n && c0 + kTile <= p.cols && !add)
        write(Int<0>{});
    else
        write(Int<1>{});
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
struct Shape {
    uint32_t tile, slices;
    uint64_t slice_rows, tiles_i, tiles_c;
};
Shape shape_of(uint64_t rows, uint64_t n, uint64_t cols) {
    Shape s;
    s.tile = 256;
    s.tiles_i = (n + s.tile - 1) / s.tile, s.tiles_c = (cols + s.tile - 1) / s.tile;
    const uint64_t tiles = s.tiles_i * s.tiles_c;
    const uint64_t want = std::min<uint64_t>((256 + tiles - 1) / tiles, std::max<uint64_t>(rows / 256, 1));
    s.slice_rows = ((rows + want - 1) / want + kStep - 1) / kStep * kStep;
    s.slices = s.slice_rows ? (uint32_t)((rows + s.slice_rows - 1) / s.slice_rows) : 0;
    return s;
}

}  // namespace

extern "C" {

size_t tlc_ckpt8_weight_grad_workspace_size(uint64_t rows, uint64_t n, uint64_t cols) {
    if (!valid_shape(rows, cols) || n < 1 || n > kMaxDim) return 0;
    const Shape s = shape_of(rows, n, cols);
    const uint64_t bytes = s.slices > 1 ? s.slices * n * cols * sizeof(float) : 0;
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
    const Shape s = shape_of(rows, n, cols);
    if (s.tiles_i * s.tiles_c > (1u << 22)) return TLC_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < tlc_ckpt8_weight_grad_workspace_size(rows, n, cols))
        return TLC_ERR_WORKSPACE;
    if (rows == 0 && accumulate) return TLC_OK;
    MatArgs p;
    p.dy = dy, p.dy_stride = dy_stride, p.codes = codes, p.scales = scales, p.rows = rows;
    p.n = (uint32_t)n, p.cols = (uint32_t)cols;
    p.code_row = (uint32_t)code_stride(cols), p.scale_row = (uint32_t)scale_stride(cols);
    p.col_scale = col_scale;
    p.dw = dw, p.dw_stride = dw_stride, p.accumulate = accumulate != 0;
    p.partial = s.slices > 1 ? static_cast<float*>(workspace) : nullptr;
    p.slice_rows = s.slice_rows;
    p.tiles = (uint32_t)(s.tiles_i * s.tiles_c);
    p.tiles_i = (uint32_t)s.tiles_i, p.tiles_c = (uint32_t)s.tiles_c;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (s.slices) {
        const uint32_t grid = p.tiles * s.slices;
        const int rc = with_dtype(dtype, [&](auto t) {
            return with_weight(t, col_scale, col_scale_dtype, [&](auto w) {
                return with_format(format, [&](auto f) {
                    return launch("tlc_ckpt8_weight_grad", st, [&] {
                        k_weight_grad<decltype(t), decltype(w), decltype(f)::value, 256><<<grid, kThreads, 0, st>>>(p);
                    });
                });
            });
        });
        if (rc || s.slices == 1) return rc;
    }
    const uint32_t blocks = (uint32_t)std::min<uint64_t>(n * ((cols + kThreads - 1) / kThreads), 1u << 20);
    return with_dtype(dtype, [&](auto t) {
        return with_weight(t, col_scale, col_scale_dtype, [&](auto w) {
            return launch("tlc_ckpt8_weight_sum", st, [&] {
                k_weight_sum<decltype(w)><<<blocks, kThreads, 0, st>>>(p, s.slices);
            });
        });
    });
}

}  // extern "C"
