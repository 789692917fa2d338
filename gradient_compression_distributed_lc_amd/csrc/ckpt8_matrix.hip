// ckpt8_matrix.hip -- the weight gradient from an 8-bit checkpoint:
//   dw[i][c] (+)= col_scale[c] * sum over rows t of dy[t][i] * x[t][c],
// over all rows or, for a weight of each expert, over the expert's own;
// x the checkpoint's values.  x is a bfloat16 number as it stands, dy is one
// (bf16), the sum of two (fp16) or of three (fp32) of them, so every product is
// exact and the sums are the matrix cores' fp32.

#include <algorithm>
#include <cmath>

#include "ckpt8.h"
#include "experts.h"
#include "launch.h"

namespace {

using namespace tlc_ckpt8;
using tlc_experts::Experts;
using tlc_experts::Span;
using tlc_internal::launch_blocks;

constexpr int kThreads = 256;  // of a group: four wavefronts, two by two

typedef short s4v __attribute__((ext_vector_type(4)));
typedef __bf16 b8v __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef f4 f4_at4 __attribute__((aligned(4)));

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
    f4* partial;         // with several: [slices][tiles], each tile as its lanes hold it; else nullptr
    uint64_t slice_rows; // rows of one slice, a multiple of 64
    uint32_t tiles, tiles_i, tiles_c;  // tiles of dw, its rows of them, and those of one row
    uint32_t first;      // block of the whole that the launch begins with
    // a weight for each expert
    Experts experts;
    uint64_t dw_expert;  // values between the experts' dw
    uint32_t slices, tiles_all;  // slices of each expert's rows; tiles of all experts
};

// Place in the matrix of tile number `tile`: neighbours in bands of 4 rows of tiles.
__device__ __forceinline__ void tile_place(const MatArgs& p, uint32_t tile, uint32_t* i, uint32_t* c) {
    const uint32_t band = tile / (4 * p.tiles_c), in_band = tile % (4 * p.tiles_c);
    const uint32_t band_rows = min(4u, p.tiles_i - band * 4);
    *i = band * 4 + in_band % band_rows;
    *c = in_band / band_rows;
}

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

// The product.  A block computes kTile x kTile values of dw, each wavefront of a
// group a quarter, as 32x32x16 products.  With two groups each takes half of
// the rows in stages of its own, and their sums are added at the end: two
// wavefronts a SIMD cover each other's waits, which the small tile needs (its
// wavefronts have half the products per operand read; 4096x4096x1024 54 -> 43
// us).  The large tile's sums leave registers for one only.  Both operands lie with the reduction (the
// rows t) as the slow index, in memory and, unchanged, in LDS: [t][column].
// The transposing LDS read turns them: 16 lanes read 4 rows of 16 columns and
// each gets 4 rows of one column.  Which 8 of the 16 rows a lane holds is the
// same for both operands, so their order does not matter.
//
// LDS: the 16-byte slots (8 columns) of row t lie at slot ^ swizzle(t).  The 4
// rows x 32 columns that half a wavefront reads at once then fall into the 64
// banks once each, and so do the slots that 8 lanes write at once (8 lanes
// hold 4 units of codes of two rows).  Without it both take two to four times
// as long (counted: 2 clocks a read and 8 a 16-byte write, no conflicts).
//
// Two stages.  While one is multiplied, the rows loaded before go to the other
// and the next ones are on their way in registers.  The block meets once a
// step, before the last products, whose operands it has then read; these run
// while the next stage's first operands are read.
//
// Both groups of a block take the same number of steps and so meet equally
// often, but where the rows end one can be in the branch-free loop and the
// other in the one with checks: they then wait at two barriers of the code.
// That is sound here because the barrier counts a workgroup's wavefronts
// whichever instruction they arrive by, a wavefront takes either loop as a
// whole (group is uniform in it), and no group reads the other's stages before
// the exchange of sums, which all reach together.
template <int kTerms, int kTile, int kStep>
struct __align__(16) Stage {
    uint16_t a[kTerms][kStep][kTile];
    uint16_t b[kStep][kTile];
};

__device__ __forceinline__ int swizzle(int t) { return (t & 3) << 2 | (t & 1); }

__device__ __forceinline__ s4v read_tr(const uint16_t* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4v*)p);
}
// Orders a wavefront's own LDS accesses across its lanes.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
// Operand of a 32x32x16 product: `p` is the lane's place in rows k .. k+7 of
// its half, with a read of rows +0..3 and one of rows +4..7.
template <int kTile>
__device__ __forceinline__ b8v operand(const uint16_t* p) {
    const s4v lo = read_tr(p), hi = read_tr(p + 4 * kTile);
    return __builtin_bit_cast(b8v, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The order of instructions in a region of kProducts products: a
// product keeps the matrix core busy for 32 clocks, in which the wavefront can
// issue about seven others.
template <int kProducts>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int i = 0; i < kProducts; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);  // vector arithmetic
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // LDS write
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // global load
    }
}

template <typename T, typename W, int FMT, int kTile, int kStep, int kGroups, bool kExperts>
__global__ __launch_bounds__(kThreads * kGroups, 1) void k_weight_grad(MatArgs p) {
    using Elem = typename T::Elem;
    constexpr int kTerms = T::kTerms;
    constexpr int kWave = kTile / 2, kTiles = kWave / 32;
    constexpr int kUnits = kTile / 8;                          // 16-byte units of a row of dy in bfloat16
    constexpr int kLoadsA = kStep * kUnits / kThreads;         // of them a lane
    constexpr int kLoadsB = kStep * kTile / 16 / kThreads;     // 16-byte units of codes a lane
    static_assert(kLoadsA >= 1 && kLoadsB >= 1, "too narrow a tile");
    using Buffer = Stage<kTerms, kTile, kStep>;
    __shared__ Buffer stages0[kGroups], stages1[kGroups];
    const int tid = threadIdx.x % kThreads;
    const int group = kGroups == 1 ? 0 : __builtin_amdgcn_readfirstlane((int)threadIdx.x / kThreads);
    Buffer &stage0 = stages0[group], &stage1 = stages1[group];

    // neighbouring tiles on one XCD: blocks go round the 8 of them. Experts' tiles
    // differ in time: in runs of neighbours an XCD gets the longest expert whole and
    // works on alone, so each gets an eighth of every expert, and the longest expert
    // is begun first. Runs, eighths, eighths with the longest first, us:
    //   8 uneven experts of 5120x1280, 16384 bf16 rows   401  281  226 (dense 218)
    //   16 of 1280x1280                                  111   90   69
    //   32 of 1024x2048                                  176  147  132-140
    //   64 of 1024x1024, 8192 rows                        98   87   89
    //   8 of 4096x4096, 16384 rows: a round each         556  556  560
    //   5 of 1000x515, 777 fp32 rows: one round           20   21   21
    uint32_t b = blockIdx.x;
    if constexpr (kExperts) {
        b = tlc_experts::xcd_share(b + p.first, p.tiles);
    } else {
        const uint32_t total = gridDim.x, per = total / 8;
        if (b < per * 8) b = b % 8 * per + b / 8;
        b += p.first;
    }
    const uint32_t slice = b / (kExperts ? p.tiles_all : p.tiles), tile = b % p.tiles;
    uint32_t tile_i, tile_c;
    tile_place(p, tile, &tile_i, &tile_c);
    const uint32_t i0 = tile_i * kTile, c0 = tile_c * kTile;
    float* dw = p.dw;
    // the group's share of the slice's rows, the same steps for each group
    uint64_t s_begin, s_end;
    if constexpr (kExperts) {
        const Span mine = tlc_experts::rows_by_length(p.experts, b % p.tiles_all / p.tiles);
        dw += mine.expert * p.dw_expert;
        b = slice * p.tiles_all + mine.expert * p.tiles + tile;
        const uint64_t cut = ((mine.end - mine.begin + p.slices - 1) / p.slices + 63) / 64 * 64;
        s_begin = min(mine.begin + slice * cut, (uint64_t)mine.end), s_end = min(s_begin + cut, (uint64_t)mine.end);
    } else {
        s_begin = slice * p.slice_rows, s_end = min(p.rows, s_begin + p.slice_rows);
    }
    const uint64_t share = ((s_end - s_begin + kGroups - 1) / kGroups + kStep - 1) / kStep * kStep;
    const uint64_t t_begin = min(s_begin + group * share, s_end), t_end = min(t_begin + share, s_end);
    const int steps = (int)(share / kStep);
    const int wave = tid >> 6, lane = tid & 63;

    // what the lane loads: rows ra + i*(rows between), columns from i0 + 8*ua; codes likewise
    const int ra = tid / kUnits, ua = tid % kUnits;
    // (codes: 4 neighbouring units of two rows in 8 lanes)
    const int pair = tid / (kTile / 8), in_pair = tid % (kTile / 8);
    const int rb = 2 * pair + (in_pair >> 2 & 1), ub = (in_pair & 3) | in_pair >> 3 << 2;
    constexpr int kRowsA = kThreads / kUnits, kRowsB = kThreads / (kTile / 16);
    // A lane past the last column loads the row's first ones, and a unit that
    // ends past it runs on into the next row: those columns of the operands
    // only reach values of dw that are not stored.  Only at the matrix's end
    // may a unit not run on, and rows past t_end have to be zeros.
    const int count = min(max((int)(p.n - i0) - ua * 8, 0), 8);
    const Elem* const pa =
        static_cast<const Elem*>(p.dy) + (t_begin + ra) * p.dy_stride + (count ? i0 + ua * 8 : 0);
    const uint32_t cb = c0 + ub * 16 < p.code_row ? c0 + ub * 16 : 0;
    const uint8_t* const pb = p.codes + (t_begin + rb) * p.code_row + cb;
    const uint8_t* const ps = p.scales + (t_begin + rb) * p.scale_row + cb / 32;
    const int here = (int)(t_end - t_begin);
    // rows from whose every unit eight columns can be read: all but the last ceil(8 / stride)
    const int tail = p.dy_stride >= 8 ? 1 : (int)((7 + p.dy_stride) / p.dy_stride);
    const int safe = t_end + tail > p.rows ? max(here - (int)(t_end + tail - p.rows), 0) : here;
    const int whole = safe / kStep;  // steps of such rows only

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
        const int t = s * kStep;
        int alone = -1;  // a row of this lane that has to be read one by one
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i) {
            const int r = t + ra + i * kRowsA;
            const bool run_on = r < safe || (r < here && count == 8);
            g.a[i] = load8<T>(pa + (uint64_t)(t + i * kRowsA) * p.dy_stride, run_on ? 8 : 0, true);
            if (!run_on && r < here) alone = i;
        }
        static_assert(kRowsA >= 8, "a lane has at most one of the last eight rows");
        if (alone >= 0) {
            const Raw8<T> v = load8<T>(pa + (uint64_t)(t + alone * kRowsA) * p.dy_stride, min(count, 7));
#pragma unroll
            for (int i = 0; i < kLoadsA; ++i)
                if (i == alone) g.a[i] = v;
        }
#pragma unroll
        for (int i = 0; i < kLoadsB; ++i) {
            const uint64_t r = t + i * kRowsB;
            g.codes[i] = u4{0, 0, 0, 0};
            g.byte[i] = 0;
            if ((int)r + rb < here) {
                g.codes[i] = *reinterpret_cast<const u4*>(pb + r * p.code_row);
                g.byte[i] = ps[r * p.scale_row];
            }
        }
    };
    auto decode = [&](const Loaded& g) {
#pragma unroll
        for (int i = 0; i < kLoadsB; ++i) decode16<FMT>(g.codes[i], g.byte[i], gx[i]);
    };
    auto store = [&](Buffer& st, const Loaded& g) {
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i) {
            const int r = ra + i * kRowsA, at = (ua ^ swizzle(r)) * 8;
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
            const int r = rb + i * kRowsB, at = (2 * ub ^ swizzle(r)) * 8;
            *reinterpret_cast<u4*>(&st.b[r][at]) = gx[i][0];
            *reinterpret_cast<u4*>(&st.b[r][at ^ 8]) = gx[i][1];
        }
    };

    // the lane's place in an operand of each 32 columns: row lane/32*8 + (lane%16)/4,
    // columns lane/16%2*16 + lane%4*4, four of them
    const int wi = (wave >> 1) * kWave, wc = (wave & 1) * kWave;
    const int row = (lane >> 5) * 8 + (lane >> 2 & 3);
    int place_a[kTiles], place_b[kTiles];
#pragma unroll
    for (int q = 0; q < kTiles; ++q) {
        const int slot = q * 4 + (lane >> 4 & 1) * 2 + (lane >> 1 & 1);
        place_a[q] = row * kTile + ((wi / 8 + slot) ^ swizzle(row)) * 8 + (lane & 1) * 4;
        place_b[q] = row * kTile + ((wc / 8 + slot) ^ swizzle(row)) * 8 + (lane & 1) * 4;
    }

    f16v acc[kTiles][kTiles] = {};
    auto operands_b = [&](const Buffer& st, int k, b8v* f) {
#pragma unroll
        for (int c = 0; c < kTiles; ++c)
            f[c] = operand<kTile>(&st.b[0][0] + k * 16 * kTile + place_b[c]);
    };
    auto operands_a = [&](const Buffer& st, int k, int term, b8v* f) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
            f[i] = operand<kTile>(&st.a[term][0][0] + k * 16 * kTile + place_a[i]);
    };
    auto multiply = [&](const b8v* fa, const b8v* fb) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
                acc[i][c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[c], acc[i][c], 0, 0, 0);
    };

    // A step is kSubs times 16 rows, each of kTerms products of the wavefront's
    // tile.  The operands of the next product are read while one runs; those of
    // the step's last product are in registers when the block meets.
    constexpr int kSubs = kStep / 16, kRounds = kSubs * kTerms;
    b8v fa[2][kTiles], fb[2][kTiles];
    auto round = [&](const Buffer& now, int q) {  // product q, and the reads for q + 1
        if (q % kTerms == 0 && q / kTerms + 1 < kSubs) operands_b(now, q / kTerms + 1, fb[(q / kTerms + 1) & 1]);
        operands_a(now, (q + 1) / kTerms, (q + 1) % kTerms, fa[(q + 1) & 1]);
        multiply(fa[q & 1], fb[q / kTerms & 1]);
    };
    // Step s: multiplies `now`, stores step s+1 to `next`, loads step s+3 into
    // the registers that frees, and decodes the codes of step s+2.  kMain: all
    // of it without a branch, so that one schedule spans the products and
    // everything else.
    auto step = [&](Buffer& now, Buffer& next, Loaded& here_g, Loaded& next_g, int s, auto main) {
        constexpr bool kMain = decltype(main)::value;
        if (kMain || s >= 0) round(now, 0);
        if (kMain || (s + 1 >= 0 && s + 1 < steps)) store(next, next_g);
        if constexpr (kMain)
            load_whole(next_g, s + 3);
        else if (s + 3 >= 0 && s + 3 < steps)
            load(next_g, s + 3);
        if (kMain || s >= 0) {
#pragma unroll
            for (int q = 1; q + 1 < kRounds; ++q) round(now, q);
        }
        if constexpr (kMain && kTerms == 1) interleave<kTiles * kTiles * (kRounds - 1)>();
        __syncthreads();
        b8v last_a[kTiles], last_b[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) last_a[i] = fa[(kRounds - 1) & 1][i], last_b[i] = fb[(kSubs - 1) & 1][i];
        if (kMain || (s + 1 >= 0 && s + 1 < steps)) {
            operands_a(next, 0, 0, fa[0]);
            operands_b(next, 0, fb[0]);
        }
        if (kMain || s >= 0) multiply(last_a, last_b);
        if (kMain || (s + 2 >= 0 && s + 2 < steps)) decode(here_g);
        if constexpr (kMain) interleave<kTiles * kTiles>();
    };
    // The steps before 0 fill the pipeline; they and the last ones are one loop.
    for (int s = -4; s < steps; s += 2) {
        if (s >= 0)
            for (; s + 4 < whole; s += 2) {
                step(stage0, stage1, g0, g1, s, Int<1>{});
                step(stage1, stage0, g1, g0, s + 1, Int<1>{});
            }
        step(stage0, stage1, g0, g1, s, Int<0>{});
        if (s + 1 < steps) step(stage1, stage0, g1, g0, s + 1, Int<0>{});
    }

    // register j of a lane: row 8*(j/4) + 4*(lane/32) + j%4, column lane%32.
    // One row of the wavefront's 32x32 parts to where it belongs:
    const uint32_t col0 = c0 + wc + (lane & 31);
    float cs[kTiles];
#pragma unroll
    for (int c = 0; c < kTiles; ++c) cs[c] = column_scale<W>(p.col_scale, min(col0 + c * 32, p.cols - 1));
    const bool direct = i0 + kTile <= p.n && c0 + kTile <= p.cols && !p.accumulate;
    auto write = [&](int i, const f16v* v) {
        if (p.partial) {  // four rows a store, each lane's registers side by side: the sum's business to sort out
            f4* const out = p.partial + (uint64_t)b * (kTile * kTile / 4) + wave * (kTile * kTile / 16) + lane;
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    out[((i * kTiles + c) * 4 + j) * 64] =
                        f4{v[c][4 * j], v[c][4 * j + 1], v[c][4 * j + 2], v[c][4 * j + 3]};
            return;
        }
        if (direct) {
            float* const o = dw + (i0 + wi + i * 32 + (lane >> 5) * 4) * p.dw_stride + col0;
#pragma unroll
            for (int j = 0; j < 16; ++j)
#pragma unroll
                for (int c = 0; c < kTiles; ++c) o[((j >> 2) * 8 + (j & 3)) * p.dw_stride + c * 32] = v[c][j] * cs[c];
            return;
        }
        // An edge, or dw is added to: 32 rows through LDS, so that a lane has 16
        // bytes of a row and eight reads of dw under way.  (8x8192x8192: 65 us
        // directly and 77 so; added to, 422 by a loop of single values and 129
        // so.)  Nothing reads the stages after the last meeting.  The registers
        // this takes beside the large tile's sums send 32 of those through
        // scratch, once a tile after the main loop: 16384x8192x8192 1.69 ms
        // against 1.67 with the loop of single values, 64x4096x4096 20 us
        // against 19.
        constexpr int kHere = kGroups == 1 ? 2 : 4;  // wavefronts in each array of stages
        static_assert(sizeof(stages0) >= kHere * 32 * kWave * sizeof(float), "their rows fit");
        const int w = group * 4 + wave;
        float* const mine = (w < kHere ? reinterpret_cast<float*>(stages0) : reinterpret_cast<float*>(stages1)) +
                            w % kHere * 32 * kWave;
        if constexpr (kGroups == 2) __syncthreads();  // the sums' exchange is read
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
                mine[((lane >> 5) * 4 + (j >> 2) * 8 + (j & 3)) * kWave + (lane & 31) + c * 32] = v[c][j] * cs[c];
        wave_sync();
        const uint32_t r0 = i0 + wi + i * 32, w0 = c0 + wc;
#pragma unroll 1
        for (int q = 0; q < kWave / 8; q += 8) {
            f4 old[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const uint32_t e = ((q + u) * 64 + lane) * 4, r = r0 + e / kWave, c = w0 + e % kWave;
                old[u] = f4{0.0f, 0.0f, 0.0f, 0.0f};
                if (p.accumulate && r < p.n && c + 4 <= p.cols)
                    old[u] = *reinterpret_cast<const f4_at4*>(dw + r * p.dw_stride + c);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const uint32_t e = ((q + u) * 64 + lane) * 4, r = r0 + e / kWave, c = w0 + e % kWave;
                const f4 s = *reinterpret_cast<const f4*>(mine + e);
                if (r < p.n && c + 4 <= p.cols)
                    *reinterpret_cast<f4_at4*>(dw + r * p.dw_stride + c) = p.accumulate ? old[u] + s : s;
            }
        }
        // the last one to three columns of the matrix, a row a lane
        const uint32_t last = p.cols & ~3u;
        if (lane < 32 && last >= w0 && last < w0 + kWave && r0 + lane < p.n)
            for (uint32_t c = last; c < p.cols; ++c) {
                float* const o = dw + (r0 + lane) * p.dw_stride + c;
                const float s = mine[lane * kWave + c - w0];
                *o = p.accumulate ? *o + s : s;
            }
        wave_sync();
    };
    if constexpr (kGroups == 1) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i) write(i, acc[i]);
    } else {
        // each group takes one row of parts: it gets the other group's sums of
        // that row and gives its own of the other; the first group's come first
        static_assert(kGroups == 2 && kTiles == 2, "a row of parts for each group");
        static_assert(sizeof(stages0) >= kThreads * kGroups * sizeof(f16v), "one part's sums fit");
        f4* const box = reinterpret_cast<f4*>(stages0);
        f16v keep[kTiles];
#pragma unroll
        for (int c = 0; c < kTiles; ++c) {
            const f16v give = group ? acc[0][c] : acc[1][c];
            keep[c] = group ? acc[1][c] : acc[0][c];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j)
                box[(group * 4 + j) * kThreads + tid] =
                    f4{give[4 * j], give[4 * j + 1], give[4 * j + 2], give[4 * j + 3]};
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f4 other = box[((group ^ 1) * 4 + j) * kThreads + tid];
#pragma unroll
                for (int e = 0; e < 4; ++e) keep[c][4 * j + e] += other[e];
            }
        }
        write(group, keep);
    }
}

// dw (+)= col_scale * the slices' sums, added in order; no slices: 0.
template <typename W>
__global__ __launch_bounds__(kThreads) void k_weight_sum(MatArgs p, uint32_t slices, uint32_t tile_size) {
    const uint32_t per = tile_size * tile_size / 4;  // f4 of a tile
    const uint32_t b = p.first + blockIdx.x;
    const uint32_t tile = b / (per / kThreads), v = b % (per / kThreads) * kThreads + threadIdx.x;
    const f4* const in = p.partial + (uint64_t)tile * per + v;
    const uint64_t next = (uint64_t)p.tiles_all * per;
    f4 s = {};
    uint32_t k = 0;
    for (; k + 4 <= slices; k += 4) {
        const f4 a = in[k * next], b = in[(k + 1) * next], c = in[(k + 2) * next], d = in[(k + 3) * next];
        s += a;
        s += b;
        s += c;
        s += d;
    }
    for (; k < slices; ++k) s += in[k * next];
    uint32_t ti, tc;
    tile_place(p, tile % p.tiles, &ti, &tc);
    float* const dw = p.dw + (uint64_t)(tile / p.tiles) * p.dw_expert;
    // the lane's place in the product: wavefront, 32x32 part, four rows of one column
    const uint32_t parts = tile_size / 64, lane = v % 64, part = v / 256 % (parts * parts), wave = v / (per / 4);
    const uint32_t row = ti * tile_size + (wave >> 1) * (tile_size / 2) + part / parts * 32 + v / 64 % 4 * 8 +
                         (lane >> 5) * 4;
    const uint32_t col = tc * tile_size + (wave & 1) * (tile_size / 2) + part % parts * 32 + (lane & 31);
    if (col >= p.cols) return;
    const float cs = column_scale<W>(p.col_scale, col);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (row + j < p.n) {
            float* const o = dw + (row + j) * p.dw_stride + col;
            *o = p.accumulate ? *o + s[j] * cs : s[j] * cs;
        }
}

// The tile and into how many slices the rows are cut, by the least of an
// estimate in microseconds.  Measured, one block a CU: 32 rows of a 256x256
// tile take 0.82 us (bf16; 0.92 for int8), 1.66 (fp16) and 2.6 (fp32), of a
// 128x128 tile 0.29 (0.32), 0.54 and 0.78: 0.8 and 0.32 a term of dy are within
// a quarter.  A tile's beginning and end take 14 and 5 us.  Slices fill the chip
// where the tiles do not (or leave a last round mostly empty) and cost writing
// and reading their sums.  Tiles of 256 and of 128, e4m3, us:
//                     bf16          fp16          fp32
//   16384x4096x4096   440  587      856  1075     1340  1577
//   1024x4096x4096    44   63       71   91       100   120
//   300x4096x4096     28   41       37   47       47    57
//   4096x4096x1024    59   44       84   75       113   103
//   2048x2048x2048    45   28       60   43       74    56
//   512x1024x4096     24   14       38   17       53    22
// The estimate takes the faster one in all of them but fp32 4096x4096x1024.
// 8192x1024x1024 in tiles of 128 takes 94 us in one slice and 32 in four.
struct Shape {
    uint32_t tile, slices;
    uint64_t slice_rows, tiles_i, tiles_c;
};
// For a weight of each expert: every expert's rows are cut into as many
// slices, and the estimate takes them as equally many.
Shape shape_of(uint64_t rows, uint64_t n, uint64_t cols, int terms, uint64_t experts = 1) {
    rows = (rows + experts - 1) / experts;
    Shape best = {};
    double least = 0.0;
    for (uint32_t tile = 128; tile <= 256; tile *= 2) {
        const uint64_t ti = (n + tile - 1) / tile, tc = (cols + tile - 1) / tile;
        for (uint64_t k : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
            if (k > 1 && rows / k < 128) break;
            const uint64_t cut = ((rows + k - 1) / k + 63) / 64 * 64, slices = cut ? (rows + cut - 1) / cut : 0;
            const double blocks = (double)ti * (double)tc * (double)slices * (double)experts;
            double us = std::ceil(blocks / 256) *
                        (tile == 256 ? 14.0 + 0.8 * terms * (double)(cut / 32) : 5.0 + 0.32 * terms * (double)(cut / 32));
            if (slices > 1) us += 4.0 + (2.0 * slices + 1.0) * (double)n * (double)cols * (double)experts * 4.0 / 5.5e6;
            if (!best.tile || us < least) best = {tile, (uint32_t)slices, cut, ti, tc}, least = us;
        }
    }
    return best;
}

uint64_t workspace_of(const Shape& s, uint64_t experts = 1) {
    return s.slices > 1 ? s.slices * experts * s.tiles_i * s.tiles_c * s.tile * s.tile * sizeof(float) : 256;
}

// The launches of either call, p filled but for what the shape decides.
template <bool kExperts>
int weight_grad(MatArgs p, const Shape& s, int dtype, int col_scale_dtype, int format, void* workspace,
                hipStream_t st) {
    p.partial = s.slices > 1 ? static_cast<f4*>(workspace) : nullptr;
    p.slice_rows = s.slice_rows, p.slices = s.slices;
    p.tiles = (uint32_t)(s.tiles_i * s.tiles_c);
    p.tiles_i = (uint32_t)s.tiles_i, p.tiles_c = (uint32_t)s.tiles_c;
    p.tiles_all = kExperts ? p.tiles * p.experts.count : p.tiles;
    const void* const col_scale = p.col_scale;
    if (s.slices) {
        const uint64_t all = (uint64_t)p.tiles_all * s.slices;
        const uint32_t threads = s.tile == 256 ? kThreads : 2 * kThreads;
        const char* const name = kExperts ? "tlc_expert_weight_grad" : "tlc_ckpt8_weight_grad";
        const int rc = with_dtype(dtype, [&](auto t) {
            return with_weight(t, col_scale, col_scale_dtype, [&](auto w) {
                return with_format(format, [&](auto f) {
                    return launch_blocks(name, st, all, threads, [&](uint64_t first, uint32_t blocks) {
                        using T = decltype(t);
                        using W = decltype(w);
                        constexpr int F = decltype(f)::value;
                        p.first = (uint32_t)first;
                        // The small tile with one term: 64 rows a step, with more 32, whose two groups' stages
                        // of 64 would need 192 KB of LDS.  bf16 int8 with 64 and with 32: 4096x4096x1024 48.3 and
                        // 49.4 us, 2048x2048x2048 29.2 and 29.9, 8192x1024x1024 33.5 and 34.1, 512x1024x4096 14.8
                        // and 14.2.
                        if (s.tile == 256)
                            k_weight_grad<T, W, F, 256, 32, 1, kExperts><<<blocks, threads, 0, st>>>(p);
                        else
                            k_weight_grad<T, W, F, 128, T::kTerms == 1 ? 64 : 32, 2, kExperts>
                                <<<blocks, threads, 0, st>>>(p);
                    });
                });
            });
        });
        if (rc || s.slices == 1) return rc;
    }
    const uint64_t all = (uint64_t)p.tiles_all * (s.tile * s.tile / 4 / kThreads);
    return with_dtype(dtype, [&](auto t) {
        return with_weight(t, col_scale, col_scale_dtype, [&](auto w) {
            return launch_blocks("tlc_ckpt8_weight_sum", st, all, kThreads, [&](uint64_t first, uint32_t blocks) {
                p.first = (uint32_t)first;
                k_weight_sum<decltype(w)><<<blocks, kThreads, 0, st>>>(p, s.slices, s.tile);
            });
        });
    });
}

}  // namespace

extern "C" {

size_t tlc_ckpt8_weight_grad_workspace_size(uint64_t rows, uint64_t n, uint64_t cols) {
    if (!valid_shape(rows, cols) || n < 1 || n > kMaxDim) return 0;
    uint64_t bytes = 0;
    for (int terms = 1; terms <= 3; ++terms)  // of any dtype
        bytes = std::max(bytes, workspace_of(shape_of(rows, n, cols, terms)));
    return bytes;
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
    if (((n + 127) / 128) * ((cols + 127) / 128) > (1u << 24)) return TLC_ERR_INVALID_ARG;
    const Shape s = shape_of(rows, n, cols, dtype == TLC_F32 ? 3 : dtype == TLC_F16 ? 2 : 1);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < workspace_of(s)) return TLC_ERR_WORKSPACE;
    if (rows == 0 && accumulate) return TLC_OK;
    MatArgs p = {};
    p.dy = dy, p.dy_stride = dy_stride, p.codes = codes, p.scales = scales, p.rows = rows;
    p.n = (uint32_t)n, p.cols = (uint32_t)cols;
    p.code_row = (uint32_t)code_stride(cols), p.scale_row = (uint32_t)scale_stride(cols);
    p.col_scale = col_scale;
    p.dw = dw, p.dw_stride = dw_stride, p.accumulate = accumulate != 0;
    return weight_grad<false>(p, s, dtype, col_scale_dtype, format, workspace, static_cast<hipStream_t>(stream));
}

size_t tlc_expert_weight_grad_workspace_size(uint64_t rows, uint64_t n, uint64_t cols, uint64_t experts) {
    if (!valid_shape(rows, cols) || n < 1 || n > kMaxDim || experts < 1 || experts > tlc_experts::kMaxExperts) return 0;
    uint64_t bytes = 0;
    for (int terms = 1; terms <= 3; ++terms)  // of any dtype
        bytes = std::max(bytes, workspace_of(shape_of(rows, n, cols, terms, experts), experts));
    return bytes;
}

int tlc_expert_weight_grad(const void* dy, uint64_t dy_stride, int dtype, uint64_t rows, uint64_t n, int format,
                           const uint8_t* codes, const uint8_t* scales, uint64_t cols, const uint64_t* offsets,
                           uint64_t experts, const void* col_scale, int col_scale_dtype, float* dw, uint64_t dw_stride,
                           uint64_t dw_expert_stride, int accumulate, void* workspace, size_t workspace_bytes,
                           tlc_stream_t stream) {
    if (!valid_dtype(dtype) || !valid_format(format) || !valid_shape(rows, cols) || n < 1 || n > kMaxDim ||
        !valid_matrix(dw, TLC_F32, cols, dw_stride) || experts < 1 || experts > tlc_experts::kMaxExperts)
        return TLC_ERR_INVALID_ARG;
    if (offsets ? !aligned(offsets, 8) : experts != 1) return TLC_ERR_INVALID_ARG;
    if (dw_expert_stride >> 48 || (experts > 1 && dw_expert_stride < (n - 1) * dw_stride + cols))
        return TLC_ERR_INVALID_ARG;
    if (rows && (!valid_matrix(dy, dtype, n, dy_stride) || !valid_checkpoint(codes, scales)))
        return TLC_ERR_INVALID_ARG;
    if (!valid_weight(col_scale, col_scale_dtype, dtype)) return TLC_ERR_INVALID_ARG;
    if (((n + 127) / 128) * ((cols + 127) / 128) * experts > (1u << 24)) return TLC_ERR_INVALID_ARG;
    const Shape s = shape_of(rows, n, cols, dtype == TLC_F32 ? 3 : dtype == TLC_F16 ? 2 : 1, experts);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < workspace_of(s, experts))
        return TLC_ERR_WORKSPACE;
    if (rows == 0 && accumulate) return TLC_OK;
    MatArgs p = {};
    p.dy = dy, p.dy_stride = dy_stride, p.codes = codes, p.scales = scales, p.rows = rows;
    p.n = (uint32_t)n, p.cols = (uint32_t)cols;
    p.code_row = (uint32_t)code_stride(cols), p.scale_row = (uint32_t)scale_stride(cols);
    p.col_scale = col_scale;
    p.dw = dw, p.dw_stride = dw_stride, p.accumulate = accumulate != 0;
    p.experts = {offsets, (uint32_t)experts, (uint32_t)rows};
    p.dw_expert = dw_expert_stride;
    return weight_grad<true>(p, s, dtype, col_scale_dtype, format, workspace, static_cast<hipStream_t>(stream));
}

}  // extern "C"
