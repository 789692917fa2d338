// products.hip -- products of rows with a weight, or with the weight of each
// row's expert:
//   y[t][o] = sum over k of a[t][k] * w[o][k]      (both with the reduction as the fast index)
//   y[t][c] = sum over o of a[t][o] * w[o][c]      (the input gradient: the weight's rows are the reduction)
// in bf16, fp16, fp32 and, the first form, in 8-bit integers with a scale per
// row of either side.  16-bit and fp32 sums are the matrix cores' fp32, integer
// sums are exact in 32 bits.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "ckpt8.h"
#include "experts.h"
#include "launch.h"

namespace {

using namespace tlc_ckpt8;
using namespace tlc_experts;
using tlc_internal::launch;
using tlc_internal::launch_blocks;

constexpr int kThreads = 256;

typedef int i4 __attribute__((ext_vector_type(4)));
typedef short s4v __attribute__((ext_vector_type(4)));
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
    uint32_t* partial;                      // with several slices: their sums, [slices][rows][partial_row]
    uint32_t partial_row, slices, slice_k;  // n up to a multiple of 8; a slice's share of k, whole steps
    uint32_t tiles_n;
    int tail;                               // a last round of few large tiles is left to, or is, smaller ones
    uint32_t first;                         // block of the whole that the launch begins with
};

// A product of kRows rows by kRows rows, 32 over 32 bytes of the reduction or 16
// over 64 (8 bits: 16 only): a lane holds 16 bytes of row lane%kRows on either
// side, which ones by lane/kRows.
template <typename E, int kRows>
struct Sums {
    using Type = typename std::conditional<kRows == 32, f16v, f4>::type;
};
template <>
struct Sums<I8, 16> {
    using Type = i4;
};
template <typename E, int kRows, typename Sum = typename Sums<E, kRows>::Type>
__device__ __forceinline__ Sum multiply(u4 a, u4 b, Sum c) {
    constexpr bool k32 = kRows == 32;
    if constexpr (std::is_same<E, I8>::value) {
        static_assert(!k32, "8 bits multiply 16 rows");
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i4, a), __builtin_bit_cast(i4, b), c, 0, 0, 0);
    } else if constexpr (std::is_same<E, BF16>::value) {
        const b8v x = __builtin_bit_cast(b8v, a), y = __builtin_bit_cast(b8v, b);
        if constexpr (k32)
            return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, c, 0, 0, 0);
        else
            return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
    } else if constexpr (std::is_same<E, F16>::value) {
        const h8v x = __builtin_bit_cast(h8v, a), y = __builtin_bit_cast(h8v, b);
        if constexpr (k32)
            return __builtin_amdgcn_mfma_f32_32x32x16_f16(x, y, c, 0, 0, 0);
        else
            return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, c, 0, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // the reduction's order inside does not matter where both sides have it
            if constexpr (k32)
                c = __builtin_amdgcn_mfma_f32_32x32x2f32(from_bits(a[j]), from_bits(b[j]), c, 0, 0, 0);
            else
                c = __builtin_amdgcn_mfma_f32_16x16x4f32(from_bits(a[j]), from_bits(b[j]), c, 0, 0, 0);
        }
        return c;
    }
}

// `bytes` behind a pointer that all lanes share.  The compiler is kept from
// taking the sum apart, or a loop's loads would have a 64-bit pointer in
// registers each instead of one and 32-bit distances.
template <typename Elem>
__device__ __forceinline__ const Elem* later(const Elem* p, uint32_t bytes) {
    asm("" : "+v"(bytes));
    return reinterpret_cast<const Elem*>(reinterpret_cast<const char*>(p) + bytes);
}

// Sixteen bytes at any element's boundary.
template <typename Elem>
__device__ __forceinline__ u4 load16(const Elem* p) {
    if constexpr (sizeof(Elem) == 1)
        return *reinterpret_cast<const u4*>(p);  // codes are aligned
    else if constexpr (sizeof(Elem) == 2)
        return *reinterpret_cast<const u4_at2*>(p);
    else
        return *reinterpret_cast<const u4_at4*>(p);
}

// Elements first .. of a row of `limit` elements, at least sixteen bytes long:
// what lies past the row is 0.  A chunk that the row ends in is read from the
// row's last sixteen bytes and moved, word by word: a 64-bit shift by an amount
// in the last register of a wave takes another amount once a second wave lives
// on the SIMD, and the compiler put it there (fp32, few rows: wrong results as
// soon as there were more blocks than compute units).
template <typename Elem>
__device__ __forceinline__ u4 load16_cut(const Elem* row, uint32_t first, uint32_t limit) {
    const uint32_t at = min(first, limit - (uint32_t)(16 / sizeof(Elem)));
    u4 v = load16(row + at);
    const uint32_t s = min((first - at) * (uint32_t)sizeof(Elem), 16u);  // bytes past the row
    if (s & 16) v = u4{0, 0, 0, 0};
    if (s & 8) v = u4{v.z, v.w, 0, 0};
    if (s & 4) v = u4{v.y, v.z, v.w, 0};
    if constexpr (sizeof(Elem) < 4) {
        const uint32_t b = s % 4 * 8;
        v = u4{__builtin_amdgcn_alignbit(v.y, v.x, b), __builtin_amdgcn_alignbit(v.z, v.y, b),
               __builtin_amdgcn_alignbit(v.w, v.z, b), v.w >> b};
    }
    return v;
}

// A sum times the scales, a's first: a scale is at least 2^-126 and a sum that
// is not 0 at least 1, so that nothing is lost below; where a's scale is so large
// that this could leave fp32's range above, w's first.  Three roundings.
constexpr float kFar = 0x1p96f;
__device__ __forceinline__ float scaled(int sum, float sa, float sw) {
    const bool far = sa > kFar;
    return (float)sum * (far ? sw : sa) * (far ? sa : sw);
}

// Orders a wavefront's own LDS accesses across its lanes.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ s4v read_tr(const void* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4v*)p);
}

// The order of instructions among kProducts products: LDS reads, LDS writes and
// loads, each kind spread evenly over them, and the kinds apart from each other.
template <int kProducts, int kReads, int kWrites, int kLoads>
__device__ __forceinline__ void interleave() {
    // how many of n have come by the i-th product, each `early` quarters of its distance before the even place
    constexpr auto by = [](int i, int n, int early) { return n ? (4 * i * n + early * kProducts) / (4 * kProducts) : 0; };
#pragma unroll
    for (int i = 0; i < kProducts; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
        for (int r = by(i, kReads, 0); r < by(i + 1, kReads, 0); ++r) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
        for (int r = by(i, kWrites, 3); r < by(i + 1, kWrites, 3); ++r)
            __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
#pragma unroll
        for (int r = by(i, kLoads, 1); r < by(i + 1, kLoads, 1); ++r)
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
}

// Tile `b` of tiles_t by tiles_n: neighbours in bands of 4 tiles of rows.
struct Place {
    uint32_t t, n;
};
__device__ __forceinline__ Place place_of(uint32_t b, uint32_t tiles_t, uint32_t tiles_n) {
    const uint32_t band = b / (4 * tiles_n), in_band = b % (4 * tiles_n), rows = min(4u, tiles_t - band * 4);
    return {band * 4 + in_band % rows, in_band / rows};
}

// Of so many 256x256 tiles, those of the last round, where it is half empty or
// more: another launch computes them in 128x128 tiles, which fill the chip.
__host__ __device__ inline uint32_t tail_of(uint32_t tiles) { return tiles % 256 <= 128 ? tiles % 256 : 0; }

// Inner weights of 16 bits: the 16-byte slots (8 columns) of row r lie at
// slot ^ swizzle(r), so that what half a wavefront reads at once, 4 rows of 32
// columns or 8 rows of 16, falls into the 64 banks once each.
template <int kRows>
__device__ __forceinline__ int swizzle(int r) {
    return (r & 3) << 2 | (r & 1) | (kRows == 16 ? (r >> 3 & 1) << 1 : 0);
}

// A block computes kTile x kTile values of y, each of its four wavefronts a
// quarter, in steps of 128 bytes of the reduction.
//
// Two stages of LDS.  While one is multiplied, the step loaded before goes to
// the other, and as its registers are freed the step after is loaded into them:
// a load has a whole step's products to arrive in.  The block meets once a step,
// before the last part of the products, whose operands it has then read; these
// run while the next stage's first operands are read.
//
// A 256x256 tile's sums fill a wavefront's accumulation registers, so one
// wavefront a SIMD; a 128x128 tile leaves room for two.  Products of 16 rows
// take less power than those of 32, which is what bounds large sizes
// (16384x8192x8192 in 8 bits 898 -> 851 us, bf16 1625 -> 1555); the inner weight
// in the larger tile stays at 32, where 16 spill.  There 8 bits take 825 us
// (2.67 POP/s), bf16 1521 (1.45 PFLOP/s), the inner weight 1550, fp16 1600 and
// 1665; on zeros, at full clocks, 659 and 1229.  Loads straight to LDS, which
// have to be sent off all at once, stall the issue: bf16 1790 us.  A tile that
// stands alone has about 12 us beside its steps: 4096x4096x128 in 8 bits takes
// 14.9 us, half of it the results' way through LDS and to memory.
template <typename E, typename Out, bool kInner, int kTile>
__global__ __launch_bounds__(kThreads, kTile == 256 ? 1 : 2) void k_product(ProductArgs p) {
    using Elem = typename E::Elem;
    constexpr int kRows = sizeof(Elem) == 4 || (kInner && kTile == 256) ? 32 : 16;  // of a product
    constexpr int kParts = 64 / kRows, kSubs = 8 / kParts;     // 16-byte chunks of a row in it; of them in a step
    using Acc = typename Sums<E, kRows>::Type;
    constexpr int kPer = 16 / sizeof(Elem);       // elements of a 16-byte chunk
    constexpr int kStep = 128 / sizeof(Elem);     // of the reduction in a step
    constexpr int kLoads = kTile * 8 / kThreads;  // chunks a lane, of either operand
    constexpr int kWave = kTile / 2, kTiles = kWave / kRows;
    struct Stage {
        u4 a[kTile * 8], w[kTile * 8];
    };
    __shared__ Stage stage0, stage1;

    uint32_t b = p.first + blockIdx.x, slice = 0;
    Span at;
    uint32_t o0;
    if (kTile == 128 && p.tail) {
        const uint32_t across = (p.n + 255) / 256, down = tiles_of(p.experts, 256), large = down * across;
        const uint32_t rest = tail_of(large);
        if (b >= rest * 4) return;
        b = xcd_place(b, rest * 4);
        const Place place = place_of(large - rest + b / 4, down, across);
        at = tile_rows(p.experts, 256, place.t);
        at.begin += b / 2 % 2 * 128;
        at.end = min(at.end, at.begin + 128);
        o0 = place.n * 256 + b % 2 * 128;
        if (o0 >= p.n) return;
    } else {
        const uint32_t tiles_t = tiles_of(p.experts, kTile), tiles = tiles_t * p.tiles_n;
        const uint32_t total = p.tail ? tiles - tail_of(tiles) : tiles * p.slices;
        if (b >= total) return;
        b = xcd_place(b, total);
        if (p.slices > 1) slice = b / tiles, b -= slice * tiles;
        const Place place = place_of(b, tiles_t, p.tiles_n);
        at = tile_rows(p.experts, kTile, place.t);
        o0 = place.n * kTile;
    }
    if (at.begin >= at.end) return;  // the lower half of a short tile, or offsets that change meanwhile

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const uint32_t k_first = slice * p.slice_k, k_here = min(p.k - k_first, p.slice_k);
    const Elem* const a = static_cast<const Elem*>(p.a) + at.begin * p.a_stride + k_first;
    const Elem* const w = static_cast<const Elem*>(p.w) + at.expert * p.w_expert +
                          (kInner ? k_first : o0) * p.w_stride + (kInner ? 0 : k_first);
    const int steps = (int)((k_here + kStep - 1) / kStep);
    // Steps whose every chunk can be read as it lies.  A chunk past the inner
    // weight's last column runs on into the next row, so not in the last row;
    // columns past the last one only reach values that are not stored.
    const int whole = (int)((k_here - (kInner && p.n % kPer ? 1 : 0)) / kStep);

    // Rows of 128 bytes: slot c of row r holds chunk c ^ (r/2 % 8), so that the
    // 16 rows that lanes read at once fall into all 64 banks.  The inner weight's
    // rows are the reduction and kTile columns long: see operand_columns.
    const int row = tid / 8, chunk = tid % 8;
    const int place_a = row * 8 + (chunk ^ (row >> 1 & 7));
    const uint32_t last_a = at.end - at.begin - 1, last_w = p.n - 1 - o0;
    constexpr int kChunks = kTile / kPer;  // of a row of the inner weight
    constexpr int kInnerRows = kThreads / kChunks;
    static_assert(kInnerRows % 4 == 0, "a lane's rows have one swizzle");
    const int inner_row = tid / kChunks;
    const int inner_chunk = tid % kChunks;
    auto place_w = [&](int i) {
        if constexpr (!kInner) return i * kThreads + place_a;
        const int r = inner_row + i * kInnerRows;
        return r * kChunks + (sizeof(Elem) == 2 ? inner_chunk ^ swizzle<kRows>(r) : inner_chunk);
    };
    const uint32_t inner_col = o0 + inner_chunk * kPer;

    uint32_t from_a[kLoads], from_w[kInner ? 1 : kLoads];  // bytes
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        from_a[i] = min((uint32_t)row + i * 32, last_a) * (uint32_t)(p.a_stride * sizeof(Elem)) + chunk * 16;
    if constexpr (kInner) {
        from_w[0] = inner_row * (uint32_t)(p.w_stride * sizeof(Elem)) +
                    (inner_col < p.n ? inner_col : 0) * (uint32_t)sizeof(Elem);
    } else {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            from_w[i] = min((uint32_t)row + i * 32, last_w) * (uint32_t)(p.w_stride * sizeof(Elem)) + chunk * 16;
    }
    u4 ga[kLoads], gw[kLoads];
    auto load_whole = [&](int s, int from, int to) {
        const Elem* const pa = a + (uint64_t)s * kStep;
        const Elem* const pw = w + (uint64_t)s * kStep * (kInner ? p.w_stride : 1);
#pragma unroll
        for (int i = from; i < to; ++i) {
            ga[i] = load16(later(pa, from_a[i]));
            gw[i] = load16(kInner ? later(pw + i * kInnerRows * p.w_stride, from_w[0])
                                  : later(pw, from_w[kInner ? 0 : i]));
        }
    };
    auto load = [&](int s, int from, int to) {
        if (s < whole) return load_whole(s, from, to);
        // in the whole row, which has sixteen bytes where a slice's end may not
        const uint32_t k0 = k_first + s * kStep + chunk * kPer;
#pragma unroll
        for (int i = from; i < to; ++i) {
            ga[i] = load16_cut(later(a - k_first, from_a[i] - chunk * 16), k0, p.k);
            if constexpr (!kInner) {
                gw[i] = load16_cut(later(w - k_first, from_w[i] - chunk * 16), k0, p.k);
            } else {
                const uint32_t o = s * kStep + inner_row + i * kInnerRows;
                gw[i] = load16_cut(w + min(o, k_here - 1) * p.w_stride, inner_col, p.n);
                if (o >= k_here) gw[i] = u4{0, 0, 0, 0};
            }
        }
    };
    auto store = [&](Stage& st, int from, int to) {
#pragma unroll
        for (int i = from; i < to; ++i) {
            st.a[i * kThreads + place_a] = ga[i];
            st.w[place_w(i)] = gw[i];
        }
    };

    const int wi = (wave >> 1) * kWave, wc = (wave & 1) * kWave;
    const int r_lane = lane % kRows, part = lane / kRows;
    Acc acc[kTiles][kTiles] = {};
    auto operand_rows = [&](const u4* st, int sub, int from) {  // of kRows rows beginning with `from`
        return st[(from + r_lane) * 8 + ((sub * kParts + part) ^ (r_lane >> 1 & 7))];
    };
    // Columns of rows of the reduction.  16 bits: the transposing read gives
    // each of 16 lanes 4 rows of one column from 4 rows of 16 columns.
    auto operand_columns = [&](const u4* st, int sub, int from) {
        if constexpr (sizeof(Elem) == 2) {
            const int r = part * 8 + (lane >> 2 & 3);
            const int slot = from / 8 + (kRows == 32 ? (lane >> 4 & 1) * 2 : 0) + (lane >> 1 & 1);
            const char* q = reinterpret_cast<const char*>(st) + (sub * kParts * 8 + r) * kTile * 2 +
                            (slot ^ swizzle<kRows>(r)) * 16 + (lane & 1) * 8;
            const s4v lo = read_tr(q), hi = read_tr(q + 4 * kTile * 2);
            return __builtin_bit_cast(u4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const uint32_t* q =
                reinterpret_cast<const uint32_t*>(st) + (sub * kParts * 4 + part * 4) * kTile + from + r_lane;
            return u4{q[0], q[kTile], q[2 * kTile], q[3 * kTile]};
        }
    };
    u4 fa[2][kTiles], fw[2][kTiles];
    auto operands = [&](const Stage& st, int sub) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
            fw[sub & 1][i] =
                kInner ? operand_columns(st.w, sub, wc + i * kRows) : operand_rows(st.w, sub, wc + i * kRows);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) fa[sub & 1][i] = operand_rows(st.a, sub, wi + i * kRows);
    };
    auto products = [&](const u4* ra, const u4* rw) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int c = 0; c < kTiles; ++c) acc[i][c] = multiply<E, kRows>(rw[c], ra[i], acc[i][c]);
    };
    // of a sub-step; the inner fp32 weight is read value by value and left to the compiler
    constexpr bool kSchedule = sizeof(Elem) <= 2 || !kInner;
    constexpr int kProducts = kTiles * kTiles * (sizeof(Elem) == 4 ? 4 : 1), kReads = kTiles * (kInner ? 3 : 2);
    // Step s multiplies `now`.  The first chunks of step s + 1 are in `next` when
    // it begins; it stores the others and, when `now` has been read, the first
    // ones of step s + 2, and loads into each register that frees what will be
    // stored from it a step later.  kMain: all of it, of whole steps, without a
    // branch, so that one schedule spans it.
    constexpr int kFirst = kLoads / kSubs;  // those stored during the last sub-step
    auto step = [&](Stage& now, Stage& next, int s, auto main) {
        constexpr bool kMain = decltype(main)::value;
        if (kMain || (s + 1 >= 0 && s + 1 < steps)) store(next, kFirst, kLoads);
        if constexpr (kMain)
            load_whole(s + 2, kFirst, kLoads);
        else if (s + 2 >= 0 && s + 2 < steps)
            load(s + 2, kFirst, kLoads);
        if (kMain || s >= 0) {
#pragma unroll
            for (int sub = 0; sub < kSubs - 1; ++sub) {
                operands(now, sub + 1);
                products(fa[sub & 1], fw[sub & 1]);
            }
        }
        if constexpr (kMain && kSchedule)
            interleave<(kSubs - 1) * kProducts, (kSubs - 1) * kReads, 2 * (kLoads - kFirst), 2 * (kLoads - kFirst)>();
        __syncthreads();
        u4 la[kTiles], lw[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) la[i] = fa[1][i], lw[i] = fw[1][i];
        if (kMain || (s + 1 >= 0 && s + 1 < steps)) operands(next, 0);
        if (kMain || (s + 2 >= 0 && s + 2 < steps)) store(now, 0, kFirst);
        if constexpr (kMain)
            load_whole(s + 3, 0, kFirst);
        else if (s + 3 < steps)
            load(s + 3, 0, kFirst);
        if (kMain || s >= 0) products(la, lw);
        if constexpr (kMain && kSchedule) interleave<kProducts, kReads, 2 * kFirst, 2 * kFirst>();
    };
    // The steps before 0 fill the pipeline.
    for (int s = -3; s < steps; ++s) {
        if (s >= 0 && s % 2 == 0 && s + 4 < whole) {
            // Nothing under way at the loop's beginning: else the compiler, which
            // does not know how much that is, waits in every turn for loads that
            // were only just sent off (vmcnt(7) in place of 15).
            __builtin_amdgcn_s_waitcnt(0x0F70);
            for (; s + 4 < whole; s += 2) {
                step(stage0, stage1, s, Int<1>{});
                step(stage1, stage0, s + 1, Int<1>{});
            }
        }
        step(s & 1 ? stage1 : stage0, s & 1 ? stage0 : stage1, s, Int<0>{});
    }
    __syncthreads();

    // register j of a lane: row lane%16, column 4*(lane/16) + j (of 32 rows: row
    // lane%32, column 8*(j/4) + 4*(lane/32) + j%4).
    // 64 rows at a time through LDS, so that a lane has eight values of a row: 16
    // bytes of row r at place ^ (r%16), which spreads a column over the banks.
    // Short loops: code that runs once costs more to fetch than to run.
    static_assert(2 * sizeof(Stage) >= 4 * 64 * kWave * sizeof(uint32_t), "the wavefronts' rows fit");
    u4* const mine = reinterpret_cast<u4*>(wave < 2 ? &stage0 : &stage1) + wave % 2 * 16 * kWave;
    constexpr int kAcross = kWave / 8, kDown = 64 / kAcross, kDeep = 4;
    const uint32_t col = o0 + wc + lane % kAcross * 8;
    const int count = (int)min((int64_t)p.n - (int64_t)col, (int64_t)8);
    const bool add = std::is_same<E, I8>::value && std::is_same<Out, F32>::value && p.accumulate;
    float sw[8];
    if constexpr (std::is_same<E, I8>::value) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sw[j] = j < count ? p.w_scales[(uint64_t)at.expert * p.n + col + j] : 0.0f;
    }
    float row_scales[kTiles * kRows / 64] = {};  // a row a lane
    if constexpr (std::is_same<E, I8>::value) {
#pragma unroll
        for (int g = 0; g < kTiles * kRows / 64; ++g)
            row_scales[g] = p.a_scales[min(at.begin + wi + g * 64 + lane, at.end - 1)];
    }
#pragma unroll
    for (int i = 0; i < kTiles; i += 64 / kRows) {
        // a's scales that large are rare: the usual order alone saves two of six operations a value
        const float mine_sa = row_scales[i * kRows / 64];
        const bool far = std::is_same<E, I8>::value && __any(mine_sa > kFar);
#pragma unroll
        for (int h = 0; h < 64 / kRows; ++h)
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
#pragma unroll
                for (int j = 0; j < kRows * kRows / 64; j += 4) {
                    const auto& v = acc[i + h][c];
                    const int r = h * kRows + r_lane, to = (c * kRows + j * 2) / 4 + part;
                    *reinterpret_cast<typename Sums<E, 16>::Type*>(mine + r * (kWave / 4) + (to ^ (r & 15))) =
                        typename Sums<E, 16>::Type{v[j], v[j + 1], v[j + 2], v[j + 3]};
                }
        wave_sync();
        const uint32_t t0 = at.begin + wi + i * kRows;
#pragma unroll 1
        for (int q = 0; q < 64 && t0 + q < at.end; q += kDown * kDeep) {
            u4 in[kDeep][2];
            float sa[kDeep];
#pragma unroll
            for (int d = 0; d < kDeep; ++d) {
                const uint32_t r = q + d * kDown + lane / kAcross;
                const u4* const from = mine + r * (kWave / 4);
                in[d][0] = from[lane % kAcross * 2 ^ (r & 15)], in[d][1] = from[(lane % kAcross * 2 + 1) ^ (r & 15)];
                if constexpr (std::is_same<E, I8>::value) sa[d] = __shfl(mine_sa, (int)r);
            }
#pragma unroll
            for (int d = 0; d < kDeep; ++d) {
                const uint32_t t = t0 + q + d * kDown + lane / kAcross;
                if (p.partial) {
                    u4* const o = reinterpret_cast<u4*>(
                        p.partial + ((uint64_t)slice * p.experts.rows + t) * p.partial_row + col);
                    if (t < at.end && count > 0) o[0] = in[d][0], o[1] = in[d][1];
                    continue;
                }
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t u = in[d][j / 4][j % 4];
                    if constexpr (std::is_same<E, I8>::value)
                        v[j] = (float)(int)u * sa[d] * sw[j];
                    else
                        v[j] = from_bits(u);
                }
                if constexpr (std::is_same<E, I8>::value) {
                    if (far) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = scaled((int)in[d][j / 4][j % 4], sa[d], sw[j]);
                    }
                }
                if (t >= at.end || count < 8) continue;
                typename Out::Elem* const o = static_cast<typename Out::Elem*>(p.y) + t * p.y_stride + col;
                if (add) {
                    float old[8];
                    unpack8<Out>(load8<Out>(o, 8, true), old);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += old[j];
                }
                store8<Out>(o, 8, pack8<Out>(v));
            }
        }
        // the last one to seven columns of y, a row a lane
        const uint32_t ragged = p.n & ~7u, t = t0 + lane;
        if (!p.partial && ragged < p.n && ragged >= o0 + wc && ragged < o0 + wc + kWave && t < at.end) {
#pragma unroll 1
            for (uint32_t c = ragged; c < p.n; ++c) {
                typename Out::Elem* const o = static_cast<typename Out::Elem*>(p.y) + t * p.y_stride + c;
                const uint32_t in_row = c - (o0 + wc);
                const uint32_t u = reinterpret_cast<const uint32_t*>(
                    mine + lane * (kWave / 4) + (in_row / 4 ^ (lane & 15)))[in_row % 4];
                float v;
                if constexpr (std::is_same<E, I8>::value)
                    v = scaled((int)u, p.a_scales[t], p.w_scales[(uint64_t)at.expert * p.n + c]);
                else
                    v = from_bits(u);
                if (add) v += (float)*o;
                *o = (typename Out::Elem)v;
            }
        }
        wave_sync();
    }
}

// Few rows: a block computes 16x16 values of y, its eight wavefronts taking the
// reduction in turns of 128 bytes.  Operands go from memory to the matrix cores
// without LDS: w is read once in all, the few rows of a once for each block.
// Two or four times the columns a block (so fewer reads of a), 4 or 16
// wavefronts and 8 turns under way measured the same or slower (1x8192x4096
// bf16 17.0 us with its launch; 16.8 to 28.3).  A row of 8192x4096 bf16, 67 MB,
// takes about 11 us of its own, 16 rows of 8192x8192 40.
template <typename E, typename Out>
__global__ __launch_bounds__(512) void k_product_few(ProductArgs p) {
    constexpr int kWaves = 8, kDeep = 4;  // turns under way
    using Elem = typename E::Elem;
    using Acc = typename Sums<E, 16>::Type;
    constexpr int kPer = 16 / sizeof(Elem), kTurn = 128 / sizeof(Elem);
    __shared__ uint32_t box[kWaves][4][64];
    const uint32_t b = p.first + blockIdx.x, tile = b / p.tiles_n;
    if (tile >= tiles_of(p.experts, 16)) return;
    const Span at = tile_rows(p.experts, 16, tile);
    if (at.begin >= at.end) return;
    const uint32_t o0 = b % p.tiles_n * 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t row = lane % 16, part = lane / 16;
    const Elem* const a = static_cast<const Elem*>(p.a) + min(at.begin + row, at.end - 1) * p.a_stride;
    const Elem* const w = static_cast<const Elem*>(p.w) + at.expert * p.w_expert + min(o0 + row, p.n - 1) * p.w_stride;
    const int whole = (int)(p.k / kTurn);
    Acc acc = {};
    int turn = wave;
    for (; turn + (kDeep - 1) * kWaves < whole; turn += kDeep * kWaves) {
        u4 ga[kDeep][2], gw[kDeep][2];
#pragma unroll
        for (int d = 0; d < kDeep; ++d)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t k = (turn + d * kWaves) * kTurn + (j * 4 + part) * kPer;
                gw[d][j] = load16(w + k);
                ga[d][j] = load16(a + k);
            }
#pragma unroll
        for (int d = 0; d < kDeep; ++d)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc = multiply<E, 16>(gw[d][j], ga[d][j], acc);
    }
    for (; turn * kTurn < (int)p.k; turn += kWaves) {
        u4 ga[2], gw[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t k = turn * kTurn + (j * 4 + part) * kPer;
            gw[j] = turn < whole ? load16(w + k) : load16_cut(w, k, p.k);
            ga[j] = turn < whole ? load16(a + k) : load16_cut(a, k, p.k);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) acc = multiply<E, 16>(gw[j], ga[j], acc);
    }
    // register j of a lane: row 4*(lane/16) + j of w, row lane%16 of a
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const auto v = acc[j];
        box[wave][j][lane] = __builtin_bit_cast(uint32_t, v);
    }
    __syncthreads();
    const uint32_t c = threadIdx.x % 16, r = threadIdx.x / 16, t = at.begin + r, o = o0 + c;
    if (t >= at.end || r >= 16 || o >= p.n) return;
    typename std::conditional<std::is_same<E, I8>::value, int, float>::type sum = 0;
#pragma unroll
    for (int u = 0; u < kWaves; ++u) {
        const uint32_t v = box[u][c % 4][c / 4 * 16 + r];
        if constexpr (std::is_same<E, I8>::value)
            sum += (int)v;
        else
            sum += from_bits(v);
    }
    float y;
    if constexpr (std::is_same<E, I8>::value)
        y = scaled(sum, p.a_scales[t], p.w_scales[(uint64_t)at.expert * p.n + o]);
    else
        y = sum;
    typename Out::Elem* const out = static_cast<typename Out::Elem*>(p.y) + t * p.y_stride + o;
    if (std::is_same<E, I8>::value && std::is_same<Out, F32>::value && p.accumulate) y += (float)*out;
    *out = (typename Out::Elem)y;
}

// y from the slices' sums, added in order: eight columns of a row a thread.
template <typename E, typename Out>
__global__ __launch_bounds__(kThreads) void k_product_sum(ProductArgs p) {
    constexpr uint32_t kRows = 32, kAcross = kThreads / kRows;  // of a block
    const uint32_t b = p.first + blockIdx.x, tile = b / p.tiles_n;
    if (tile >= tiles_of(p.experts, kRows)) return;
    const Span at = tile_rows(p.experts, kRows, tile);
    const uint32_t t = at.begin + threadIdx.x / kAcross, col = (b % p.tiles_n * kAcross + threadIdx.x % kAcross) * 8;
    if (t >= at.end || col >= p.n) return;
    const uint32_t* const in = p.partial + (uint64_t)t * p.partial_row + col;
    const uint64_t next = (uint64_t)p.experts.rows * p.partial_row;
    typename std::conditional<std::is_same<E, I8>::value, int, float>::type sum[8] = {};
#pragma unroll 4
    for (uint32_t s = 0; s < p.slices; ++s) {
        const u4 lo = *reinterpret_cast<const u4*>(in + s * next), hi = *reinterpret_cast<const u4*>(in + s * next + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t u = j < 4 ? lo[j & 3] : hi[j & 3];
            if constexpr (std::is_same<E, I8>::value)
                sum[j] += (int)u;
            else
                sum[j] += from_bits(u);
        }
    }
    const int count = (int)min(p.n - col, 8u);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (std::is_same<E, I8>::value)
            v[j] = j < count ? scaled(sum[j], p.a_scales[t], p.w_scales[(uint64_t)at.expert * p.n + col + j]) : 0.0f;
        else
            v[j] = sum[j];
    }
    typename Out::Elem* const o = static_cast<typename Out::Elem*>(p.y) + t * p.y_stride + col;
    if (std::is_same<E, I8>::value && std::is_same<Out, F32>::value && p.accumulate) {
        float old[8];
        unpack8<Out>(load8<Out>(o, count), old);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += old[j];
    }
    store8<Out>(o, count, pack8<Out>(v));
}

// Rows of less than 16 bytes: a value a thread.
template <typename Elem>
bool narrow(uint64_t n, uint64_t k, bool inner) {
    return std::min(k, inner ? n : k) < 16 / sizeof(Elem);
}
template <typename E, bool kInner>
__global__ __launch_bounds__(kThreads) void k_product_narrow(ProductArgs p, uint64_t first) {
    using Elem = typename E::Elem;
    const uint64_t v = (first + blockIdx.x) * kThreads + threadIdx.x;
    const uint32_t t = (uint32_t)(v / p.n), o = (uint32_t)(v % p.n);
    // the expert: the last whose rows begin at or before t and do not end there
    uint32_t expert = 0;
    bool found = !p.experts.offsets;
    if (p.experts.offsets) {
        uint32_t before = 0;
        for (uint32_t e = 0; e < p.experts.count && !found; ++e) {
            const uint32_t begin = max(before, held(p.experts, e)), end = max(begin, held(p.experts, e + 1));
            found = t >= begin && t < end;
            expert = e, before = end;
        }
    }
    if (t >= p.experts.rows || !found) return;
    const Elem* const a = static_cast<const Elem*>(p.a) + t * p.a_stride;
    const Elem* const w = static_cast<const Elem*>(p.w) + expert * p.w_expert + (kInner ? o : o * p.w_stride);
    float sum = 0.0f;
    for (uint32_t k = 0; k < p.k; ++k) sum = fmaf((float)a[k], (float)w[kInner ? k * p.w_stride : k], sum);
    static_cast<Elem*>(p.y)[t * p.y_stride + o] = (Elem)sum;
}

// The tile and the slices of the reduction, by the least of an estimate in
// microseconds.  Measured, in steps of 128 bytes: a 128x128 tile takes 0.5 us a
// step alone on a CU, two at once 1.0, a 256x256 tile 1.4 to 1.6 by the power
// that the whole call draws (one round of 4096x4096 1.38 to 1.46, eight rounds of
// 16384x8192x8192 1.49 in bf16 and 1.61 in 8 bits; taken as 1.55), in 16 bits
// and in 8 (fp32, in the smaller tile only: 2.0 and 4.6); a tile's beginning and
// end take 4 and 8 us.  Slices fill the chip where the tiles do not and cost
// writing and reading their sums.  Rows of experts are taken as equally many:
// half a tile more for each.
//   bf16, tiles of 128 and 256 in one slice, and the best in slices, us:
//   16384x4096x4096   504  407
//   4096x4096x1024     42   36
//   4096x1024x4096     41   81
//   2048x2048x2048     24   47
//   512x4096x4096      37   79   2 slices of 128: 31
//   128x4096x4096      36   78   8 slices of 128: 20
//   1024x1024x16384   123  274   4 slices of 128: 47
//   32 experts of 1024x2048, 4096 rows   29   49
// The estimate takes the fastest in all of them.
struct Shape {
    uint32_t tile, slices, slice_k;
};
Shape shape_of(uint64_t rows, uint64_t n, uint64_t k, uint64_t experts, bool grouped, int size) {
    const uint64_t step = 128 / size, steps = (k + step - 1) / step;
    Shape best = {};
    double least = 0.0;
    for (uint32_t tile = 128; tile <= (size == 4 ? 128 : 256); tile *= 2) {
        const uint64_t worst = most_tiles(rows, experts, tile, grouped);
        const double tiles_t = grouped ? std::min((double)worst, (double)rows / tile + 0.5 * (double)experts) : worst;
        for (uint64_t slices : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
            if (slices > 1 && steps < 4 * slices) break;
            const uint64_t share = (steps + slices - 1) / slices, cut = (steps + share - 1) / share;
            if (worst * ((n + tile - 1) / tile) * cut > 0xFFFFFFFFull) break;
            const double blocks = std::max(1.0, std::ceil(tiles_t) * (double)((n + tile - 1) / tile) * (double)cut);
            double us;
            if (tile == 256) {
                const double rest = cut == 1 ? (double)tail_of((uint32_t)std::min(blocks, 4e9)) : 0.0;
                us = std::ceil((blocks - rest) / 256) * (1.55 * (double)share + 8.0);
                if (rest > 0.0) us += (rest <= 64 ? 0.5 : 1.0) * (double)share + 7.0;
            } else {
                const double one = (size == 4 ? 2.0 : 0.5) * (double)share, two = (size == 4 ? 4.6 : 1.0) * (double)share;
                const double full = std::floor(blocks / 512), rest = blocks - full * 512;
                us = full * (two + 4.0) + (rest <= 0.0 ? 0.0 : rest <= 256 ? one + 4.0 : two + 4.0);
            }
            if (cut > 1) us += 4.0 + (2.0 * (double)cut + 1.0) * (double)rows * (double)n * 4.0 / 5.5e6;
            if (!best.tile || us < least) best = {tile, (uint32_t)cut, (uint32_t)(share * step)}, least = us;
        }
    }
    return best;
}

// Whether rows are so few that w's bytes alone count: 8 to an expert on average
// and 16 more, in fp32, whose tile is slow, 32 to an expert, which is where both
// measured the same for rows spread evenly.  Kernels for few rows and for tiles
// (with slices), us with the launch, in 8 bits, bf16 and fp32:
//   1 expert of 4096x4096, 16 rows    9, 12, 25 and 16, 19, 51
//                          32 rows   12, 19, 38 and 17, 18, 51
//                          64 rows   20, 33, 67 and 19, 19, 53
//   16 of 2048x4096, 4 rows each     39, 60, 138 and 54, 82, 368
//                    16 rows each    48, 83, 165 and 44, 82, 348
//   32 of 1024x2048, 32 rows each    49, 74, 144 and 24, 41, 175
// What that rule does not see, since the host does not: rows that are nearly all
// one expert's, whose weight is then read once for each 16 of them.  All on one:
//   64 of 4096x4096, 528 rows        147 and 259 us in 8 bits and bf16, in tiles 23 and 35
//                                    (spread evenly 260 and 466, in tiles 262 and 490)
//   32 of 2048x2048, 1024 rows       238 in fp32, in tiles 77 (spread evenly 265)
bool few(uint64_t rows, uint64_t experts, int size) { return rows <= (size == 4 ? 32 * experts : 8 * experts + 16); }

uint64_t partial_row(uint64_t n) { return (n + 7) / 8 * 8; }
uint64_t workspace_of(const Shape& s, uint64_t rows, uint64_t n) {
    return s.slices > 1 ? (s.slices * rows * partial_row(n) * 4 + 255) / 256 * 256 : 0;
}

template <typename E, typename Out, bool kInner>
int product(const char* name, ProductArgs p, void* workspace, size_t workspace_bytes, hipStream_t st) {
    using Elem = typename E::Elem;
    const bool grouped = p.experts.offsets != nullptr;
    if constexpr (!std::is_same<E, I8>::value) {
        if (narrow<Elem>(p.n, p.k, kInner)) {
            const uint64_t blocks = ((uint64_t)p.experts.rows * p.n + kThreads - 1) / kThreads;
            return launch_blocks(name, st, blocks, kThreads, [&](uint64_t first, uint32_t here) {
                k_product_narrow<E, kInner><<<here, kThreads, 0, st>>>(p, first);
            });
        }
    }
    if constexpr (!kInner) {
        if (few(p.experts.rows, p.experts.count, sizeof(Elem))) {
            p.tiles_n = (p.n + 15) / 16;
            const uint64_t tiles_t = most_tiles(p.experts.rows, p.experts.count, 16, grouped);
            return launch_blocks(name, st, tiles_t * p.tiles_n, 512, [&](uint64_t first, uint32_t blocks) {
                p.first = (uint32_t)first;
                k_product_few<E, Out><<<blocks, 512, 0, st>>>(p);
            });
        }
    }
    const Shape s = shape_of(p.experts.rows, p.n, p.k, p.experts.count, grouped, sizeof(Elem));
    const uint64_t need = workspace_of(s, p.experts.rows, p.n);
    if (need && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return TLC_ERR_WORKSPACE;
    p.slices = s.slices, p.slice_k = s.slice_k, p.partial_row = (uint32_t)partial_row(p.n);
    p.partial = s.slices > 1 ? static_cast<uint32_t*>(workspace) : nullptr;
    auto go = [&](auto tile) {
        constexpr int kTile = decltype(tile)::value;
        p.tiles_n = (p.n + kTile - 1) / kTile;
        const uint64_t tiles_t = most_tiles(p.experts.rows, p.experts.count, kTile, grouped);
        return launch_blocks(name, st, tiles_t * p.tiles_n * s.slices, kThreads, [&](uint64_t first, uint32_t blocks) {
            p.first = (uint32_t)first;
            k_product<E, Out, kInner, kTile><<<blocks, kThreads, 0, st>>>(p);
        });
    };
    int rc = TLC_OK;
    if constexpr (sizeof(Elem) == 4) {
        rc = go(Int<128>{});
    } else if (s.tile == 128) {
        rc = go(Int<128>{});
    } else {
        const uint64_t large = most_tiles(p.experts.rows, p.experts.count, 256, grouped) * ((p.n + 255) / 256);
        p.tail = s.slices == 1 && (grouped || tail_of((uint32_t)large));
        rc = go(Int<256>{});
        if (!rc && p.tail)
            rc = launch(name, st, [&] {
                p.first = 0;
                k_product<E, Out, kInner, 128><<<(uint32_t)std::min<uint64_t>(large, 128) * 4, kThreads, 0, st>>>(p);
            });
    }
    if (rc || s.slices == 1) return rc;
    p.tiles_n = (p.partial_row / 8 + 7) / 8;
    const uint64_t tiles_t = most_tiles(p.experts.rows, p.experts.count, 32, grouped);
    return launch_blocks("tlc_product_sum", st, tiles_t * p.tiles_n, kThreads, [&](uint64_t first, uint32_t blocks) {
        p.first = (uint32_t)first;
        k_product_sum<E, Out><<<blocks, kThreads, 0, st>>>(p);
    });
}

constexpr uint64_t kMaxTiles = 1u << 24;   // of 128 x 128
constexpr uint64_t kMaxStride = 1u << 22;  // a tile's rows, 256 of 16 bits or 128 of fp32, lie within 2^31 bytes

bool valid_product(uint64_t rows, uint64_t n, uint64_t k, uint64_t experts) {
    return valid_shape(rows, n) && k >= 1 && k <= kMaxDim && experts >= 1 && experts <= kMaxExperts &&
           most_tiles(rows, experts, 128, true) * ((n + 127) / 128) <= kMaxTiles;
}
bool valid_offsets(const void* offsets, uint64_t experts) { return offsets ? aligned(offsets, 8) : experts == 1; }

// Of one expert, with offsets and without: what either call may need.
size_t product_workspace(uint64_t rows, uint64_t n, uint64_t k, uint64_t experts, int size, bool inner) {
    if (rows < 1 || (!inner && few(rows, experts, size)) || !valid_product(rows, n, k, experts)) return 0;
    uint64_t bytes = workspace_of(shape_of(rows, n, k, experts, true, size), rows, n);
    if (experts == 1) bytes = std::max(bytes, workspace_of(shape_of(rows, n, k, 1, false, size), rows, n));
    return bytes;
}

int expert_call(const char* name, bool inner, const void* a, uint64_t a_stride, int dtype, uint64_t rows,
                uint64_t k, const void* w, uint64_t w_stride, uint64_t w_expert_stride, uint64_t w_cols, uint64_t n,
                const uint64_t* offsets, uint64_t experts, void* y, uint64_t y_stride, void* workspace,
                size_t workspace_bytes, tlc_stream_t stream) {
    if (!valid_dtype(dtype) || !valid_product(rows, n, k, experts) || !valid_offsets(offsets, experts) || w_expert_stride >> 48 ||
        a_stride > kMaxStride || w_stride > kMaxStride)
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
        return inner ? product<T, T, true>(name, p, workspace, workspace_bytes, st)
                     : product<T, T, false>(name, p, workspace, workspace_bytes, st);
    });
}

}  // namespace

extern "C" {

size_t tlc_q8_product_workspace_size(uint64_t rows, uint64_t n, uint64_t k, uint64_t experts) {
    const uint64_t stride = tlc_q8_code_stride(k);
    return stride ? product_workspace(rows, n, stride, experts, 1, false) : 0;
}

size_t tlc_expert_product_workspace_size(uint64_t rows, uint64_t k, uint64_t n, uint64_t experts, int dtype) {
    if (!valid_dtype(dtype)) return 0;
    const int size = dtype == TLC_F32 ? 4 : 2;
    return k < 16u / size ? 0 : product_workspace(rows, n, k, experts, size, false);
}

size_t tlc_expert_input_grad_workspace_size(uint64_t rows, uint64_t n, uint64_t k, uint64_t experts, int dtype) {
    if (!valid_dtype(dtype)) return 0;
    const int size = dtype == TLC_F32 ? 4 : 2;
    return std::min(n, k) < 16u / size ? 0 : product_workspace(rows, k, n, experts, size, true);
}

int tlc_q8_product(const int8_t* a, const float* a_scales, uint64_t rows, const int8_t* w, const float* w_scales,
                   uint64_t n, uint64_t k, const uint64_t* offsets, uint64_t experts, void* y, uint64_t y_stride,
                   int dtype, int accumulate, void* workspace, size_t workspace_bytes, tlc_stream_t stream) {
    const uint64_t stride = tlc_q8_code_stride(k);
    if (!valid_dtype(dtype) || !stride || !valid_product(rows, n, k, experts) || !valid_offsets(offsets, experts) ||
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
        return product<I8, decltype(t), false>("tlc_q8_product", p, workspace, workspace_bytes,
                                               static_cast<hipStream_t>(stream));
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
