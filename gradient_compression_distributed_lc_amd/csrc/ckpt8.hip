// ckpt8.hip -- 8-bit checkpoints of activations: pack and unpack, the
// activation functions and the root-mean-square norm with their gradients.
// The weight gradient from a checkpoint is in ckpt8_matrix.hip.
//
// Every kernel here reads each input once and writes each output once; all are
// bound by HBM.  A lane holds eight consecutive values (one 16-byte access in
// 16 bits, two in fp32), so that a group of 32 columns is four lanes and its
// largest magnitude takes two cross-lane moves.

#include <algorithm>

#include "ckpt8.h"
#include "launch.h"

namespace {

using namespace tlc_ckpt8;
using tlc_internal::launch;
using tlc_internal::launch_blocks;

constexpr int kThreads = 256;

// ---- activation functions --------------------------------------------------
//
// f(x) = x*P(x) with P the normal distribution function (gelu), the logistic
// function of 2*sqrt(2/pi)*(x + 0.044715x^3) (gelu_tanh: (1+tanh u)/2 is the
// logistic function of 2u) or of x (silu); f'(x) = P(x) + x*P'(x).
// fp32 tensors take the library's erfc and exp; 16-bit ones the hardware's
// exp2 and reciprocal, and for gelu a fit of P's tail: with t = 1/(1 + p|x|),
// P(-|x|) = exp(-x^2/2) * t*Q(t), Q of degree 7 and p fitted to the least
// largest relative error (8.2e-8 for all |x| <= 13.4, past which P is below
// 2^-126).  In 16 bits x*x is exact in fp32, so what P is off by relative to
// itself is the exponent's rounding, x^2/2 * 2^-23.4, and a few 2^-24: f, f' and
// the codes made of f keep their type's precision down to where f vanishes.

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhScale = 0.7978845608028654f;  // sqrt(2/pi)

__device__ __forceinline__ float fast_logistic(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// The logistic function of u, and with kBoth that of -u in *rest: of
// 1/(1 + e^-|u|) and e^-|u|/(1 + e^-|u|) neither cancels, where 1 - p would be
// off by 2^-25 however small it is (times x*u' in the slope of gelu_tanh,
// hundreds of roundings of it in fp32).  16-bit tensors take 1 - p: 2^-24 of
// x*u', which is below 40 where 1 - p is not 0 yet, is a hundredth of their
// rounding.
template <bool kPrecise, bool kBoth>
__device__ __forceinline__ float logistic(float u, float* rest) {
    if constexpr (!kPrecise) {
        const float p = fast_logistic(u);
        if constexpr (kBoth) *rest = 1.0f - p;
        return p;
    } else {
        const float e = expf(-fabsf(u)), high = 1.0f / (1.0f + e), low = e * high;
        if constexpr (kBoth) *rest = u < 0.0f ? high : low;
        return u < 0.0f ? low : high;
    }
}

// P(x), and with kSlope also f'(x).
template <int A, bool kPrecise, bool kSlope>
__device__ __forceinline__ float act_p(float x, float* slope) {
    float p, q;  // q: the logistic function of the negative argument
    if constexpr (A == TLC_ACT_GELU) {
        float g;  // exp(-x^2/2)
        if constexpr (kPrecise) {
            p = 0.5f * erfcf(-0.70710678118654752f * x);
            g = kSlope ? expf(-0.5f * x * x) : 0.0f;
        } else {
            const float t = __builtin_amdgcn_rcpf(fmaf(0.30389324f, fabsf(x), 1.0f));
            g = __builtin_amdgcn_exp2f(x * x * (-0.5f * kLog2e));
            float r = fmaf(t, 0.0368811004f, -0.155570209f);
            r = fmaf(t, r, 0.192927569f);
            r = fmaf(t, r, -0.0437285975f);
            r = fmaf(t, r, 0.123851091f);
            r = fmaf(t, r, 0.102307118f);
            r = fmaf(t, r, 0.122140631f);
            r = fmaf(t, r, 0.121191330f);
            r = r * t * g;
            p = x < 0.0f ? r : 1.0f - r;
        }
        if constexpr (kSlope) *slope = fmaf(x * 0.3989422804014327f, g, p);
    } else if constexpr (A == TLC_ACT_GELU_TANH) {
        // past 30 the logistic function is 0 or 1, and the cube would overflow later
        const float c = x != x ? x : fminf(fmaxf(x, -30.0f), 30.0f), cc = c * c;
        const float u = 2.0f * kTanhScale * c * fmaf(0.044715f, cc, 1.0f);
        p = logistic<kPrecise, kSlope>(u, &q);
        if constexpr (kSlope) {
            const float du = 2.0f * kTanhScale * fmaf(0.134145f, cc, 1.0f);
            *slope = fmaf(c * p * q, du, p);
        }
    } else {
        p = logistic<kPrecise, kSlope>(x, &q);
        if constexpr (kSlope) *slope = fmaf(x * p, q, p);
    }
    return p;
}

// ---- the walk over a matrix ------------------------------------------------
//
// A unit is eight columns of one row; a row has 4 units per group, so that
// pads are written too.  A block takes kThreads*U consecutive units whatever
// the rows' length, so that narrow matrices fill their wavefronts as wide ones
// do.

struct Walk {
    uint64_t units;       // rows * per_row
    uint64_t first;       // block of the whole that the launch begins with
    uint64_t magic;       // ceil(2^64 / per_row): row of a unit below 2^32
    uint32_t per_row;     // 4 * ceil(cols / 32)
    uint32_t magic32;     // ceil(2^32 / per_row): rows inside a block
    uint32_t cols;
    uint32_t scale_row;   // bytes between rows of scales
};

inline Walk walk_of(uint64_t rows, uint64_t cols) {
    Walk w;
    w.per_row = (uint32_t)(4 * groups_of(cols));
    w.units = rows * w.per_row;
    w.first = 0;
    w.magic = ~0ull / w.per_row + 1;
    w.magic32 = 0xFFFFFFFFu / w.per_row + 1;
    w.cols = (uint32_t)cols;
    w.scale_row = (uint32_t)scale_stride(cols);
    return w;
}

struct Place {
    uint64_t row;
    uint32_t unit;  // in the row
    int n;          // values inside the matrix, 0..8; -1: no unit
};

template <int U>
__device__ __forceinline__ void places(const Walk& w, Place* at) {
    const uint64_t first = (w.first + blockIdx.x) * (kThreads * U);
    const uint64_t row0 = first >> 32 ? first / w.per_row : __umul64hi(first, w.magic);
    const uint32_t unit0 = (uint32_t)(first - row0 * w.per_row);
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const uint32_t v = unit0 + threadIdx.x + i * kThreads;
        const uint32_t q = w.per_row >= kThreads * U ? (uint32_t)(v >= w.per_row) : __umulhi(v, w.magic32);
        at[i].row = row0 + q;
        at[i].unit = v - q * w.per_row;
        const int left = (int)(w.cols - at[i].unit * 8);
        at[i].n = first + threadIdx.x + i * kThreads < w.units ? min(max(left, 0), 8) : -1;
    }
}

__device__ __forceinline__ void store_codes(uint8_t* codes, uint8_t* scales, const Walk& w, const Place& p, u2 c,
                                            uint32_t byte) {
    if (p.n < 0) return;
    __builtin_nontemporal_store(c, reinterpret_cast<u2*>(codes + (p.row * w.per_row + p.unit) * 8));
    if ((p.unit & 3) == 0) scales[p.row * w.scale_row + p.unit / 4] = (uint8_t)byte;
    // the scales' own pads, at the end of the row
    if (p.unit == w.per_row - 1)
        for (uint32_t g = w.per_row / 4; g < w.scale_row; ++g) scales[p.row * w.scale_row + g] = 0;
}

__device__ __forceinline__ void load_codes(const uint8_t* codes, const uint8_t* scales, const Walk& w, const Place& p,
                                           u2* c, uint32_t* byte) {
    *c = u2{0, 0};
    *byte = 0;
    if (p.n <= 0) return;
    *c = __builtin_nontemporal_load(reinterpret_cast<const u2*>(codes + (p.row * w.per_row + p.unit) * 8));
    *byte = scales[p.row * w.scale_row + p.unit / 4];
}

// Pack a matrix (kInputs 0), or apply the activation function A and pack its
// one or two inputs in the same pass.
template <typename T, int FMT, int A, int kInputs>
__global__ __launch_bounds__(kThreads) void k_act(Walk w, const typename T::Elem* a, uint64_t a_stride,
                                                  const typename T::Elem* b, uint64_t b_stride, typename T::Elem* y,
                                                  uint64_t y_stride, uint8_t* __restrict__ a_codes,
                                                  uint8_t* __restrict__ a_scales, uint8_t* __restrict__ b_codes,
                                                  uint8_t* __restrict__ b_scales) {
    constexpr int U = 2;
    constexpr bool kPrecise = T::kTerms == 3;
    Place at[U];
    places<U>(w, at);
    Raw8<T> ra[U], rb[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        ra[i] = load8<T, kInputs == 0>(a + at[i].row * a_stride + at[i].unit * 8ull, at[i].n);
        if constexpr (kInputs == 2) rb[i] = load8<T>(b + at[i].row * b_stride + at[i].unit * 8ull, at[i].n);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        float va[8], vb[8];
        unpack8<T>(ra[i], va);
        uint32_t byte = scale_byte<FMT>(max_of_group(amax8(va)));
        store_codes(a_codes, a_scales, w, at[i], encode8<FMT>(va, byte), byte);
        if constexpr (kInputs == 2) {
            unpack8<T>(rb[i], vb);
            byte = scale_byte<FMT>(max_of_group(amax8(vb)));
            store_codes(b_codes, b_scales, w, at[i], encode8<FMT>(vb, byte), byte);
        }
        if constexpr (kInputs >= 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float f = va[j] * act_p<A, kPrecise, false>(va[j], nullptr);
                va[j] = kInputs == 2 ? f * vb[j] : f;
            }
            if (at[i].n > 0) store8<T>(y + at[i].row * y_stride + at[i].unit * 8ull, at[i].n, pack8<T>(va));
        }
    }
}

template <typename T, int FMT>
__global__ __launch_bounds__(kThreads) void k_unpack(Walk w, const uint8_t* __restrict__ codes,
                                                     const uint8_t* __restrict__ scales,
                                                     typename T::Elem* __restrict__ y, uint64_t y_stride) {
    constexpr int U = 2;  // 32768x4096 to bf16: 66 us, 68 with four, 72 with eight
    Place at[U];
    places<U>(w, at);
    u2 c[U];
    uint32_t byte[U];
#pragma unroll
    for (int i = 0; i < U; ++i) load_codes(codes, scales, w, at[i], &c[i], &byte[i]);
#pragma unroll
    for (int i = 0; i < U; ++i) {
        float v[8];
        decode8<FMT>(c[i], byte[i], v);
        if (at[i].n > 0) store8<T>(y + at[i].row * y_stride + at[i].unit * 8ull, at[i].n, pack8<T>(v));
    }
}

// The gradient of y = f(a) or f(a)*b from the checkpoints of a and b:
// da = dy*f'(a)(*b), db = dy*f(a), and if wanted the checkpoint of y again.
template <typename T, int FMT, int A, bool kGated>
__global__ __launch_bounds__(kThreads) void k_act_grad(
    Walk w, const uint8_t* __restrict__ a_codes, const uint8_t* __restrict__ a_scales,
    const uint8_t* __restrict__ b_codes, const uint8_t* __restrict__ b_scales, const typename T::Elem* dy,
    uint64_t dy_stride, typename T::Elem* da, uint64_t da_stride, typename T::Elem* db, uint64_t db_stride,
    uint8_t* __restrict__ y_codes, uint8_t* __restrict__ y_scales) {
    // two checkpoints are enough under way with one unit a lane (16384x8192: 208 -> 197 us)
    constexpr int U = kGated ? 1 : 2;
    constexpr bool kPrecise = T::kTerms == 3;
    Place at[U];
    places<U>(w, at);
    u2 ca[U], cb[U];
    uint32_t ea[U], eb[U];
    Raw8<T> rd[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        load_codes(a_codes, a_scales, w, at[i], &ca[i], &ea[i]);
        if constexpr (kGated) load_codes(b_codes, b_scales, w, at[i], &cb[i], &eb[i]);
        rd[i] = load8<T, true>(dy + at[i].row * dy_stride + at[i].unit * 8ull, at[i].n);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        float va[8], vb[8], vd[8], vy[8];
        decode8<FMT>(ca[i], ea[i], va);
        if constexpr (kGated) decode8<FMT>(cb[i], eb[i], vb);
        unpack8<T>(rd[i], vd);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float slope;
            const float f = va[j] * act_p<A, kPrecise, true>(va[j], &slope);
            if constexpr (kGated) {
                vy[j] = f * vb[j];
                va[j] = vd[j] * vb[j] * slope;
                vb[j] = vd[j] * f;
            } else {
                vy[j] = f;
                va[j] = vd[j] * slope;
            }
        }
        if (at[i].n > 0) {
            store8<T>(da + at[i].row * da_stride + at[i].unit * 8ull, at[i].n, pack8<T>(va));
            if constexpr (kGated) store8<T>(db + at[i].row * db_stride + at[i].unit * 8ull, at[i].n, pack8<T>(vb));
        }
        if (y_codes) {
            const uint32_t byte = scale_byte<FMT>(max_of_group(amax8(vy)));
            store_codes(y_codes, y_scales, w, at[i], encode8<FMT>(vy, byte), byte);
        }
    }
}

// ---- root-mean-square norm -------------------------------------------------
//
// sum = x + residual, rounded to the type (what the next layer and the
// backward pass see); rstd = (mean(sum^2) + eps)^(-1/2); n = sum*rstd; y = n*w.
// A row stays in registers between the sum of its squares and its output:
// `waves` wavefronts of one block hold it, kVec units a lane.  A code is the
// nearest one to the value in 64 bits: squares, their sum, rstd and the product
// with it are fp64 (as fast a multiply-add as fp32 on this chip, and hidden
// behind 9 bytes moved per value), so codes next to a border do not depend on
// the order of the sum.

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// The sum of v over the `waves` wavefronts of a row.  Every thread of the
// block comes here; sm holds one value per wavefront and is free again after
// the next barrier.
template <typename S>
__device__ __forceinline__ S row_sum(S v, int waves, S* sm) {
    v = wave_sum(v);
    if (waves == 1) return v;
    const int wave = threadIdx.x >> 6, first = wave / waves * waves;
    if ((threadIdx.x & 63) == 0) sm[wave] = v;
    __syncthreads();
    S t = sm[first];
    for (int k = 1; k < waves; ++k) t += sm[first + k];
    return t;
}

// fp64 to the nearest e4m3 through fp32: the fp32 number is the value cut
// after 21 bits with its last bit set if anything was cut off, which the
// second rounding (to 4 bits) cannot take for a tie.
__device__ __forceinline__ float cut_odd(double v) {
    // below 2^-20 every code is 0; the bound keeps the exponent in fp32's range
    const uint64_t u = __builtin_bit_cast(uint64_t, fmax(fabs(v), 0x1p-20));
    const uint32_t sign = (uint32_t)(__builtin_bit_cast(uint64_t, v) >> 32) & 0x80000000u;
    const uint32_t mag = ((uint32_t)(u >> 32) << 3 | (uint32_t)((uint32_t)u != 0)) - (896u << 23);
    return from_bits(mag | sign);
}

template <int FMT>
__device__ __forceinline__ u2 encode8_64(const double* v, double factor, uint32_t byte) {
    if (byte == 255) return u2{0, 0};
    u2 r;
    if constexpr (FMT == TLC_CKPT8_INT8) {
        uint32_t q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const double t = fma(v[j], factor, 6755399441055744.0);  // 1.5*2^52: an integer in the low bits
            q[j] = (uint32_t)__builtin_bit_cast(uint64_t, t);
        }
        r.x = low_bytes(q[0], q[1], q[2], q[3]);
        r.y = low_bytes(q[4], q[5], q[6], q[7]);
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = cut_odd(v[4 * j + k] * factor);
            uint32_t t = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
            r[j] = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], t, true);
        }
    }
    return r;
}

struct NormArgs {
    const void *x, *residual;
    uint64_t x_stride, residual_stride;
    void *sum, *y;
    uint64_t sum_stride, y_stride;
    const void* weight;
    int weighted;
    double eps;
    uint8_t *codes, *scales;
    float* rstd;
    uint64_t rows;
    uint64_t first;                   // block of the whole that the launch begins with
    uint32_t cols, units, scale_row;  // units of a row, pads among them
    int waves;
};

template <typename T, typename W, int FMT, int kVec>
__global__ __launch_bounds__(1024) void k_norm(NormArgs p) {
    using Elem = typename T::Elem;
    __shared__ double sm[16];
    const int wave = threadIdx.x >> 6, rows_here = max(1, (int)(blockDim.x >> 6) / p.waves);
    const uint64_t row = (p.first + blockIdx.x) * rows_here + wave / p.waves;
    const bool live = row < p.rows;
    const uint32_t lane = (wave % p.waves) * 64 + (threadIdx.x & 63), lanes = p.waves * 64;
    float v[kVec][8];
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const uint32_t unit = lane + i * lanes;
        const int n = live && unit < p.units ? min(max((int)p.cols - (int)unit * 8, 0), 8) : 0;
        unpack8<T>(load8<T>(static_cast<const Elem*>(p.x) + row * p.x_stride + unit * 8ull, n), v[i]);
        if (p.residual) {
            float r[8];
            unpack8<T>(load8<T>(static_cast<const Elem*>(p.residual) + row * p.residual_stride + unit * 8ull, n), r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] += r[j];
            const Raw8<T> t = pack8<T>(v[i]);
            if (p.sum && n > 0) store8<T>(static_cast<Elem*>(p.sum) + row * p.sum_stride + unit * 8ull, n, t);
            unpack8<T>(t, v[i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fma((double)v[i][j], (double)v[i][j], ss);
    }
    ss = row_sum(ss, p.waves, sm);
    const double rstd = 1.0 / sqrt(ss / (double)p.cols + p.eps);
    const float rstd32 = (float)rstd;
    if (p.rstd && live && lane == 0) p.rstd[row] = rstd32;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const uint32_t unit = lane + i * lanes;
        const int n = live && unit < p.units ? min(max((int)p.cols - (int)unit * 8, 0), 8) : 0;
        float w[8];
        if (p.weight) unpack8<W>(load8<W>(static_cast<const typename W::Elem*>(p.weight) + unit * 8ull, n), w);
        if (p.codes) {
            double d[8], amax;
            uint32_t byte;
            if (p.weight && p.weighted) {
                double bad = 0.0;
                amax = 0.0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    d[j] = (double)v[i][j] * rstd * (double)w[j];
                    amax = fmax(amax, fabs(d[j]));
                    bad = fma(d[j], 0.0, bad);  // NaN once a value is not finite
                }
                if (bad != bad) amax = bad;
                // NaN's bits lie above every number's
                uint64_t m = __builtin_bit_cast(uint64_t, amax) & 0x7FFFFFFFFFFFFFFFull;
                m = max(m, (uint64_t)__shfl_xor((unsigned long long)m, 1, 64));
                m = max(m, (uint64_t)__shfl_xor((unsigned long long)m, 2, 64));
                byte = scale_byte64<FMT>(__builtin_bit_cast(double, m));
                if (byte == (uint32_t)Format<FMT>::kHigh) {
                    const double top = (double)Format<FMT>::kMax * (double)scale_of(byte);
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[j] = fmin(fmax(d[j], -top), top);
                }
            } else {
                amax = (double)from_bits(max_of_group(amax8(v[i]))) * rstd;
                byte = scale_byte64<FMT>(amax);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = (double)v[i][j] * rstd;
            }
            const u2 c = encode8_64<FMT>(d, (double)inverse_scale(byte), byte);
            if (live && unit < p.units) {
                __builtin_nontemporal_store(c, reinterpret_cast<u2*>(p.codes + (row * p.units + unit) * 8));
                if ((unit & 3) == 0) p.scales[row * p.scale_row + unit / 4] = (uint8_t)byte;
                if (unit == p.units - 1)
                    for (uint32_t g = p.units / 4; g < p.scale_row; ++g) p.scales[row * p.scale_row + g] = 0;
            }
        }
        if (p.y && n > 0) {
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (T::kTerms == 3) {  // one rounding
                    const double n = (double)v[i][j] * rstd;
                    o[j] = (float)(p.weight ? n * (double)w[j] : n);
                } else {  // 3 * 2^-24 beside the type's own rounding (16384x4096 bf16 100 us, 105 in 64 bits)
                    o[j] = v[i][j] * rstd32;
                    if (p.weight) o[j] *= w[j];
                }
            }
            store8<T>(static_cast<Elem*>(p.y) + row * p.y_stride + unit * 8ull, n, pack8<T>(o));
        }
    }
}

// Gradient of the norm (FMT 0: from the sum): with n the normalised row (from its checkpoint, or
// sum*rstd) and g = dy*w,
//   dx = dsum + rstd*(g - n*mean(g*n)),   dw = sum over rows of dy*n.
// A block walks over rows block, block + grid, ..., the next row's values on
// their way while one is worked on; a lane keeps the dw of its columns in
// registers.  The block's rows of them are added through LDS and written once,
// as one row of `partial`, which k_norm_dw adds in order: the same bits every
// run, no atomics.
struct NormGradArgs {
    const void *dy, *dsum, *sum;
    uint64_t dy_stride, dsum_stride, sum_stride;
    const uint8_t *codes, *scales;
    const void* weight;
    const float* rstd;
    void* dx;
    uint64_t dx_stride;
    float* partial;  // [blocks][cols], or nullptr
    uint64_t rows;
    uint32_t cols, units, scale_row;
    int waves;
};

template <typename T, typename W, int FMT, int kVec>
__global__ __launch_bounds__(1024) void k_norm_grad(NormGradArgs p) {
    using Elem = typename T::Elem;
    __shared__ float sm[2][16];
    __shared__ float sdw[kThreads * 8];  // of 4 wavefronts with 8 columns a lane at a time
    const int wave = threadIdx.x >> 6, rows_here = max(1, (int)(blockDim.x >> 6) / p.waves);
    const uint32_t lane = (wave % p.waves) * 64 + (threadIdx.x & 63), lanes = p.waves * 64;
    constexpr bool kCodes = FMT != 0;
    struct Row {
        Raw8<T> dy[kVec], add[kVec], sum[kCodes ? 1 : kVec];  // dy, dsum and the sum, or instead of it:
        u2 codes[kCodes ? kVec : 1];
        uint32_t byte[kCodes ? kVec : 1];
        float rstd;
    };
    const auto count = [&](int i) {
        const uint32_t unit = lane + i * lanes;
        return unit < p.units ? min(max((int)p.cols - (int)unit * 8, 0), 8) : 0;
    };
    const auto load = [&](Row& r, uint64_t row) {
        const bool live = row < p.rows;
        r.rstd = live ? p.rstd[row] : 0.0f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const uint32_t unit = lane + i * lanes;
            const int n = live ? count(i) : 0;
            r.dy[i] = load8<T, true>(static_cast<const Elem*>(p.dy) + row * p.dy_stride + unit * 8ull, n);
            r.add[i] = load8<T, true>(static_cast<const Elem*>(p.dsum) + row * p.dsum_stride + unit * 8ull,
                                      p.dsum ? n : 0);
            if constexpr (kCodes) {
                r.codes[i] = u2{0, 0};
                r.byte[i] = 0;
                if (n > 0) {
                    r.codes[i] =
                        __builtin_nontemporal_load(reinterpret_cast<const u2*>(p.codes + (row * p.units + unit) * 8));
                    r.byte[i] = p.scales[row * p.scale_row + unit / 4];
                }
            } else {
                r.sum[i] = load8<T, true>(static_cast<const Elem*>(p.sum) + row * p.sum_stride + unit * 8ull, n);
            }
        }
    };
    float w[kVec][8], dw[kVec][8];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        if (p.weight)
            unpack8<W>(load8<W>(static_cast<const typename W::Elem*>(p.weight) + (lane + i * lanes) * 8ull, count(i)),
                       w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!p.weight) w[i][j] = 1.0f;
            dw[i][j] = 0.0f;
        }
    }
    int turn = 0;
    Row now, next;
    const uint64_t stride = (uint64_t)gridDim.x * rows_here;
    uint64_t base = (uint64_t)blockIdx.x * rows_here;
    // Two units a lane do not fit the 128 registers of a 1024-thread block with
    // the next row (and without it 3 of them, 9 to 12 in fp32, go through
    // scratch): 4096x16384 bf16 takes 108 us, 4.4 TB/s, where 16384x4096 takes 91.
    constexpr bool kAhead = kVec == 1;
    if constexpr (kAhead) load(now, base + wave / p.waves);
    // every wavefront of a block makes the same turns: barriers lie inside
    for (; base < p.rows; base += stride) {
        const uint64_t row = base + wave / p.waves;
        const bool live = row < p.rows;
        if constexpr (kAhead)
            load(next, row + stride);
        else
            load(now, row);
        float g[kVec][8], nv[kVec][8], dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int n = count(i);
            unpack8<T>(now.dy[i], g[i]);
            if constexpr (kCodes) {
                decode8<FMT>(now.codes[i], now.byte[i], nv[i]);
            } else {
                unpack8<T>(now.sum[i], nv[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) nv[i][j] *= now.rstd;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j < n) dw[i][j] = fmaf(g[i][j], nv[i][j], dw[i][j]);
                g[i][j] *= w[i][j];
                if (j < n) dot = fmaf(g[i][j], nv[i][j], dot);
            }
        }
        dot = row_sum(dot, p.waves, sm[turn]);
        turn ^= 1;  // the other half is read until the next barrier
        const float mean = dot / (float)p.cols;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int n = live ? count(i) : 0;
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = now.rstd * (g[i][j] - nv[i][j] * mean);
            float d[8];
            unpack8<T>(now.add[i], d);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] += d[j];
            if (n > 0)
                store8<T>(static_cast<Elem*>(p.dx) + row * p.dx_stride + (lane + i * lanes) * 8ull, n, pack8<T>(o));
        }
        if constexpr (kAhead) now = next;
    }
    if (!p.partial) return;
    float* const out = p.partial + (uint64_t)blockIdx.x * p.cols;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        if (rows_here > 1) {  // waves of 1 or 2: the block's rows add up, in order
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) sdw[(j * rows_here + wave / p.waves) * lanes + lane] = dw[i][j];
            __syncthreads();
            if (wave / p.waves == 0)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    for (int r = 1; r < rows_here; ++r) dw[i][j] += sdw[(j * rows_here + r) * lanes + lane];
        }
        const int n = count(i);
        if (n > 0 && wave / p.waves == 0) store8<F32>(out + (lane + i * lanes) * 8ull, n, pack8<F32>(dw[i]));
    }
}

// dw[c] (+)= sum over the partial rows, in order: 32 strips of rows per block,
// each added by one lane per column with four loads under way, then the strips.
constexpr int kStrips = 32;
__global__ __launch_bounds__(32 * kStrips) void k_norm_dw(const float* __restrict__ partial, uint32_t parts,
                                                          uint32_t cols, float* dw, int accumulate) {
    __shared__ float sm[kStrips][32];
    const uint32_t c = blockIdx.x * 32 + (threadIdx.x & 31), strip = threadIdx.x >> 5;
    float s = 0.0f;
    if (c < cols) {
        uint32_t r = strip;
        for (; r + 3 * kStrips < parts; r += 4 * kStrips) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = partial[(uint64_t)(r + k * kStrips) * cols + c];
#pragma unroll
            for (int k = 0; k < 4; ++k) s += v[k];
        }
        for (; r < parts; r += kStrips) s += partial[(uint64_t)r * cols + c];
    }
    sm[strip][threadIdx.x & 31] = s;
    __syncthreads();
    if (strip || c >= cols) return;
#pragma unroll
    for (int k = 1; k < kStrips; ++k) s += sm[k][threadIdx.x & 31];
    dw[c] = accumulate ? dw[c] + s : s;
}

// ---- host ------------------------------------------------------------------

constexpr uint64_t kNormMaxCols = 16384;  // 16 wavefronts of 2 units a lane

struct NormShape {
    int waves, vec, threads;
    uint32_t rows_here;
};
// Wavefronts of a row are a power of two, so that a block holds whole rows: a
// row that fills them badly (128 columns a quarter of a wavefront, 5000 columns
// 10 of 16) leaves lanes without a unit.
NormShape norm_shape(uint64_t cols) {
    const uint64_t units = 4 * groups_of(cols);
    NormShape s;
    // a unit a lane up to 8192 columns, two past them
    s.vec = units <= 16 * 64 ? 1 : 2;
    s.waves = 1;
    while ((uint64_t)s.waves * 64 * s.vec < units) s.waves *= 2;
    s.threads = std::max(kThreads, s.waves * 64);
    s.rows_here = (uint32_t)(s.threads / 64 / s.waves);
    return s;
}
// Blocks of the gradient: two rows a wavefront at least, so that the partial
// sums stay below what they sum.
constexpr uint64_t kNormGradBlocks = 512;
uint64_t norm_grad_blocks(uint64_t rows, const NormShape& s) {
    return std::min<uint64_t>((rows + 2 * s.rows_here - 1) / (2 * s.rows_here), kNormGradBlocks);
}

template <typename Fn>
int with_vec(int vec, Fn&& fn) {
    return vec == 1 ? fn(Int<1>{}) : fn(Int<2>{});
}

template <typename Fn>
int with_saved(int format, Fn&& fn) {
    return format ? with_format(format, fn) : fn(Int<0>{});
}

// Launches a kernel over a walk with `per_lane` units a lane: fn(walk, blocks).
template <typename Fn>
int launch_walk(const char* name, hipStream_t st, Walk w, uint64_t per_lane, Fn&& fn) {
    const uint64_t per_block = kThreads * per_lane;
    return launch_blocks(name, st, (w.units + per_block - 1) / per_block, kThreads,
                         [&](uint64_t first, uint32_t blocks) {
                             w.first = first;
                             fn(w, blocks);
                         });
}

template <typename Fn>
int with_act(int act, Fn&& fn) {
    return act == TLC_ACT_GELU        ? fn(Int<TLC_ACT_GELU>{})
           : act == TLC_ACT_GELU_TANH ? fn(Int<TLC_ACT_GELU_TANH>{})
                                      : fn(Int<TLC_ACT_SILU>{});
}
bool valid_act(int a) { return a == TLC_ACT_GELU || a == TLC_ACT_GELU_TANH || a == TLC_ACT_SILU; }

int run_act(int inputs, int act, const void* a, uint64_t a_stride, const void* b, uint64_t b_stride, int dtype,
            uint64_t rows, uint64_t cols, void* y, uint64_t y_stride, int format, uint8_t* a_codes, uint8_t* a_scales,
            uint8_t* b_codes, uint8_t* b_scales, hipStream_t st) {
    if (!valid_dtype(dtype) || !valid_format(format) || !valid_shape(rows, cols) || (inputs >= 1 && !valid_act(act)))
        return TLC_ERR_INVALID_ARG;
    if (rows == 0) return TLC_OK;
    if (!valid_matrix(a, dtype, cols, a_stride) || !valid_checkpoint(a_codes, a_scales)) return TLC_ERR_INVALID_ARG;
    if (inputs >= 1 && !valid_matrix(y, dtype, cols, y_stride)) return TLC_ERR_INVALID_ARG;
    if (inputs == 2 && (!valid_matrix(b, dtype, cols, b_stride) || !valid_checkpoint(b_codes, b_scales)))
        return TLC_ERR_INVALID_ARG;
    const Walk walk = walk_of(rows, cols);
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        using E = typename T::Elem;
        return with_format(format, [&](auto f) {
            constexpr int F = decltype(f)::value;
            const E* const pa = static_cast<const E*>(a);
            const E* const pb = static_cast<const E*>(b);
            E* const py = static_cast<E*>(y);
            if (inputs == 0)
                return launch_walk("tlc_ckpt8_pack", st, walk, 2, [&](const Walk& w, uint32_t blocks) {
                    k_act<T, F, TLC_ACT_SILU, 0><<<blocks, kThreads, 0, st>>>(w, pa, a_stride, nullptr, 0, nullptr, 0,
                                                                             a_codes, a_scales, nullptr, nullptr);
                });
            return with_act(act, [&](auto k) {
                constexpr int A = decltype(k)::value;
                return launch_walk("tlc_ckpt8_act", st, walk, 2, [&](const Walk& w, uint32_t blocks) {
                    if (inputs == 1)
                        k_act<T, F, A, 1><<<blocks, kThreads, 0, st>>>(w, pa, a_stride, nullptr, 0, py, y_stride,
                                                                       a_codes, a_scales, nullptr, nullptr);
                    else
                        k_act<T, F, A, 2><<<blocks, kThreads, 0, st>>>(w, pa, a_stride, pb, b_stride, py, y_stride,
                                                                       a_codes, a_scales, b_codes, b_scales);
                });
            });
        });
    });
}

}  // namespace

extern "C" {

uint64_t tlc_ckpt8_code_stride(uint64_t cols) { return cols >= 1 && cols <= kMaxDim ? code_stride(cols) : 0; }
uint64_t tlc_ckpt8_scale_stride(uint64_t cols) { return cols >= 1 && cols <= kMaxDim ? scale_stride(cols) : 0; }

int tlc_ckpt8_pack(const void* x, uint64_t x_stride, int dtype, uint64_t rows, uint64_t cols, int format,
                   uint8_t* codes, uint8_t* scales, tlc_stream_t stream) {
    return run_act(0, 0, x, x_stride, nullptr, 0, dtype, rows, cols, nullptr, 0, format, codes, scales, nullptr,
                   nullptr, static_cast<hipStream_t>(stream));
}

int tlc_ckpt8_unpack(const uint8_t* codes, const uint8_t* scales, int format, uint64_t rows, uint64_t cols, void* y,
                     uint64_t y_stride, int dtype, tlc_stream_t stream) {
    if (!valid_dtype(dtype) || !valid_format(format) || !valid_shape(rows, cols)) return TLC_ERR_INVALID_ARG;
    if (rows == 0) return TLC_OK;
    if (!valid_matrix(y, dtype, cols, y_stride) || !valid_checkpoint(codes, scales)) return TLC_ERR_INVALID_ARG;
    const Walk walk = walk_of(rows, cols);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        return with_format(format, [&](auto f) {
            return launch_walk("tlc_ckpt8_unpack", st, walk, 2, [&](const Walk& w, uint32_t blocks) {
                k_unpack<T, decltype(f)::value>
                    <<<blocks, kThreads, 0, st>>>(w, codes, scales, static_cast<typename T::Elem*>(y), y_stride);
            });
        });
    });
}

int tlc_ckpt8_act(int act, const void* a, uint64_t a_stride, const void* b, uint64_t b_stride, int dtype,
                  uint64_t rows, uint64_t cols, void* y, uint64_t y_stride, int format, uint8_t* a_codes,
                  uint8_t* a_scales, uint8_t* b_codes, uint8_t* b_scales, tlc_stream_t stream) {
    if (!b && (b_codes || b_scales)) return TLC_ERR_INVALID_ARG;
    return run_act(b ? 2 : 1, act, a, a_stride, b, b_stride, dtype, rows, cols, y, y_stride, format, a_codes, a_scales,
                   b_codes, b_scales, static_cast<hipStream_t>(stream));
}

int tlc_ckpt8_act_grad(int act, const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                       const uint8_t* b_scales, int format, const void* dy, uint64_t dy_stride, int dtype,
                       uint64_t rows, uint64_t cols, void* da, uint64_t da_stride, void* db, uint64_t db_stride,
                       uint8_t* y_codes, uint8_t* y_scales, tlc_stream_t stream) {
    const bool gated = b_codes || b_scales || db;
    if (!valid_act(act) || !valid_dtype(dtype) || !valid_format(format) || !valid_shape(rows, cols))
        return TLC_ERR_INVALID_ARG;
    if (rows == 0) return TLC_OK;
    if (!valid_matrix(dy, dtype, cols, dy_stride) || !valid_matrix(da, dtype, cols, da_stride) ||
        !valid_checkpoint(a_codes, a_scales))
        return TLC_ERR_INVALID_ARG;
    if (gated && (!valid_matrix(db, dtype, cols, db_stride) || !valid_checkpoint(b_codes, b_scales)))
        return TLC_ERR_INVALID_ARG;
    if ((y_codes || y_scales) && !valid_checkpoint(y_codes, y_scales)) return TLC_ERR_INVALID_ARG;
    const Walk walk = walk_of(rows, cols);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        using E = typename T::Elem;
        return with_format(format, [&](auto f) {
            constexpr int F = decltype(f)::value;
            return with_act(act, [&](auto k) {
                constexpr int A = decltype(k)::value;
                return launch_walk("tlc_ckpt8_act_grad", st, walk, gated ? 1 : 2, [&](const Walk& w, uint32_t blocks) {
                    if (gated)
                        k_act_grad<T, F, A, true><<<blocks, kThreads, 0, st>>>(
                            w, a_codes, a_scales, b_codes, b_scales, static_cast<const E*>(dy), dy_stride,
                            static_cast<E*>(da), da_stride, static_cast<E*>(db), db_stride, y_codes, y_scales);
                    else
                        k_act_grad<T, F, A, false><<<blocks, kThreads, 0, st>>>(
                            w, a_codes, a_scales, nullptr, nullptr, static_cast<const E*>(dy), dy_stride,
                            static_cast<E*>(da), da_stride, nullptr, 0, y_codes, y_scales);
                });
            });
        });
    });
}

int tlc_ckpt8_norm(const void* x, uint64_t x_stride, const void* residual, uint64_t residual_stride, int dtype,
                   uint64_t rows, uint64_t cols, const void* weight, int weight_dtype, float eps, int weighted,
                   void* sum, uint64_t sum_stride, void* y, uint64_t y_stride, int format, uint8_t* codes,
                   uint8_t* scales, float* rstd, tlc_stream_t stream) {
    if (!valid_dtype(dtype) || !valid_shape(rows, cols) || cols > kNormMaxCols || !(eps > 0.0f) ||
        !(eps < __builtin_inff()) || !valid_weight(weight, weight_dtype, dtype) || (weighted && !weight))
        return TLC_ERR_INVALID_ARG;
    if (rows == 0) return TLC_OK;
    if (!valid_matrix(x, dtype, cols, x_stride)) return TLC_ERR_INVALID_ARG;
    if (residual && !valid_matrix(residual, dtype, cols, residual_stride)) return TLC_ERR_INVALID_ARG;
    if (sum && (!residual || !valid_matrix(sum, dtype, cols, sum_stride))) return TLC_ERR_INVALID_ARG;
    if (y && !valid_matrix(y, dtype, cols, y_stride)) return TLC_ERR_INVALID_ARG;
    if ((codes || scales) && (!valid_format(format) || !valid_checkpoint(codes, scales))) return TLC_ERR_INVALID_ARG;
    if (!y && !codes) return TLC_ERR_INVALID_ARG;
    if (rstd && !aligned(rstd, 4)) return TLC_ERR_INVALID_ARG;
    const NormShape s = norm_shape(cols);
    NormArgs p;
    p.x = x, p.residual = residual, p.x_stride = x_stride, p.residual_stride = residual_stride;
    p.sum = sum, p.y = y, p.sum_stride = sum_stride, p.y_stride = y_stride;
    p.weight = weight, p.weighted = weighted != 0, p.eps = (double)eps;
    p.codes = codes, p.scales = scales, p.rstd = rstd, p.rows = rows;
    p.cols = (uint32_t)cols, p.units = (uint32_t)(4 * groups_of(cols)), p.scale_row = (uint32_t)scale_stride(cols);
    p.waves = s.waves;
    const uint64_t all = (rows + s.rows_here - 1) / s.rows_here;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return with_dtype(dtype, [&](auto t) {
        return with_weight(t, weight, weight_dtype, [&](auto w) {
            return with_format(format, [&](auto f) {
                return with_vec(s.vec, [&](auto v) {
                    return launch_blocks("tlc_ckpt8_norm", st, all, s.threads, [&](uint64_t first, uint32_t blocks) {
                        p.first = first;
                        k_norm<decltype(t), decltype(w), decltype(f)::value, decltype(v)::value>
                            <<<blocks, s.threads, 0, st>>>(p);
                    });
                });
            });
        });
    });
}

size_t tlc_ckpt8_norm_grad_workspace_size(uint64_t rows, uint64_t cols) {
    if (!valid_shape(rows, cols) || cols > kNormMaxCols) return 0;
    const NormShape s = norm_shape(cols);
    return std::max<size_t>((norm_grad_blocks(rows, s) * cols * sizeof(float) + 255) / 256 * 256, 256);
}

int tlc_ckpt8_norm_grad(const void* dy, uint64_t dy_stride, const void* dsum, uint64_t dsum_stride, int dtype,
                        uint64_t rows, uint64_t cols, const void* sum, uint64_t sum_stride, int format,
                        const uint8_t* codes, const uint8_t* scales, const float* rstd, const void* weight,
                        int weight_dtype, void* dx, uint64_t dx_stride, float* dw, int accumulate, void* workspace,
                        size_t workspace_bytes, tlc_stream_t stream) {
    if (!valid_dtype(dtype) || !valid_shape(rows, cols) || cols > kNormMaxCols ||
        !valid_weight(weight, weight_dtype, dtype))
        return TLC_ERR_INVALID_ARG;
    if (rows) {
        if (!valid_matrix(dy, dtype, cols, dy_stride) || !valid_matrix(dx, dtype, cols, dx_stride) || !rstd ||
            !aligned(rstd, 4))
            return TLC_ERR_INVALID_ARG;
        if (dsum && !valid_matrix(dsum, dtype, cols, dsum_stride)) return TLC_ERR_INVALID_ARG;
        if (codes || scales) {
            if (sum || !valid_format(format) || !valid_checkpoint(codes, scales)) return TLC_ERR_INVALID_ARG;
        } else if (!valid_matrix(sum, dtype, cols, sum_stride)) {
            return TLC_ERR_INVALID_ARG;
        }
    }
    if (dw && !aligned(dw, 4)) return TLC_ERR_INVALID_ARG;
    const size_t need = tlc_ckpt8_norm_grad_workspace_size(rows, cols);
    if (dw && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return TLC_ERR_WORKSPACE;
    const NormShape s = norm_shape(cols);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const uint32_t blocks = (uint32_t)norm_grad_blocks(rows, s);
    float* const partial = dw ? static_cast<float*>(workspace) : nullptr;
    if (rows) {
        NormGradArgs p;
        p.dy = dy, p.dsum = dsum, p.sum = sum;
        p.dy_stride = dy_stride, p.dsum_stride = dsum_stride, p.sum_stride = sum_stride;
        p.codes = codes, p.scales = scales, p.weight = weight, p.rstd = rstd;
        p.dx = dx, p.dx_stride = dx_stride, p.partial = partial, p.rows = rows;
        p.cols = (uint32_t)cols, p.units = (uint32_t)(4 * groups_of(cols));
        p.scale_row = (uint32_t)scale_stride(cols), p.waves = s.waves;
        const int rc = with_dtype(dtype, [&](auto t) {
            return with_weight(t, weight, weight_dtype, [&](auto w) {
                return with_saved(codes ? format : 0, [&](auto f) {
                    return with_vec(s.vec, [&](auto v) {
                        return launch("tlc_ckpt8_norm_grad", st, [&] {
                            k_norm_grad<decltype(t), decltype(w), decltype(f)::value, decltype(v)::value>
                                <<<blocks, s.threads, 0, st>>>(p);
                        });
                    });
                });
            });
        });
        if (rc) return rc;
    }
    if (!dw || (!rows && accumulate)) return TLC_OK;
    return launch("tlc_ckpt8_norm_dw", st, [&] {
        k_norm_dw<<<(uint32_t)((cols + 31) / 32), 32 * kStrips, 0, st>>>(partial, blocks, (uint32_t)cols, dw,
                                                                         accumulate != 0);
    });
}

}  // extern "C"
