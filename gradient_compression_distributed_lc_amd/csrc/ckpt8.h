// ckpt8.h -- device and host helpers of the 8-bit checkpoint operators
// (internal; the public declarations are in include/tlc.h).
//
// A checkpoint keeps a matrix as one byte per value and one power-of-two scale
// per 32 columns of a row.  With amax the largest magnitude of the 32 values
// and C the largest code (127, or 448 in e4m3), the scale is 2^e for the least
// e with amax <= C*2^e, and a code is the nearest one to x*2^-e.  Both
// multiplications by a power of two are exact, so a value code*2^e has at most
// 8 significant bits: it is a bfloat16 number, and the matrix product reads it
// as one without a second rounding.
#ifndef TLC_CKPT8_H
#define TLC_CKPT8_H

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "tlc.h"

namespace tlc_ckpt8 {

typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
// Rows of a matrix start at any element, so 16-byte accesses are only aligned
// to their elements; gfx950 takes them as one access all the same.
typedef u4 u4_at2 __attribute__((aligned(2)));
typedef u4 u4_at4 __attribute__((aligned(4)));

struct F32 {
    using Elem = float;
    static constexpr int kVecs = 2;  // 16-byte accesses for eight values
    static constexpr int kTerms = 3; // bfloat16 numbers whose sum is any value of the type
};
struct F16 {
    using Elem = _Float16;
    static constexpr int kVecs = 1;
    static constexpr int kTerms = 2;
};
struct BF16 {
    using Elem = __bf16;
    static constexpr int kVecs = 1;
    static constexpr int kTerms = 1;
};

__device__ __forceinline__ float from_bits(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ uint32_t to_bits(float f) { return __builtin_bit_cast(uint32_t, f); }

// Eight consecutive values as they lie in memory.
template <typename T>
struct Raw8 {
    u4 w[T::kVecs];
};

// The first n (at most 8) of the eight values at p, the rest 0.  `whole`: n is
// 8 or 0.  kNt: nontemporally.  Measured: reads of what the call alone needs
// gain by it (32768x4096 bf16 packed in 64 us instead of 68, 16384x4096 gelu
// gradient 53 instead of 58); the activation's and the norm's inputs, which the
// kernel before has just written, do not (4096x4096 gelu 16.5 us instead of
// 15.4).
template <typename T, bool kNt = false>
__device__ __forceinline__ Raw8<T> load8(const typename T::Elem* p, int n, bool whole = false) {
    Raw8<T> r = {};
    if (n >= 8) {
        if constexpr (T::kVecs == 2) {
            const u4_at4* const q = reinterpret_cast<const u4_at4*>(p);
            r.w[0] = kNt ? __builtin_nontemporal_load(q) : *q;
            r.w[1] = kNt ? __builtin_nontemporal_load(q + 1) : q[1];
        } else {
            const u4_at2* const q = reinterpret_cast<const u4_at2*>(p);
            r.w[0] = kNt ? __builtin_nontemporal_load(q) : *q;
        }
    } else if (!whole) {
        if constexpr (T::kVecs == 2) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
            for (int j = 0; j < 8; ++j) r.w[j / 4][j % 4] = j < n ? q[j] : 0u;
        } else {
            const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t lo = 2 * j < n ? q[2 * j] : 0u, hi = 2 * j + 1 < n ? q[2 * j + 1] : 0u;
                r.w[0][j] = lo | hi << 16;
            }
        }
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float* v) {
    if constexpr (T::kVecs == 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = from_bits(r.w[j / 4][j % 4]);
    } else if constexpr (T::kTerms == 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = from_bits(r.w[0][j] << 16);
            v[2 * j + 1] = from_bits(r.w[0][j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const h2 h = __builtin_bit_cast(h2, (uint32_t)r.w[0][j]);
            v[2 * j] = (float)h.x;
            v[2 * j + 1] = (float)h.y;
        }
    }
}

// One rounding to the type, to nearest even.
template <typename T>
__device__ __forceinline__ Raw8<T> pack8(const float* v) {
    Raw8<T> r;
    if constexpr (T::kVecs == 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.w[j / 4][j % 4] = to_bits(v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f2 p = {v[2 * j], v[2 * j + 1]};
            if constexpr (T::kTerms == 1)
                r.w[0][j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, b2));
            else
                r.w[0][j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, h2));
        }
    }
    return r;
}

// Results are written once and not read again here: nontemporally (4096x4096
// bf16 gelu 17.4 -> 15.4 us, 16384x4096 norm 112 -> 100).
template <typename T>
__device__ __forceinline__ void store8(typename T::Elem* p, int n, const Raw8<T>& r) {
    if (n >= 8) {
        if constexpr (T::kVecs == 2) {
            __builtin_nontemporal_store(r.w[0], reinterpret_cast<u4_at4*>(p));
            __builtin_nontemporal_store(r.w[1], reinterpret_cast<u4_at4*>(p + 4));
        } else {
            __builtin_nontemporal_store(r.w[0], reinterpret_cast<u4_at2*>(p));
        }
    } else {
        if constexpr (T::kVecs == 2) {
            uint32_t* q = reinterpret_cast<uint32_t*>(p);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) q[j] = r.w[j / 4][j % 4];
        } else {
            uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) q[j] = (uint16_t)(r.w[0][j / 2] >> (16 * (j & 1)));
        }
    }
}

// ---- the format ------------------------------------------------------------

template <int FMT>
struct Format;
template <>
struct Format<TLC_CKPT8_INT8> {
    static constexpr float kMax = 127.0f;           // = 0x1.FCp6
    static constexpr uint32_t kMantMax = 0x7E0000;  // its fraction bits
    static constexpr int kExp = 6;
    static constexpr int kLow = 1, kHigh = 248;     // scale bytes: every value a normal, finite fp32 number
};
template <>
struct Format<TLC_CKPT8_E4M3> {
    static constexpr float kMax = 448.0f;  // = 0x1.Cp8; the least code is 2^-9
    static constexpr uint32_t kMantMax = 0x600000;
    static constexpr int kExp = 8;
    static constexpr int kLow = 10, kHigh = 246;
};

// Scale byte (e + 127) of a group whose largest magnitude has these bits: the
// addition carries into the exponent exactly where the fraction is above C's.
// 0: all values 0.  255: a value is not finite (NaN compares as the largest).
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    using F = Format<FMT>;
    if (amax_bits == 0) return 0;
    if (amax_bits >= 0x7F800000u) return 255;
    const int b = (int)((amax_bits + (0x7FFFFFu - F::kMantMax)) >> 23) - F::kExp;
    return (uint32_t)min(max(b, F::kLow), F::kHigh);
}
// The same for a magnitude in 64 bits.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte64(double amax) {
    using F = Format<FMT>;
    const uint64_t u = __builtin_bit_cast(uint64_t, amax) & 0x7FFFFFFFFFFFFFFFull;
    if (u == 0) return 0;
    if (u >= 0x7FF0000000000000ull) return 255;
    const int b = (int)((u + (((uint64_t)(0x7FFFFFu - F::kMantMax) << 29) | 0x1FFFFFFFull)) >> 52) - 896 - F::kExp;
    return (uint32_t)min(max(b, F::kLow), F::kHigh);
}

// 2^e of a byte, with 0 for 0 and infinity for 255 (times its codes, 0: NaN).
__device__ __forceinline__ float scale_of(uint32_t byte) { return from_bits(byte << 23); }
// 2^-e, exact for the bytes scale_byte gives.
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return from_bits((254u - byte) << 23); }

__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x0C0C0400u), cd = __builtin_amdgcn_perm(d, c, 0x04000C0Cu);
    return ab | cd;
}

// Codes of eight values of a group with this scale byte.
template <int FMT>
__device__ __forceinline__ u2 encode8(const float* x, uint32_t byte) {
    using F = Format<FMT>;
    if (byte == 255) return u2{0, 0};
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = x[j];
    if (byte == F::kHigh) {  // the largest scale: what lies above its codes is held to the largest
        const float top = F::kMax * scale_of(F::kHigh);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = fminf(fmaxf(v[j], -top), top);
    }
    const float inv = inverse_scale(byte);
    u2 r;
    if constexpr (FMT == TLC_CKPT8_INT8) {
        // 1.5*2^23 + q rounds q = v*2^-e to an integer, to nearest even, and
        // holds it in its low byte; v*2^-e itself is exact
        uint32_t q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = to_bits(fmaf(v[j], inv, 12582912.0f));
        r.x = low_bytes(q[0], q[1], q[2], q[3]);
        r.y = low_bytes(q[4], q[5], q[6], q[7]);
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j] * inv, v[4 * j + 1] * inv, 0, false);
            r[j] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j + 2] * inv, v[4 * j + 3] * inv, w, true);
        }
    }
    return r;
}

template <int FMT>
__device__ __forceinline__ void decode8(u2 codes, uint32_t byte, float* v) {
    const float s = scale_of(byte);
    if constexpr (FMT == TLC_CKPT8_INT8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (float)(int8_t)(codes[j / 4] >> (8 * (j & 3))) * s;
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8(codes[j], false);
            const f2 b = __builtin_amdgcn_cvt_pk_f32_fp8(codes[j], true);
            v[4 * j] = a.x * s;
            v[4 * j + 1] = a.y * s;
            v[4 * j + 2] = b.x * s;
            v[4 * j + 3] = b.y * s;
        }
    }
}

// Bits of the largest magnitude of eight values; integer order puts infinity
// and then NaN above every finite value.
__device__ __forceinline__ uint32_t amax8(const float* v) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, to_bits(v[j]) & 0x7FFFFFFFu);
    return m;
}
// The largest over the four lanes that hold a group (lanes 4k .. 4k+3).
__device__ __forceinline__ uint32_t max_of_group(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));  // lane ^ 1
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));  // lane ^ 2
}

// ---- host ------------------------------------------------------------------

constexpr uint64_t kMaxDim = 0x7FFFFFFFull;  // rows, columns and row strides
inline uint64_t groups_of(uint64_t cols) { return (cols + 31) / 32; }
inline uint64_t code_stride(uint64_t cols) { return 32 * groups_of(cols); }
inline uint64_t scale_stride(uint64_t cols) { return (groups_of(cols) + 3) / 4 * 4; }

inline bool valid_dtype(int t) { return t == TLC_F32 || t == TLC_F16 || t == TLC_BF16; }
inline bool valid_format(int f) { return f == TLC_CKPT8_INT8 || f == TLC_CKPT8_E4M3; }
inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
inline bool valid_shape(uint64_t rows, uint64_t cols) { return rows <= kMaxDim && cols >= 1 && cols <= kMaxDim; }
// A matrix the call reads or writes: there, aligned to its elements, rows apart.
inline bool valid_matrix(const void* p, int dtype, uint64_t cols, uint64_t stride) {
    return p && aligned(p, dtype == TLC_F32 ? 4 : 2) && stride >= cols && stride <= kMaxDim;
}
inline bool valid_checkpoint(const void* codes, const void* scales) {
    return codes && scales && aligned(codes, 16) && aligned(scales, 4);
}

// Calls fn with the type and the format as template arguments.
template <typename Fn>
int with_dtype(int dtype, Fn&& fn) {
    return dtype == TLC_F32 ? fn(F32{}) : dtype == TLC_F16 ? fn(F16{}) : fn(BF16{});
}
// A weight vector is of the matrix's type or fp32, a template argument of the
// kernels that read one.
inline bool valid_weight(const void* p, int weight_dtype, int dtype) {
    return !p || ((weight_dtype == TLC_F32 || weight_dtype == dtype) && aligned(p, weight_dtype == TLC_F32 ? 4 : 2));
}
template <typename T, typename Fn>
int with_weight(T, const void* p, int weight_dtype, Fn&& fn) {
    if constexpr (T::kTerms != 3)
        if (p && weight_dtype != TLC_F32) return fn(T{});
    return fn(F32{});
}
template <int N>
struct Int {
    static constexpr int value = N;
};
template <typename Fn>
int with_format(int format, Fn&& fn) {
    return format == TLC_CKPT8_INT8 ? fn(Int<TLC_CKPT8_INT8>{}) : fn(Int<TLC_CKPT8_E4M3>{});
}

}  // namespace tlc_ckpt8

#endif  // TLC_CKPT8_H
