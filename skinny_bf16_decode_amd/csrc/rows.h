// Rows of BF16, FP16 or fp32 values in 16-byte vectors or eight at a time, and
// their roundings to 8 and 4 bits, with a scale for each row or a power of two
// for each block of 32: shared by the kernels that read and quantize rows.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/skinny.h"

namespace skinny {

typedef __attribute__((ext_vector_type(4))) unsigned int u32x4;
typedef __attribute__((ext_vector_type(2))) unsigned int u32x2;

template <int TYPE>
struct Elem;
template <>
struct Elem<SKINNY_TYPE_BF16> {
    typedef unsigned short raw;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float get(raw v) { return __uint_as_float((unsigned)v << 16); }
    static __device__ __forceinline__ raw put(float v) { return __builtin_bit_cast(raw, (__bf16)v); }
    static __device__ __forceinline__ void unpack(u32x4 v, float (&f)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned int w = v[i];
            f[2 * i] = __uint_as_float(w << 16);
            f[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
        }
    }
};
template <>
struct Elem<SKINNY_TYPE_F16> {
    typedef unsigned short raw;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float get(raw v) { return (float)__builtin_bit_cast(_Float16, v); }
    static __device__ __forceinline__ raw put(float v) { return __builtin_bit_cast(raw, (_Float16)v); }
    static __device__ __forceinline__ void unpack(u32x4 v, float (&f)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned int w = v[i];
            f[2 * i] = get((raw)(w & 0xFFFFu));
            f[2 * i + 1] = get((raw)(w >> 16));
        }
    }
};
template <>
struct Elem<SKINNY_TYPE_F32> {
    typedef float raw;
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float get(raw v) { return v; }
    static __device__ __forceinline__ raw put(float v) { return v; }
    static __device__ __forceinline__ void unpack(u32x4 v, float (&f)[4])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned int w = v[i];
            f[i] = __uint_as_float(w);
        }
    }
};

// Magnitude bits of an fp32 value: ordered as unsigned integers like the
// values, with infinity and NaN (which a maximum of floats would drop) on top.
__device__ __forceinline__ unsigned mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ unsigned wave_max_u(unsigned v)
{
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
        const unsigned o = (unsigned)__shfl_xor((int)v, s, 64);
        v = o > v ? o : v;
    }
    return v;
}

// What a row's values are multiplied with, in two steps: lift (a power of
// two), then 127 / (lifted maximum), rounded to fp32 once.
struct RowScale {
    float lift, inverse;
    bool fine;                  // finite and not all zero
};

__device__ __forceinline__ RowScale row_scale(unsigned top_bits, float &scale)
{
    RowScale r;
    const float top = __uint_as_float(top_bits);
    const bool finite = top_bits < 0x7F800000u;
    r.fine = finite && top_bits != 0u;
    r.lift = top < 0x1p-60f ? 0x1p64f : 1.0f;
    r.inverse = r.fine ? __fdiv_rn(127.0f, top * r.lift) : 0.0f;
    scale = finite ? __fdiv_rn(top, 127.0f) : __uint_as_float(0x7FC00000u);
    return r;
}

__device__ __forceinline__ int to_int8(float v, const RowScale &r)
{
    return r.fine ? (int)rintf(__fmul_rn(__fmul_rn(v, r.lift), r.inverse)) : 0;
}

// ---------------------------------------------------------------------------
// Eight neighbouring elements (an octet) of a row of any type
// ---------------------------------------------------------------------------

struct Octet {
    u32x4 a, b;                 // as they lie in memory; b: the second half of an fp32 octet
};

// Octet o of a row of K elements.  VEC: whole octets at 16-byte aligned places;
// else element by element, zero past K.
template <bool VEC>
__device__ __forceinline__ Octet load_octet(const void *row, int type, int o, long long K)
{
    Octet v;
    v.a = v.b = u32x4{0u, 0u, 0u, 0u};
    if constexpr (VEC) {
        const u32x4 *p = static_cast<const u32x4 *>(row);
        if (type == SKINNY_TYPE_F32) {
            v.a = p[2 * (long long)o];
            v.b = p[2 * (long long)o + 1];
        } else {
            v.a = p[o];
        }
    } else {
        const long long first = 8 * (long long)o;
        if (type == SKINNY_TYPE_F32) {
            const unsigned *p = static_cast<const unsigned *>(row) + first;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v.a[e] = first + e < K ? p[e] : 0u;
                v.b[e] = first + 4 + e < K ? p[4 + e] : 0u;
            }
        } else {
            const unsigned short *p = static_cast<const unsigned short *>(row) + first;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const unsigned lo = first + 2 * e < K ? p[2 * e] : 0u;
                const unsigned hi = first + 2 * e + 1 < K ? p[2 * e + 1] : 0u;
                v.a[e] = lo | hi << 16;
            }
        }
    }
    return v;
}

__device__ __forceinline__ void unpack_octet(const Octet &v, int type, float (&f)[8])
{
    if (type == SKINNY_TYPE_F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned lo = v.a[e], hi = v.b[e];
            f[e] = __uint_as_float(lo);
            f[4 + e] = __uint_as_float(hi);
        }
    } else if (type == SKINNY_TYPE_F16) {
        Elem<SKINNY_TYPE_F16>::unpack(v.a, f);
    } else {
        Elem<SKINNY_TYPE_BF16>::unpack(v.a, f);
    }
}

// f to the type, as it lies in memory; f becomes what the type holds of it.
__device__ __forceinline__ Octet pack_octet(int type, float (&f)[8])
{
    Octet v;
    v.a = v.b = u32x4{0u, 0u, 0u, 0u};
    if (type == SKINNY_TYPE_F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v.a[e] = __float_as_uint(f[e]);
            v.b[e] = __float_as_uint(f[4 + e]);
        }
        return v;
    }
    if (type == SKINNY_TYPE_F16) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v.a[e] = Elem<SKINNY_TYPE_F16>::put(f[2 * e]) | (unsigned)Elem<SKINNY_TYPE_F16>::put(f[2 * e + 1]) << 16;
        Elem<SKINNY_TYPE_F16>::unpack(v.a, f);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v.a[e] = Elem<SKINNY_TYPE_BF16>::put(f[2 * e]) | (unsigned)Elem<SKINNY_TYPE_BF16>::put(f[2 * e + 1]) << 16;
        Elem<SKINNY_TYPE_BF16>::unpack(v.a, f);
    }
    return v;
}

template <bool VEC>
__device__ __forceinline__ void store_octet(void *row, int type, int o, long long K, const Octet &v)
{
    if constexpr (VEC) {
        u32x4 *p = static_cast<u32x4 *>(row);
        if (type == SKINNY_TYPE_F32) {
            p[2 * (long long)o] = v.a;
            p[2 * (long long)o + 1] = v.b;
        } else {
            p[o] = v.a;
        }
    } else {
        const long long first = 8 * (long long)o;
        if (type == SKINNY_TYPE_F32) {
            unsigned *p = static_cast<unsigned *>(row) + first;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (first + e < K)
                    p[e] = v.a[e];
                if (first + 4 + e < K)
                    p[4 + e] = v.b[e];
            }
        } else {
            unsigned short *p = static_cast<unsigned short *>(row) + first;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const unsigned w = v.a[e / 2];
                if (first + e < K)
                    p[e] = (unsigned short)(w >> (16 * (e & 1)));
            }
        }
    }
}

// Codes of an octet, BITS each, to the row's bytes q.  VEC: q and its pitch are multiples of BITS bytes.
template <bool VEC, int BITS>
__device__ __forceinline__ void store_codes(unsigned char *q, int o, u32x2 codes)
{
    unsigned char *p = q + (long long)o * BITS;
    if constexpr (VEC) {
        if constexpr (BITS == 8)
            *reinterpret_cast<u32x2 *>(p) = codes;
        else
            *reinterpret_cast<unsigned *>(p) = codes[0];
    } else {
#pragma unroll
        for (int e = 0; e < BITS; ++e) {
            const unsigned w = codes[e / 4];
            p[e] = (unsigned char)(w >> (8 * (e & 3)));
        }
    }
}

// 1 / (1 + exp(-x)) in place.  exp(-x) = 2^t (1 + d ln 2) with t + d = -x log2(e) to
// 48 bits, then the unit's reciprocal and a step of Newton's: some 3 steps of 2^-24,
// for 13 instructions a value against 30 of expf and a division (1000 x 18432
// gated and quantized: 18.6 against 23.4 us).  Where the sum may not be finite or the result subnormal,
// the formula as it is.
__device__ __forceinline__ void sigmoid(float (&x)[8])
{
    float low = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e)
        low = fminf(low, x[e]);
    if (low < -87.0f) {
        for (int e = 0; e < 8; ++e)
            x[e] = 1.0f / (1.0f + expf(-x[e]));
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float v = x[e] > 88.0f ? 88.0f : x[e];    // NaN stays
        const float t = v * -0x1.715476p+0f;
        const float d = fmaf(v, -0x1.4ae0cp-26f, fmaf(v, -0x1.715476p+0f, -t));
        const float p = __builtin_amdgcn_exp2f(t);
        const float s = 1.0f + fmaf(p * d, 0x1.62e43p-1f, p);
        const float y = __builtin_amdgcn_rcpf(s);
        x[e] = fmaf(fmaf(-s, y, 1.0f), y, y);
    }
}

// ---------------------------------------------------------------------------
// Blocks of 32 with a power of two
// ---------------------------------------------------------------------------

constexpr int kBlock = 32;

// The octet f of a block that this lane and the three others of its quad hold,
// to codes of BITS, e2m1 or e4m3 (OCP Microscaling Formats v1.0, section 6.3):
// the block's power is floor(log2 of the largest magnitude) less the type's
// largest exponent, at least -127; values go to the nearest, ties to even, and
// past the largest one (6 or 448) to that.  byte: the power + 127, or 255 for
// a block with an infinity or NaN, whose codes are 0.  Scaling is by a power of
// two, exact but for values that are subnormal then and rounded to zero.
// All four lanes of a quad have to be here.
template <int BITS>
__device__ __forceinline__ u32x2 block_codes(const float (&f)[8], unsigned &byte)
{
    unsigned top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const unsigned m = mag(f[e]);
        top = m > top ? m : top;
    }
    // lanes 1 and 2 apart in the quad
    unsigned o = (unsigned)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xF, 0xF, true);
    top = o > top ? o : top;
    o = (unsigned)__builtin_amdgcn_mov_dpp((int)top, 0x4E, 0xF, 0xF, true);
    top = o > top ? o : top;
    const bool fine = top < 0x7F800000u;
    const int power = (int)(top >> 23) - (BITS == 8 ? 8 : 2);
    const unsigned at = power > 0 ? (unsigned)power : 0u;
    byte = fine ? at : 255u;
    const float inverse = __uint_as_float((254u - at) << 23);
    u32x2 codes = u32x2{0u, 0u};
    if constexpr (BITS == 8) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = __builtin_amdgcn_fmed3f(f[e] * inverse, -448.0f, 448.0f);
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[e], v[e + 1], 0, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(v[e + 2], v[e + 3], w, true);
            codes[e / 4] = fine ? (unsigned)w : 0u;
        }
    } else {
        // clips at 6 by itself
        unsigned w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, f[0] * inverse, f[1] * inverse, 1.0f, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2] * inverse, f[3] * inverse, 1.0f, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4] * inverse, f[5] * inverse, 1.0f, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6] * inverse, f[7] * inverse, 1.0f, 3);
        codes[0] = fine ? w : 0u;
    }
    return codes;
}

// 2^(byte - 127); NaN for 255.
__device__ __forceinline__ float power_of(unsigned byte)
{
    return __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23);
}

}  // namespace skinny
