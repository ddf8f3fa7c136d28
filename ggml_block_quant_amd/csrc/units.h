// units.h -- 32 consecutive weights of a row (a "unit"), for every implemented
// format: the raw bytes held in registers between their loads and their
// decode, so that a kernel can keep a tile's loads in flight while it works on
// the tile before.
//
// Unit b is elements 32 b .. 32 b + 31 of the flattened [N][K] tensor; K is a
// multiple of 32, so a unit never crosses a row or a block.  Its elements 8 t ..
// 8 t + 7 have the values of dequant8 (decode.h), exact in fp32 or, in the
// affine formats, rounded once; FP8 gives the codes' values without the row's
// scale (the kernels apply it elsewhere): values(t, w).  halves(t, h) gives
// them as four pairs of fp16, rounded once more; pairs(t, h, l) with what that rounding
// leaves as a second fp16 each.  The tuned formats' codes reach it two at a time, as the 16-bit patterns of
// fp16's smallest numbers: a code u in the low bits is u * 2^-24, which a mixed
// multiply-add (fp32 scale times 2^24, fp16 code, fp32 offset, fp16 result)
// takes as it is, without a conversion of its own (Q4K: 13 instructions for 8
// weights, 23 through fp32).
#pragma once

#include "decode.h"

namespace ql {

// 6-bit scale and min j (of 8) of a Q4K / Q5K header, times d and dmin
__device__ __forceinline__ void header_scales(uint4 h, int j, float &S, float &T)
{
    const uint32_t sc = ((h.y >> (4 * j)) & 15u) | ((h.w >> (2 * j)) & 3u) << 4;
    const uint32_t mq = ((h.z >> (4 * j)) & 15u) | ((h.w >> (16 + 2 * j)) & 3u) << 4;
    S = f16_bits_to_f32(h.x) * (float)sc;
    T = -(f16_bits_to_f32(h.x >> 16) * (float)mq);
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ uint32_t word(const uint2 &v, int i) { return i == 0 ? v.x : v.y; }

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_f16(float a, float b)
{
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});  // v_cvt_pk_f16_f32, to nearest even
}
// fp16(s u + t) of two codes in 16 bits each, s the scale times 2^24
__device__ __forceinline__ uint32_t scale_codes(uint32_t codes, float s, float t)
{
    const f16x2 u = __builtin_bit_cast(f16x2, codes);
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)fmaf(s, (float)u.x, t), (_Float16)fmaf(s, (float)u.y, t)});
}
// hi = fp16(v), lo = fp16(v - hi) of two values
__device__ __forceinline__ void split_f16(float a, float b, uint32_t &hi, uint32_t &lo)
{
    hi = pack_f16(a, b);
    // (hi as it stands, and a factor that the compiler does not know to be -1:
    // it makes hi twice and three instructions of a difference otherwise, and
    // from this one mixed multiply-add a value)
    float minus = -1.0f;
    asm("" : "+s"(minus));
    asm("" : "+v"(hi));
    const f16x2 p = __builtin_bit_cast(f16x2, hi);
    lo = __builtin_bit_cast(uint32_t, f16x2{(_Float16)fmaf((float)p.x, minus, a), (_Float16)fmaf((float)p.y, minus, b)});
}

// Through fp32: units that give values (decode)
template <typename U> struct ByValue {
    __device__ __forceinline__ void values(int t, float w[8]) const { static_cast<const U *>(this)->decode(t, w); }
    __device__ __forceinline__ void halves(int t, uint32_t h[4]) const
    {
        float v[8];
        static_cast<const U *>(this)->decode(t, v);
#pragma unroll
        for (int j = 0; j < 4; j++)
            h[j] = pack_f16(v[2 * j], v[2 * j + 1]);
    }
    __device__ __forceinline__ void pairs(int t, uint32_t h[4], uint32_t l[4]) const
    {
        float v[8];
        static_cast<const U *>(this)->decode(t, v);
#pragma unroll
        for (int j = 0; j < 4; j++)
            split_f16(v[2 * j], v[2 * j + 1], h[j], l[j]);
    }
};
// From 16-bit codes: units that give codes(t, c, s, z), four pairs of codes,
// each pair's scale times 2^24 (or 2^20 where the codes stand four bits up),
// and the offset of the task's weights
template <typename U> struct ByCode {
    __device__ __forceinline__ void values(int t, float w[8]) const
    {
        uint32_t c[4];
        float s[4], z;
        static_cast<const U *>(this)->codes(t, c, s, z);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const f16x2 u = __builtin_bit_cast(f16x2, c[j]);
            w[2 * j] = fmaf(s[j], (float)u.x, z), w[2 * j + 1] = fmaf(s[j], (float)u.y, z);
        }
    }
    __device__ __forceinline__ void halves(int t, uint32_t h[4]) const
    {
        uint32_t c[4];
        float s[4], z;
        static_cast<const U *>(this)->codes(t, c, s, z);
#pragma unroll
        for (int j = 0; j < 4; j++)
            h[j] = scale_codes(c[j], s[j], z);
    }
    __device__ __forceinline__ void pairs(int t, uint32_t h[4], uint32_t l[4]) const
    {
        uint32_t c[4];
        float s[4], z;
        static_cast<const U *>(this)->codes(t, c, s, z);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const f16x2 u = __builtin_bit_cast(f16x2, c[j]);
            split_f16(fmaf(s[j], (float)u.x, z), fmaf(s[j], (float)u.y, z), h[j], l[j]);
        }
    }
};

// Holds back what is computed from a loaded register.  Without it the compiler
// moves a unit's first conversions up behind its load and waits for the memory
// there, steps too early (a field that is widened where it is loaded likewise:
// 16-bit fields stay 16 bits wide in a unit).
__device__ __forceinline__ void hold(uint16_t &x) { asm volatile("" : "+v"(x)); }

template <int FMT> struct Unit;

// S (u - 128) with the signed code's sign bit flipped: S u - 128 S is exact
// before its one rounding, which S times the code needs none of
template <> struct Unit<FMT_Q8_0> : ByCode<Unit<FMT_Q8_0>> {
    uint4 c0, c1;
    uint16_t d;
    float S, T;
    __device__ __forceinline__ void load(const uint8_t *__restrict__ B, const Planes &p, int64_t b)
    {
        c0 = reinterpret_cast<const uint4 *>(B)[2 * b];
        c1 = reinterpret_cast<const uint4 *>(B)[2 * b + 1];
        d = reinterpret_cast<const uint16_t *>(B + p.scales)[b];
    }
    __device__ __forceinline__ void begin()
    {
        hold(d);
        S = f16_bits_to_f32(d), T = -128.0f * S;
    }
    __device__ __forceinline__ void codes(int t, uint32_t c[4], float s[4], float &z) const
    {
        const uint32_t x = word(t < 2 ? c0 : c1, 2 * (t & 1)) ^ 0x80808080u;
        const uint32_t y = word(t < 2 ? c0 : c1, 2 * (t & 1) + 1) ^ 0x80808080u;
        c[0] = __builtin_amdgcn_perm(0u, x, 0x0c010c00u), c[1] = __builtin_amdgcn_perm(0u, x, 0x0c030c02u);
        c[2] = __builtin_amdgcn_perm(0u, y, 0x0c010c00u), c[3] = __builtin_amdgcn_perm(0u, y, 0x0c030c02u);
        s[0] = s[1] = s[2] = s[3] = S * 0x1p24f;
        z = T;
    }
};

template <> struct Unit<FMT_Q4K> : ByCode<Unit<FMT_Q4K>> {
    uint4 c, h;
    int j;
    float S, T;
    __device__ __forceinline__ void load(const uint8_t *__restrict__ B, const Planes &p, int64_t b)
    {
        c = reinterpret_cast<const uint4 *>(B)[b];
        h = reinterpret_cast<const uint4 *>(B + p.scales)[b >> 3];
        j = (int)(b & 7);
    }
    __device__ __forceinline__ void begin() { header_scales(h, j, S, T); }
    __device__ __forceinline__ void codes(int t, uint32_t x[4], float s[4], float &z) const
    {
        // elements 2 p and 2 p + 1 at nibbles p and p + 4; every second pair
        // keeps its nibbles four bits up
        const uint32_t d = word(c, t), d8 = d >> 8;
        x[0] = d & 0x000f000fu, x[1] = d & 0x00f000f0u, x[2] = d8 & 0x000f000fu, x[3] = d8 & 0x00f000f0u;
        s[0] = s[2] = S * 0x1p24f, s[1] = s[3] = S * 0x1p20f;
        z = T;
    }
};

template <> struct Unit<FMT_Q6K> : ByCode<Unit<FMT_Q6K>> {
    uint4 lo;
    uint2 hi;
    uint16_t sc, d;
    float S, S1;
    __device__ __forceinline__ void load(const uint8_t *__restrict__ B, const Planes &p, int64_t b)
    {
        const int64_t g = b >> 3;
        const int c = (int)(b & 7);
        lo = *reinterpret_cast<const uint4 *>(B + 192 * g + 16 * c);
        hi = *reinterpret_cast<const uint2 *>(B + 192 * g + 128 + 8 * c);
        sc = *reinterpret_cast<const uint16_t *>(B + p.scales + 16 * g + 2 * c);
        d = reinterpret_cast<const uint16_t *>(B + p.d)[g];
    }
    __device__ __forceinline__ void begin()
    {
        hold(sc), hold(d);
        const float f = f16_bits_to_f32(d);
        S = f * (float)(int8_t)sc, S1 = f * (float)(int8_t)(sc >> 8);
    }
    __device__ __forceinline__ void codes(int t, uint32_t x[4], float s[4], float &z) const
    {
        // elements 2 p and 2 p + 1: nibbles p and p + 4, high bits 2 p of the
        // octet and of the one 16 bits up
        const uint32_t l = word(lo, t), a = word(hi, t >> 1) >> (8 * (t & 1));
        x[0] = (l & 0x000f000fu) | ((a << 4) & 0x00300030u);
        x[1] = (l & 0x00f000f0u) | ((a << 6) & 0x03000300u);
        x[2] = ((l >> 8) & 0x000f000fu) | (a & 0x00300030u);
        x[3] = ((l >> 8) & 0x00f000f0u) | ((a << 2) & 0x03000300u);
        const float f = t < 2 ? S : S1;
        s[0] = s[2] = f * 0x1p24f, s[1] = s[3] = f * 0x1p20f;
        z = -32.0f * f;
    }
};

// Natural order (all formats below): element k of a task at field k of its
// word, the top bit (where there is one) at bit k of its byte.
template <> struct Unit<FMT_Q5K> : ByValue<Unit<FMT_Q5K>> {
    uint4 c, h;
    uint32_t hi;
    int j;
    float S, T;
    __device__ __forceinline__ void load(const uint8_t *__restrict__ B, const Planes &p, int64_t b)
    {
        c = reinterpret_cast<const uint4 *>(B)[b];
        hi = *reinterpret_cast<const uint32_t *>(B + p.hi + 4 * b);
        h = reinterpret_cast<const uint4 *>(B + p.scales)[b >> 3];
        j = (int)(b & 7);
    }
    __device__ __forceinline__ void begin() { header_scales(h, j, S, T); }
    __device__ __forceinline__ void decode(int t, float w[8]) const
    {
        const uint32_t lo = word(c, t), hb = hi >> (8 * t);
#pragma unroll
        for (int k = 0; k < 8; k++)
            w[k] = fmaf(S, (float)(((lo >> (4 * k)) & 15u) | ((hb >> k) & 1u) << 4), T);
    }
};

template <> struct Unit<FMT_Q3K> : ByValue<Unit<FMT_Q3K>> {
    uint2 c;
    uint32_t hi, s0, s2;
    uint16_t d;
    int j;
    float S, S1;
    __device__ __forceinline__ void load(const uint8_t *__restrict__ B, const Planes &p, int64_t b)
    {
        const int64_t g = b >> 3;
        j = (int)(b & 7);
        c = reinterpret_cast<const uint2 *>(B)[b];
        hi = *reinterpret_cast<const uint32_t *>(B + p.hi + 4 * b);
        const uint32_t *s3 = reinterpret_cast<const uint32_t *>(B + p.scales + 12 * g);
        s0 = s3[j >> 2], s2 = s3[2];
        d = reinterpret_cast<const uint16_t *>(B + p.d)[g];
    }
    __device__ __forceinline__ void begin()
    {
        // sub-blocks 2 j and 2 j + 1 of 16
        const int i = (2 * j) & 7;
        const uint32_t a = ((s0 >> (4 * i)) & 15u) | ((s2 >> (4 * j)) & 3u) << 4;
        const uint32_t b = ((s0 >> (4 * i + 4)) & 15u) | ((s2 >> (4 * j + 2)) & 3u) << 4;
        const float f = f16_bits_to_f32(d);
        S = f * (float)a, S1 = f * (float)b;
    }
    __device__ __forceinline__ void decode(int t, float w[8]) const
    {
        const uint32_t lo = word(c, t >> 1) >> (16 * (t & 1)), hb = hi >> (8 * t);
        const float s = t < 2 ? S : S1;
#pragma unroll
        for (int k = 0; k < 8; k++)
            w[k] = s * (float)((int)(((lo >> (2 * k)) & 3u) | ((hb >> k) & 1u) << 2) - 4);
    }
};

template <> struct Unit<FMT_Q2K> : ByValue<Unit<FMT_Q2K>> {
    uint2 c;
    uint16_t sm;
    uint32_t dd;
    float S, T, S1, T1;
    __device__ __forceinline__ void load(const uint8_t *__restrict__ B, const Planes &p, int64_t b)
    {
        c = reinterpret_cast<const uint2 *>(B)[b];
        sm = *reinterpret_cast<const uint16_t *>(B + p.scales + 2 * b);
        dd = reinterpret_cast<const uint32_t *>(B + p.d)[b >> 3];
    }
    __device__ __forceinline__ void begin()
    {
        const float d = f16_bits_to_f32(dd), m = -f16_bits_to_f32(dd >> 16);
        S = d * (float)(sm & 15u), T = m * (float)((sm >> 4) & 15u);
        S1 = d * (float)((sm >> 8) & 15u), T1 = m * (float)(sm >> 12);
    }
    __device__ __forceinline__ void decode(int t, float w[8]) const
    {
        const uint32_t lo = word(c, t >> 1) >> (16 * (t & 1));
        const float s = t < 2 ? S : S1, z = t < 2 ? T : T1;
#pragma unroll
        for (int k = 0; k < 8; k++)
            w[k] = fmaf(s, (float)((lo >> (2 * k)) & 3u), z);
    }
};

// E4M3 codes as their values
template <> struct Unit<FMT_FP8> : ByValue<Unit<FMT_FP8>> {
    uint4 c0, c1;
    __device__ __forceinline__ void load(const uint8_t *__restrict__ B, const Planes &, int64_t b)
    {
        c0 = reinterpret_cast<const uint4 *>(B)[2 * b];
        c1 = reinterpret_cast<const uint4 *>(B)[2 * b + 1];
    }
    __device__ __forceinline__ void begin() {}
    __device__ __forceinline__ void decode(int t, float w[8]) const
    {
        const int x = (int)word(t < 2 ? c0 : c1, 2 * (t & 1)), y = (int)word(t < 2 ? c0 : c1, 2 * (t & 1) + 1);
        w[0] = __builtin_amdgcn_cvt_f32_fp8(x, 0), w[1] = __builtin_amdgcn_cvt_f32_fp8(x, 1);
        w[2] = __builtin_amdgcn_cvt_f32_fp8(x, 2), w[3] = __builtin_amdgcn_cvt_f32_fp8(x, 3);
        w[4] = __builtin_amdgcn_cvt_f32_fp8(y, 0), w[5] = __builtin_amdgcn_cvt_f32_fp8(y, 1);
        w[6] = __builtin_amdgcn_cvt_f32_fp8(y, 2), w[7] = __builtin_amdgcn_cvt_f32_fp8(y, 3);
    }
};

// the 32-element blocks: Q4_0, Q5_0 (symmetric), Q4_1, Q5_1 (with a minimum)
template <int FMT> struct Unit : ByValue<Unit<FMT>> {
    static constexpr bool five = FMT == FMT_Q5_0 || FMT == FMT_Q5_1;
    static constexpr bool affine = FMT == FMT_Q4_1 || FMT == FMT_Q5_1;
    static_assert(FMT == FMT_Q4_0 || five || affine, "a 32-element block format");
    uint4 c;
    uint32_t hi;
    uint16_t d, m;
    float S, T;
    __device__ __forceinline__ void load(const uint8_t *__restrict__ B, const Planes &p, int64_t b)
    {
        c = reinterpret_cast<const uint4 *>(B)[b];
        d = reinterpret_cast<const uint16_t *>(B + p.d)[b];
        if constexpr (five)
            hi = *reinterpret_cast<const uint32_t *>(B + p.hi + 4 * b);
        if constexpr (affine)
            m = reinterpret_cast<const uint16_t *>(B + p.m)[b];
    }
    __device__ __forceinline__ void begin()
    {
        S = f16_bits_to_f32(d);
        T = affine ? f16_bits_to_f32(m) : -(FMT == FMT_Q4_0 ? 8.0f : 16.0f) * S;
    }
    __device__ __forceinline__ void decode(int t, float w[8]) const
    {
        const uint32_t lo = word(c, t), hb = five ? hi >> (8 * t) : 0u;
#pragma unroll
        for (int k = 0; k < 8; k++)
            w[k] = fmaf(S, (float)(((lo >> (4 * k)) & 15u) | ((hb >> k) & 1u) << 4), T);
    }
};

}  // namespace ql
