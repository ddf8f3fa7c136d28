// moe.hip -- the mixture-of-experts layer on block-quantized expert weights:
//   Y[t] = sum_j w[t][j] * Wd[e] . (act(Wg[e] . x_t) * (Wu[e] . x_t)),  e = ids[t][j],
// and the router's choice that produces ids and w.
//
// Two forms.
//   Few pairs an expert: two kernels.  moe_glu_kernel computes H[t][j] = act(g) * u, a
//   workgroup per (token, choice) and group of rows; moe_down_kernel computes
//   Y, a workgroup per token and group of output rows, whose lanes walk the
//   chunks of all k chosen experts' rows at once, so the join over the
//   choices is the reduction over the lanes and no partial result is stored.
//   More: the (token, choice) pairs are sorted by expert, two grouped matrix-core products run over tiles of one
//   expert's pairs, and moe_join_kernel adds each token's k results in the
//   order of its choices.
//
// Nothing is added atomically: a token's result does not depend on the order
// in which workgroups run.
#include "moe.h"
#include "decode.h"

#include <math.h>

namespace ql {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_lo(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}

// Sums of V values over the 64 lanes (V a power of two <= 64): while more
// than one is left a step keeps half of them, so V values cost about V + 4
// additions.  Lanes 0 .. V-1 end with the total of value sum_index<V>(lane).
// A halving step needs the lane that differs in bit B exactly; a plain sum
// any lane with the same lower bits, which for bits 2 to 5 is a rotation
// inside a row of 16 or a swap of rows: VALU instructions, where a shuffle
// would go through LDS (~100 cycles each, one after the other).
template <int B>
__device__ __forceinline__ float partner(float x)
{
    if constexpr (B == 0)
        return dpp<0xB1>(x);
    else if constexpr (B == 1)
        return dpp<0x4E>(x);
    else
        return __shfl_xor(x, 1 << B);
}
// the two rows of 16 of each half (rows 0 1 and 2 3), or the halves of 32, as
// two values every lane has: the lower one and the upper one
__device__ __forceinline__ void swap_rows(float x, float &lo, float &hi)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    lo = __uint_as_float(r[0]), hi = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap_halves(float x, float &lo, float &hi)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    lo = __uint_as_float(r[0]), hi = __uint_as_float(r[1]);
}
template <int B>
__device__ __forceinline__ float plain_sum(float x)
{
    float lo, hi;
    if constexpr (B == 0)
        return x + dpp<0xB1>(x);
    else if constexpr (B == 1)
        return x + dpp<0x4E>(x);
    else if constexpr (B == 2)
        return x + dpp<0x124>(x);  // row_ror:4
    else if constexpr (B == 3)
        return x + dpp<0x128>(x);  // row_ror:8
    else if constexpr (B == 4)
        swap_rows(x, lo, hi);
    else
        swap_halves(x, lo, hi);
    return lo + hi;
}
template <int LEFT, int B, int V>
__device__ __forceinline__ void sum_step(float (&v)[V], int lane)
{
    if constexpr (LEFT > 1) {
        const bool up = (lane >> B) & 1;
#pragma unroll
        for (int i = 0; i < LEFT / 2; i++) {
            const float keep = up ? v[i + LEFT / 2] : v[i], send = up ? v[i] : v[i + LEFT / 2];
            v[i] = keep + partner<B>(send);
        }
    } else {
        v[0] = plain_sum<B>(v[0]);
    }
    if constexpr (B < 5)
        sum_step<(LEFT > 1 ? LEFT / 2 : 1), B + 1>(v, lane);
}
template <int V>
__device__ __forceinline__ float wave_sums(float (&v)[V], int lane)
{
    sum_step<V, 0>(v, lane);
    return v[0];
}
template <int V>
__device__ __forceinline__ int sum_index(int lane)
{
    int idx = 0, part = V;
#pragma unroll
    for (int b = 0; b < 6; b++)
        if (part > 1) {
            part >>= 1;
            if ((lane >> b) & 1)
                idx += part;
        }
    return idx;
}

// ---------------------------------------------------------------------------
// Router: a wave per token.  Expert e sits in lane e % 64, register e / 64.
// Choices are made one by one: the wave's largest key, the lowest index among
// equal ones, which then leaves the race.
// ---------------------------------------------------------------------------
template <typename KT>
__device__ __forceinline__ KT wave_max(KT v)
{
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const KT o = __shfl_xor(v, s);
        v = o > v ? o : v;
    }
    return v;
}

__device__ __forceinline__ float wave_max(float v)
{
    float lo, hi;
    v = fmaxf(v, dpp<0xB1>(v));
    v = fmaxf(v, dpp<0x4E>(v));
    v = fmaxf(v, dpp<0x124>(v));
    v = fmaxf(v, dpp<0x128>(v));
    swap_rows(v, lo, hi);
    swap_halves(fmaxf(lo, hi), lo, hi);
    return fmaxf(lo, hi);
}

// BIAS: the key is sigmoid(x) + bias in 64 bits (where 32 would let the
// rounding of e^-x decide between close experts); otherwise it is x itself,
// in whose order both scores are.  A wave per token, its logits in registers.
// Few tokens: the launch (3.5 us for one token of 128 experts); many: the k
// rounds of a maximum over the wave (4096 tokens of 256 experts, k = 8, with
// bias: 12 us for 4 MB of logits).
template <int VPT, bool BIAS>
__global__ __launch_bounds__(256) void moe_route_kernel(const float *__restrict__ logits, int T, int E, int k, int score,
                                                        const float *__restrict__ bias, int renorm, float scale,
                                                        int32_t *__restrict__ ids, float *__restrict__ weights)
{
    using KT = std::conditional_t<BIAS, double, float>;
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T)
        return;
    const float *row = logits + (int64_t)t * E;
    KT key[VPT];
    float x[VPT], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int e = lane + 64 * i;
        float v = e < E ? row[e] : -INFINITY;
        v = v == v ? fminf(v, 3.4028234663852886e38f) : -INFINITY;  // NaN: switched off
        x[i] = v;
        m = fmaxf(m, v);
        if constexpr (BIAS)
        {
            const double b = v > -INFINITY ? (double)bias[e] : -(double)INFINITY;
            key[i] = b == b ? 1.0 / (1.0 + exp(-(double)v)) + b : -(double)INFINITY;
        }
        else
            key[i] = v;
    }
    m = wave_max(m);
    int my_id = -1;
    float my_x = 0.0f;
    for (int j = 0; j < k; j++) {
        KT best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < VPT; i++)
            if (key[i] > best)
                best = key[i], at = i;
        const KT top = wave_max(best);
        if (!(top > -(KT)INFINITY))
            break;
        // the lowest index with that key
        int e = best == top ? lane + 64 * at : 0x7FFFFFFF;
        const uint64_t who = __ballot(best == top);
        if (__popcll(who) == 1)
            e = __shfl(e, __ffsll((unsigned long long)who) - 1);
        else
#pragma unroll
            for (int s = 1; s < 64; s <<= 1)
                e = min(e, __shfl_xor(e, s));
        float xe = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; i++)
            if (e == lane + 64 * i) {
                key[i] = -(KT)INFINITY;
                xe = x[i];
            }
        xe = __shfl(xe, e & 63);
        if (lane == j) {
            my_id = e;
            my_x = xe;
        }
    }
    // the chosen experts' scores, one per lane
    double p = 0.0;
    if (score == 0) {
        float z = 1.0f;
        if (!renorm) {
            z = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; i++)
                z += x[i] > -INFINITY ? expf(x[i] - m) : 0.0f;
#pragma unroll
            for (int s = 1; s < 64; s <<= 1)
                z += __shfl_xor(z, s);
        }
        p = my_id >= 0 ? (double)(expf(my_x - m) / z) : 0.0;
    } else {
        p = my_id >= 0 ? 1.0 / (1.0 + exp(-(double)my_x)) : 0.0;
    }
    if (renorm) {
        double s = p;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
            s += __shfl_xor(s, d);
        p = s > 0.0 ? p / s : 0.0;
    }
    if (lane < k) {
        ids[(int64_t)t * k + lane] = my_id;
        weights[(int64_t)t * k + lane] = (float)(p * (double)scale);
    }
}

// ---------------------------------------------------------------------------
// Few tokens.  A row of K weights is cut into chunks of 32; a lane owns a
// chunk of the row, keeps its 32 activations in registers and walks down the
// workgroup's rows, R at a time: the loads of the next R rows are issued
// before the current ones are used, so a wave always has R to 2 R rows of
// loads in flight and the activations are read once for all of them.  Per row
// a lane forms sum q * a of its chunk and applies the block scales once, so
// only fp32 sums round; the lanes' sums are joined by wave_sums and, where a
// row takes several waves, through LDS.
// Activations: bf16 X of Q4K weights stays in bf16 pairs for v_dot2_f32_bf16
// (the 4-bit codes are exact in bf16); otherwise they are fp32, which holds
// bf16 X exactly and does not round H.
// ---------------------------------------------------------------------------
struct Mat {
    const uint8_t *B;
    Planes p;
    int64_t K;  // row length
};

template <int FMT> struct Raw { int64_t task; };
template <> struct Raw<FMT_Q4K> { uint4 c; uint32_t h; };
template <> struct Raw<FMT_Q6K> { uint4 lo; uint2 hi; uint32_t sc2, d; };
template <> struct Raw<FMT_Q8_0> { uint4 c0, c1; uint32_t d; };

__device__ __forceinline__ uint4 stream16(const uint8_t *p)
{
    const u32x4_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
}

// Where a lane's chunk c of row n lies; row n + i is i row strides on.  The
// lanes of a quad hold chunks of one group of 256.
template <int FMT> struct At {
    const uint8_t *codes, *aux, *scales, *d;  // aux: Q6K's high bits
    int64_t task;                             // the other formats
};

template <int FMT>
__device__ __forceinline__ At<FMT> at_row(const Mat &w, int64_t n, int c, int lane)
{
    At<FMT> p{};
    const int64_t sub = n * (w.K / 32) + c, g = sub >> 3;
    if constexpr (FMT == FMT_Q4K) {
        p.codes = w.B + 16 * sub;
        // one dword of the 16-byte group header per lane, shared in the quad
        p.scales = w.B + w.p.scales + 16 * g + 4 * (lane & 3);
    } else if constexpr (FMT == FMT_Q6K) {
        p.codes = w.B + 192 * g + 16 * (c & 7);
        p.aux = w.B + 192 * g + 128 + 8 * (c & 7);
        p.scales = w.B + w.p.scales + 16 * g + 2 * (c & 7);
        p.d = w.B + w.p.d + 2 * g;
    } else if constexpr (FMT == FMT_Q8_0) {
        p.codes = w.B + 32 * sub;
        p.d = w.B + w.p.scales + 2 * sub;
    } else {
        p.task = 4 * sub;
    }
    return p;
}

// the chunk `row` rows on
template <int FMT>
__device__ __forceinline__ void load_raw(const Mat &w, const At<FMT> &p, int64_t row, Raw<FMT> &r)
{
    const int64_t gs = row * (w.K / 256);  // groups (Q8_0 rows may end in a part of one)
    if constexpr (FMT == FMT_Q4K) {
        r.c = stream16(p.codes + 128 * gs);
        r.h = *reinterpret_cast<const uint32_t *>(p.scales + 16 * gs);
    } else if constexpr (FMT == FMT_Q6K) {
        r.lo = stream16(p.codes + 192 * gs);
        r.hi = *reinterpret_cast<const uint2 *>(p.aux + 192 * gs);
        r.sc2 = *reinterpret_cast<const uint16_t *>(p.scales + 16 * gs);
        r.d = *reinterpret_cast<const uint16_t *>(p.d + 2 * gs);
    } else if constexpr (FMT == FMT_Q8_0) {
        r.c0 = stream16(p.codes + row * w.K);
        r.c1 = stream16(p.codes + row * w.K + 16);
        r.d = *reinterpret_cast<const uint16_t *>(p.d + row * (w.K / 16));
    } else {
        r.task = p.task + row * (w.K / 8);
    }
}

__device__ __forceinline__ float sb(uint32_t w, int b) { return (float)(int8_t)(w >> (8 * b)); }

// Q6K: byte b of lo (hi): four times the signed code of elements 0, 4, 1, 5
// (2, 6, 3, 7) of an octet: the low nibble at bits 2-5, the two high bits
// above it, the top one flipped (u - 32 in two's complement).  H: the octet's
// high bits at bits 0-7 (even elements) and 16-23 (odd ones).
__device__ __forceinline__ void q6k_bytes(uint32_t lw, uint32_t H, uint32_t &lo, uint32_t &hi)
{
    const uint32_t H2 = H >> 2;
    const uint32_t t0 = (H & 0x00030003u) | ((H & 0x00300030u) << 4);
    const uint32_t t1 = (H2 & 0x00030003u) | ((H2 & 0x00300030u) << 4);
    lo = (((lw << 2) & 0x3C3C3C3Cu) | (t0 << 6)) ^ 0x80808080u;
    hi = (((lw >> 2) & 0x3C3C3C3Cu) | (t1 << 6)) ^ 0x80808080u;
}

// sum over the chunk of w * a (every format but Q4K, whose activations are
// bf16 pairs or digits)
template <int FMT>
__device__ __forceinline__ float dot32(const Mat &w, const Raw<FMT> &r, const float (&a)[32])
{
    if constexpr (FMT == FMT_Q6K) {
        const float d = f16_bits_to_f32(r.d);
        const uint32_t lw[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w};
        const uint32_t hw[2] = {r.hi.x, r.hi.y};
        float s[2] = {0.0f, 0.0f};  // the two sub-blocks of 16, in units of a quarter
#pragma unroll
        for (int q = 0; q < 4; q++) {
            uint32_t lo, hi;
            q6k_bytes(lw[q], hw[q >> 1] >> (8 * (q & 1)), lo, hi);
            const float *x = a + 8 * q;
            float v = s[q >> 1];
            v = fmaf(sb(lo, 0), x[0], v);
            v = fmaf(sb(lo, 1), x[4], v);
            v = fmaf(sb(lo, 2), x[1], v);
            v = fmaf(sb(lo, 3), x[5], v);
            v = fmaf(sb(hi, 0), x[2], v);
            v = fmaf(sb(hi, 1), x[6], v);
            v = fmaf(sb(hi, 2), x[3], v);
            v = fmaf(sb(hi, 3), x[7], v);
            s[q >> 1] = v;
        }
        const float Sa = d * (float)(int8_t)r.sc2, Sb = d * (float)(int8_t)(r.sc2 >> 8);
        return 0.25f * fmaf(Sa, s[0], Sb * s[1]);
    } else if constexpr (FMT == FMT_Q8_0) {
        const uint32_t cw[8] = {r.c0.x, r.c0.y, r.c0.z, r.c0.w, r.c1.x, r.c1.y, r.c1.z, r.c1.w};
        float d0 = 0.0f, d1 = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            d0 = fmaf(sb(cw[i], 0), a[4 * i], d0);
            d1 = fmaf(sb(cw[i], 1), a[4 * i + 1], d1);
            d0 = fmaf(sb(cw[i], 2), a[4 * i + 2], d0);
            d1 = fmaf(sb(cw[i], 3), a[4 * i + 3], d1);
        }
        return f16_bits_to_f32(r.d) * (d0 + d1);
    } else {
        float d0 = 0.0f;
#pragma unroll
        for (int t = 0; t < 4; t++) {
            float v[8];
            dequant8<FMT>(w.B, w.p, r.task + t, v);
#pragma unroll
            for (int i = 0; i < 8; i++)
                d0 = fmaf(v[i], a[8 * t + i], d0);
        }
        return d0;
    }
}

// The activations of a chunk as the products take them.
template <bool PAIRS> struct Acts;
template <> struct Acts<true> {
    uint32_t p[16];  // bf16 pairs (0,4), (1,5), (2,6), (3,7) of each octet
    float sum;
};
template <> struct Acts<false> {
    float a[32];
};

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16v2_t;

__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c)
{
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16v2_t, a), __builtin_bit_cast(bf16v2_t, b), c, false);
}

// bytes 2H, 2H + 1 of w, each 0 .. 15, as the bf16 pair of those numbers: as
// an E4M3 byte u is u * 2^-9
template <bool H>
__device__ __forceinline__ uint32_t nib_pair(uint32_t w)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 512.0f, H));
}

// Q4K's scale and minimum of sub-block j from the quad's header dwords
__device__ __forceinline__ void q4k_scales(uint32_t hd, int j, float &S, float &Mn)
{
    const int h = (int)hd;
    const uint32_t h0 = __builtin_amdgcn_update_dpp(0, h, 0x00, 0xF, 0xF, false);
    const uint32_t h1 = __builtin_amdgcn_update_dpp(0, h, 0x55, 0xF, 0xF, false);
    const uint32_t h2 = __builtin_amdgcn_update_dpp(0, h, 0xAA, 0xF, 0xF, false);
    const uint32_t h3 = __builtin_amdgcn_update_dpp(0, h, 0xFF, 0xF, 0xF, false);
    const uint32_t sc = __builtin_amdgcn_ubfe(h1, 4 * j, 4) | (__builtin_amdgcn_ubfe(h3, 2 * j, 2) << 4);
    const uint32_t mq = __builtin_amdgcn_ubfe(h2, 4 * j, 4) | (__builtin_amdgcn_ubfe(h3, 16 + 2 * j, 2) << 4);
    S = f16_bits_to_f32(h0) * (float)sc;
    Mn = f16_bits_to_f32(h0 >> 16) * (float)mq;
}

template <int FMT, bool PAIRS>
__device__ __forceinline__ float dot(const Mat &w, const Raw<FMT> &r, int c, const Acts<PAIRS> &x)
{
    if constexpr (PAIRS) {
        float S, Mn;
        q4k_scales(r.h, c & 7, S, Mn);
        const uint32_t cw[4] = {r.c.x, r.c.y, r.c.z, r.c.w};
        float d0 = 0.0f, d1 = 0.0f;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const uint32_t lo = cw[q] & 0x0F0F0F0Fu, hi = (cw[q] >> 4) & 0x0F0F0F0Fu;
            d0 = dot2(nib_pair<false>(lo), x.p[4 * q], d0);
            d1 = dot2(nib_pair<true>(lo), x.p[4 * q + 1], d1);
            d0 = dot2(nib_pair<false>(hi), x.p[4 * q + 2], d0);
            d1 = dot2(nib_pair<true>(hi), x.p[4 * q + 3], d1);
        }
        return fmaf(S, d0 + d1, -Mn * x.sum);
    } else {
        return dot32<FMT>(w, r, x.a);
    }
}

// ---------------------------------------------------------------------------
// H between the two kernels.  For the tuned formats a chunk of 32 is stored
// as whole numbers v = h * 2^e of 23 bits, e chosen per chunk, split into
// three signed base-256 digits (v = 65536 d2 + 256 d1 + d0), because codes
// are small whole numbers too: v_dot4_i32_i8 then takes four products an
// instruction, exactly (24 instructions a chunk instead of 32 conversions
// and 32 fused multiply-adds; Q4K 122 -> 65 VALU instructions a chunk in
// all).  A value is held to 2^-23 of the largest of its chunk.  H8 is 7
// 16-byte words a chunk: digits d0 (2), d1 (2), d2 (2), then {2^-e, sum of h}.
// The bytes stand in the order in which the format's codes come out of their
// dwords: Q8_0 as they are; Q4K and Q6K per octet 0, 4, 1, 5 (low nibbles),
// 2, 6, 3, 7 (high nibbles).  The other formats take H in fp32.
// ---------------------------------------------------------------------------
__host__ __device__ constexpr bool digits_fmt(int fmt) { return fmt == FMT_Q4K || fmt == FMT_Q6K || fmt == FMT_Q8_0; }
constexpr int HW = 7;  // 16-byte words per chunk

// place of element i in the eo order of a chunk, in bytes
__device__ __forceinline__ int eo_place(int i)
{
    const int o = i & 7;  // 0 4 1 5 2 6 3 7
    return (i & 24) | ((o & 2) << 1) | ((o & 1) << 1) | (o >> 2);
}

// One value per lane, 32 lanes (one half of a wave) a chunk: writes the chunk
// `out` (HW words).  All 32 lanes of the half take part.
__device__ __forceinline__ void write_digits(float h, uint4 *__restrict__ out, bool eo)
{
    const int i = threadIdx.x & 31;
    const float sum = plain_sum<4>(plain_sum<3>(plain_sum<2>(plain_sum<1>(plain_sum<0>(h)))));
    float m = fabsf(h), lo, hi;
    m = fmaxf(m, dpp<0xB1>(m));
    m = fmaxf(m, dpp<0x4E>(m));
    m = fmaxf(m, dpp<0x124>(m));
    m = fmaxf(m, dpp<0x128>(m));
    swap_rows(m, lo, hi);
    m = fmaxf(lo, hi);
    int e = m > 0.0f ? 23 - __builtin_amdgcn_frexp_expf(m) : 0;  // m 2^e in [2^22, 2^23)
    if (__builtin_amdgcn_ldexpf(m, e) > 8355711.0f)              // 127 (65536 + 256 + 1): the largest v
        e--;
    e = min(e, 126);  // keeps 2^-e normal (such a chunk is below 2^-103)
    const int v = (int)rintf(__builtin_amdgcn_ldexpf(h, e));
    const int d0 = (int8_t)v, v1 = (v - d0) >> 8, d1 = (int8_t)v1, d2 = (v1 - d1) >> 8;
    int8_t *b = reinterpret_cast<int8_t *>(out) + (eo ? eo_place(i) : i);
    b[0] = (int8_t)d0;
    b[32] = (int8_t)d1;
    b[64] = (int8_t)d2;
    // whole numbers hold no infinity and no NaN: the chunk's unit does
    const bool finite = m < INFINITY && sum == sum;
    if (i == 0)
        *reinterpret_cast<float2 *>(out + 6) = make_float2(finite ? __builtin_amdgcn_ldexpf(1.0f, -e) : NAN, sum);
}

struct Digits {
    uint32_t d[3][8];
    float unit, sum;  // 2^-e and sum of h, both times the choice's weight
};

__device__ __forceinline__ int dot4(uint32_t a, uint32_t b, int c) { return __builtin_amdgcn_sdot4((int)a, (int)b, c, false); }

// 65536 s2 + 256 s1 + s0.  256 s2 + s1 is a whole number below 2^24 for Q4K (32
// products of 4 and 8 bits), exact in fp32, so that only the sum rounds; for Q6K
// (16 of 8 and 8 bits) and Q8_0 (32 of them) it reaches 2^26 and 2^27 and its
// conversion rounds as well, by 2^-24 of the value.
__device__ __forceinline__ float digit_sum(int s2, int s1, int s0) { return fmaf((float)((s2 << 8) + s1), 256.0f, (float)s0); }

template <int FMT>
__device__ __forceinline__ float dot(const Raw<FMT> &r, int c, const Digits &x)
{
    int s0 = 0, s1 = 0, s2 = 0;
    if constexpr (FMT == FMT_Q4K) {
        float S, Mn;
        q4k_scales(r.h, c & 7, S, Mn);
        const uint32_t cw[4] = {r.c.x, r.c.y, r.c.z, r.c.w};
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const uint32_t lo = cw[q] & 0x0F0F0F0Fu, hi = (cw[q] >> 4) & 0x0F0F0F0Fu;
            s0 = dot4(lo, x.d[0][2 * q], s0), s0 = dot4(hi, x.d[0][2 * q + 1], s0);
            s1 = dot4(lo, x.d[1][2 * q], s1), s1 = dot4(hi, x.d[1][2 * q + 1], s1);
            s2 = dot4(lo, x.d[2][2 * q], s2), s2 = dot4(hi, x.d[2][2 * q + 1], s2);
        }
        return fmaf(S * x.unit, digit_sum(s2, s1, s0), -Mn * x.sum);
    } else if constexpr (FMT == FMT_Q6K) {
        const uint32_t lw[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w};
        const uint32_t hw[2] = {r.hi.x, r.hi.y};
        float t[2];
#pragma unroll
        for (int q = 0; q < 4; q++) {
            uint32_t lo, hi;
            q6k_bytes(lw[q], hw[q >> 1] >> (8 * (q & 1)), lo, hi);
            if (q == 2)
                t[0] = digit_sum(s2, s1, s0), s0 = s1 = s2 = 0;
            s0 = dot4(lo, x.d[0][2 * q], s0), s0 = dot4(hi, x.d[0][2 * q + 1], s0);
            s1 = dot4(lo, x.d[1][2 * q], s1), s1 = dot4(hi, x.d[1][2 * q + 1], s1);
            s2 = dot4(lo, x.d[2][2 * q], s2), s2 = dot4(hi, x.d[2][2 * q + 1], s2);
        }
        t[1] = digit_sum(s2, s1, s0);
        const float Sa = (float)(int8_t)r.sc2, Sb = (float)(int8_t)(r.sc2 >> 8);
        return 0.25f * f16_bits_to_f32(r.d) * x.unit * fmaf(Sa, t[0], Sb * t[1]);
    } else {
        const uint32_t cw[8] = {r.c0.x, r.c0.y, r.c0.z, r.c0.w, r.c1.x, r.c1.y, r.c1.z, r.c1.w};
#pragma unroll
        for (int i = 0; i < 8; i++) {
            s0 = dot4(cw[i], x.d[0][i], s0);
            s1 = dot4(cw[i], x.d[1][i], s1);
            s2 = dot4(cw[i], x.d[2][i], s2);
        }
        return f16_bits_to_f32(r.d) * x.unit * digit_sum(s2, s1, s0);
    }
}

constexpr int MAXG = 16;  // groups of R rows per workgroup

// Groups 0 .. groups - 1 of R rows: `load(g, rows)` issues a group's loads,
// `ready()` runs once they are out (the activations' set-up), `use(g, rows)`
// consumes them while the next group's are in flight.
template <typename RowsT, typename L, typename P, typename U>
__device__ __forceinline__ void walk(int groups, L load, P ready, U use)
{
    RowsT a;
    load(0, a);
    ready();
    for (int g = 0; g + 1 < groups; g++) {
        RowsT b;
        load(g + 1, b);
        use(g, a);
        a = b;
    }
    use(groups - 1, a);
}

// A workgroup computes the 32 values of one chunk of H: KS waves along a row
// (each a chunk of the row per lane and pass) times RW waves of 32 / RW rows.
// HMODE: 0 fp32, 1 digits in natural order, 2 digits in eo order.
// Bound by the weights' bytes.  One token, two experts of 14336 x 4096 Q4K (132
// MB): 26 us, 5.0 TB/s (a plain read of that size reaches 6.9); eight of 768 x
// 2048 Q8_0 (27 MB): 11 us, of which launch, ramp and the sums across lanes are
// most.  A wave keeps its chunk of X in registers over all its rows and has the
// next two rows' loads in flight; with four rows in flight registers spill.
template <int FMT, int R, int HMODE>
__global__ __launch_bounds__(512) void moe_glu_kernel(Mat wg, Mat wu, const uint16_t *__restrict__ X,
                                                       const int32_t *__restrict__ ids, void *__restrict__ H, int E, int k,
                                                       int64_t F, int act, int KS)
{
    constexpr bool PAIRS = FMT == FMT_Q4K;
    __shared__ float part[8][2 * 32];  // [wave along the row][row, gate and up], 32 rows
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6, RW = waves / KS;
    const int kw = wave % KS, rw = wave / KS, rows = 32 / RW, groups = rows / R;
    const int pair = blockIdx.y, t = pair / k;
    const int e = ids[pair];
    if (e < 0 || e >= E)
        return;  // no expert: H of the pair is never read
    const int64_t f0 = (int64_t)blockIdx.x * 32;  // F is a multiple of 32
    const int64_t row0 = (int64_t)e * F + f0 + rw * rows;
    const int C = (int)(wg.K / 32);
    for (int c0 = kw * 64; c0 < C; c0 += KS * 64) {
        const bool live = c0 + lane < C;
        const int c = live ? c0 + lane : C - 1;  // lanes past the row: a zero activation
        const uint4 *xp = reinterpret_cast<const uint4 *>(X + (int64_t)t * wg.K + 32 * (int64_t)c);
        uint4 xq[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            xq[i] = xp[i];
        Acts<PAIRS> x;
        struct Rows {
            Raw<FMT> g[R], u[R];
        };
        const At<FMT> pg = at_row<FMT>(wg, row0, c, lane), pu = at_row<FMT>(wu, row0, c, lane);
        auto load = [&](int g, Rows &w) {
#pragma unroll
            for (int r = 0; r < R; r++) {
                load_raw<FMT>(wg, pg, g * R + r, w.g[r]);
                load_raw<FMT>(wu, pu, g * R + r, w.u[r]);
            }
        };
        auto ready = [&] {
            {  // after the first loads are out
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint32_t keep = live ? ~0u : 0u;
                    const uint32_t v[4] = {xq[i].x & keep, xq[i].y & keep, xq[i].z & keep, xq[i].w & keep};
                    if constexpr (PAIRS) {
                        x.p[4 * i] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100u);
                        x.p[4 * i + 1] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302u);
                        x.p[4 * i + 2] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100u);
                        x.p[4 * i + 3] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302u);
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            sum = dot2(v[j], 0x3F803F80u, sum);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            x.a[8 * i + 2 * j] = bf16_lo(v[j]);
                            x.a[8 * i + 2 * j + 1] = bf16_hi(v[j]);
                        }
                    }
                }
                if constexpr (PAIRS)
                    x.sum = sum;
            }
        };
        auto use = [&](int g, const Rows &w) {
            float v[2 * R];
#pragma unroll
            for (int r = 0; r < R; r++) {
                v[r] = dot<FMT, PAIRS>(wg, w.g[r], c, x);
                v[R + r] = dot<FMT, PAIRS>(wu, w.u[r], c, x);
            }
            const float tot = wave_sums<2 * R>(v, lane);
            if (lane < 2 * R) {
                const int i = sum_index<2 * R>(lane);  // gate rows, then up rows
                float &p = part[kw][(i >= R ? 32 : 0) + rw * rows + g * R + i % R];
                p = c0 == kw * 64 ? tot : p + tot;
            }
        };
        walk<Rows>(groups, load, ready, use);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        float gs = 0.0f, us = 0.0f;
        for (int w = 0; w < KS; w++) {
            gs += part[w][threadIdx.x];
            us += part[w][32 + threadIdx.x];
        }
        const float h = act_f32(act, gs) * us;
        if constexpr (HMODE == 0)
            static_cast<float *>(H)[(int64_t)pair * F + f0 + threadIdx.x] = h;
        else
            write_digits(h, static_cast<uint4 *>(H) + HW * (pair * (F / 32) + blockIdx.x), HMODE == 2);
    }
}

// Rows n0 .. of Y for token blockIdx.y: lane l of a wave holds chunks l, l +
// 64 KS, .. of the k choices' rows laid end to end, so that short rows of F
// still fill whole waves and no partial result goes through memory.  Bound by
// the weights' bytes and, near them, by the decode (digits: 122 -> 65 VALU
// instructions a chunk, 47 -> 17 us): two experts of 4096 x 14336 Q4K (66 MB)
// 16.5 us, 4.0 TB/s; eight of 2048 x 768 Q8_0 (13 MB) 6 us.
template <int FMT, int R>
__global__ __launch_bounds__(512) void moe_down_kernel(Mat wd, const void *__restrict__ H,
                                                        const int32_t *__restrict__ ids, const float *__restrict__ weights,
                                                        float *__restrict__ Y, int E, int k, int64_t K, int groups)
{
    constexpr bool DIG = digits_fmt(FMT);
    __shared__ float part[MAXG][8][R];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), KS = blockDim.x >> 6;
    const int t = blockIdx.y;
    const int64_t n0 = (int64_t)blockIdx.x * (groups * R);
    const int left = (int)(K - n0 < groups * R ? K - n0 : groups * R);  // rows there are
    const int CF = (int)(wd.K / 32), items = k * CF;
    for (int i0 = wave * 64; i0 < items; i0 += KS * 64) {
        const int it = min(i0 + lane, items - 1);
        const int slot = (int)((unsigned)it / (unsigned)CF), c = it - slot * CF;
        int e = ids[t * k + slot];
        const bool live = i0 + lane < items && e >= 0 && e < E;
        // (H of a choice without an expert was never written: whatever is there
        // is replaced by zero)
        const float wt = live ? weights[t * k + slot] : 0.0f;
        e = live ? e : 0;
        const int64_t chunk = ((int64_t)t * k + slot) * CF + c;
        const uint4 *hp = static_cast<const uint4 *>(H) + (DIG ? HW : 8) * chunk;
        uint4 hq[DIG ? HW : 8];
#pragma unroll
        for (int i = 0; i < (DIG ? HW : 8); i++)
            hq[i] = hp[i];
        std::conditional_t<DIG, Digits, Acts<false>> x;
        struct Rows {
            Raw<FMT> w[R];
        };
        const At<FMT> pd = at_row<FMT>(wd, (int64_t)e * K + n0, c, lane);
        auto load = [&](int g, Rows &w) {
#pragma unroll
            for (int r = 0; r < R; r++)
                load_raw<FMT>(wd, pd, g * R + r < left ? g * R + r : left - 1, w.w[r]);
        };
        auto ready = [&] {
            {
                if constexpr (DIG) {
#pragma unroll
                    for (int j = 0; j < 3; j++) {
                        x.d[j][0] = hq[2 * j].x, x.d[j][1] = hq[2 * j].y, x.d[j][2] = hq[2 * j].z, x.d[j][3] = hq[2 * j].w;
                        x.d[j][4] = hq[2 * j + 1].x, x.d[j][5] = hq[2 * j + 1].y, x.d[j][6] = hq[2 * j + 1].z,
                        x.d[j][7] = hq[2 * j + 1].w;
                    }
                    x.unit = live ? __uint_as_float(hq[6].x) * wt : 0.0f;
                    x.sum = live ? __uint_as_float(hq[6].y) * wt : 0.0f;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        x.a[4 * i] = live ? __uint_as_float(hq[i].x) * wt : 0.0f;
                        x.a[4 * i + 1] = live ? __uint_as_float(hq[i].y) * wt : 0.0f;
                        x.a[4 * i + 2] = live ? __uint_as_float(hq[i].z) * wt : 0.0f;
                        x.a[4 * i + 3] = live ? __uint_as_float(hq[i].w) * wt : 0.0f;
                    }
                }
            }
        };
        auto use = [&](int g, const Rows &w) {
            float v[R];
#pragma unroll
            for (int r = 0; r < R; r++) {
                if constexpr (DIG)
                    v[r] = dot<FMT>(w.w[r], c, x);
                else
                    v[r] = dot<FMT, false>(wd, w.w[r], c, x);
            }
            const float tot = wave_sums<R>(v, lane);
            if (lane < R) {
                float &p = part[g][wave][sum_index<R>(lane)];
                p = i0 == wave * 64 ? tot : p + tot;
            }
        };
        walk<Rows>(groups, load, ready, use);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < groups * R; i += blockDim.x) {
        float s = 0.0f;
        for (int w = 0; w < KS; w++)
            s += part[i / R][w][i % R];
        if (n0 + i < K)
            Y[(int64_t)t * K + n0 + i] = s;
    }
}

// ---------------------------------------------------------------------------
// More tokens: sort the pairs by expert.  One workgroup; counts and cursors
// in LDS.  The order of an expert's pairs varies from run to run, but a
// pair's results do not depend on its place.  4.7 us for 48 pairs, 18 us for
// 4096 (beside the preparation of X), and in proportion beyond, where the
// products grow as fast.
// ---------------------------------------------------------------------------
struct Plan {
    int32_t *tiles;   // [4]: numbers of tiles and of pairs with an expert; then {expert, first, count, 0} per tile
    int32_t *pair;    // sorted place -> pair
    int32_t *place;   // pair -> sorted place, -1 without an expert
};
constexpr int MAXE = 1024;

__device__ void plan_block(const int32_t *__restrict__ ids, int P, int E, int BM, const Plan &pl)
{
    __shared__ int cnt[MAXE], off[MAXE], til[MAXE], scan[2][1024];
    const int tid = threadIdx.x;
    cnt[tid] = 0;
    __syncthreads();
    for (int p = tid; p < P; p += 1024) {
        const int e = ids[p];
        if (e >= 0 && e < E)
            atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    // inclusive scans of the counts and of the tile counts
    const int c = cnt[tid], nt = (c + BM - 1) / BM;
    scan[0][tid] = c;
    scan[1][tid] = nt;
    __syncthreads();
    for (int s = 1; s < 1024; s <<= 1) {
        const int a = tid >= s ? scan[0][tid - s] : 0, b = tid >= s ? scan[1][tid - s] : 0;
        __syncthreads();
        scan[0][tid] += a;
        scan[1][tid] += b;
        __syncthreads();
    }
    off[tid] = scan[0][tid] - c;
    til[tid] = scan[1][tid] - nt;
    if (tid == 1023) {
        pl.tiles[0] = scan[1][tid];
        pl.tiles[1] = scan[0][tid];
    }
    cnt[tid] = 0;
    int4 *tl = reinterpret_cast<int4 *>(pl.tiles + 4);
    for (int i = 0; i < nt; i++)
        tl[til[tid] + i] = make_int4(tid, off[tid] + i * BM, min(BM, c - i * BM), 0);
    __syncthreads();
    for (int p = tid; p < P; p += 1024) {
        const int e = ids[p];
        int at = -1;
        if (e >= 0 && e < E) {
            at = off[e] + atomicAdd(&cnt[e], 1);
            pl.pair[at] = p;
        }
        pl.place[p] = at;
    }
}

__global__ __launch_bounds__(1024) void moe_plan_kernel(const int32_t *__restrict__ ids, int P, int E, int BM, Plan pl)
{
    plan_block(ids, P, E, BM, pl);
}

// Y[t] = sum_j w[t][j] * P[place of (t, j)], in the order of j.  Bytes: 2048
// tokens of 4096, two choices: 101 MB in 18 us, 5.5 TB/s.
__global__ __launch_bounds__(256) void moe_join_kernel(const float *__restrict__ Pd, const int32_t *__restrict__ place,
                                                       const float *__restrict__ weights, float *__restrict__ Y, int k,
                                                       int64_t K)
{
    const int t = blockIdx.x;
    const int64_t n = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 4;
    if (n >= K)
        return;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int j = 0; j < k; j++) {
        const int at = place[(int64_t)t * k + j];
        if (at < 0)
            continue;
        const float w = weights[(int64_t)t * k + j];
        const float4 v = *reinterpret_cast<const float4 *>(Pd + (int64_t)at * K + n);
        s.x = fmaf(w, v.x, s.x);
        s.y = fmaf(w, v.y, s.y);
        s.z = fmaf(w, v.z, s.z);
        s.w = fmaf(w, v.w, s.w);
    }
    *reinterpret_cast<float4 *>(Y + (int64_t)t * K + n) = s;
}

// ---------------------------------------------------------------------------
// Grouped matrix-core products.  A workgroup of four waves takes one tile of
// up to 16 TM pairs of an expert and 64 NT rows of its weights; the pairs'
// activations are staged in LDS in slabs of 128 (double buffered) and shared
// by the waves.  Lane (g, r) decodes block 4 s + g of its rows in slab s
// (dequant8, exact in fp32) and feeds four v_mfma_f32_16x16x32_bf16 steps
// whose k order inside the slab is the same on both operands.  Each fp32
// value enters as a bf16 pair hi + lo (16 bits of it): weights as hi and lo,
// X is bf16 already, H as hi and lo, dropping lo * lo; error at most about
// 2^-16 of sum |w||x|.  Bound by the decode (dequant8 and the bf16 split of
// every weight): 32 experts of 768 x 2048 Q5K, four a token, 256 tokens: 127 us
// for the whole layer; 8 of 4096 x 4096 Q4_0, two a token, 32 tokens: 204 us.
// ---------------------------------------------------------------------------
constexpr int SLAB = 128, PITCH = 2 * SLAB + 16;

__device__ __forceinline__ void split_bf16(float a, float b, uint32_t &hi, uint32_t &lo)
{
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const b2 h = {(__bf16)a, (__bf16)b};
    hi = __builtin_bit_cast(uint32_t, h);
    const b2 l = {(__bf16)(a - (float)h.x), (__bf16)(b - (float)h.y)};
    lo = __builtin_bit_cast(uint32_t, l);
}

// GLU: X rows are gathered by pair, rows i < NT / 2 of a wave's row tiles are
// gate rows and the others the same rows of up; writes H hi / lo.  Otherwise:
// A = H by sorted place, writes Pd.
template <int FMT, int TM, int NT, bool GLU>
__global__ __launch_bounds__(256) void moe_gemm_kernel(Mat w0, Mat w1, const uint16_t *__restrict__ A,
                                                       const uint16_t *__restrict__ Alo, Plan pl, int k, int64_t N, int act,
                                                       uint16_t *__restrict__ Hhi, uint16_t *__restrict__ Hlo,
                                                       float *__restrict__ Pd)
{
    constexpr int BM = 16 * TM, PL = GLU ? 1 : 2;  // planes of A
    constexpr int NF = GLU ? NT / 2 : NT;          // row tiles of outputs per wave
    static_assert(!GLU || NT % 2 == 0, "gate and up tiles");
    __shared__ __attribute__((aligned(16))) uint8_t sX[2][PL][BM * PITCH];
    if ((int)blockIdx.x >= pl.tiles[0])
        return;
    const int4 tile = reinterpret_cast<const int4 *>(pl.tiles + 4)[blockIdx.x];
    const int expert = tile.x, first = tile.y, count = tile.z;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g = lane >> 4, r16 = lane & 15;
    const int64_t K = w0.K, n_wave = (int64_t)blockIdx.y * (64 * NF) + wave * 16 * NF;
    const int nslab = (int)((K + SLAB - 1) / SLAB);
    const int blocks = (int)(K / 32);
    int64_t wpiece[NT];
#pragma unroll
    for (int i = 0; i < NT; i++)
        wpiece[i] = ((int64_t)expert * N + min(n_wave + 16 * (i % NF) + r16, N - 1)) * (K / 8);
    // rows of A this thread stages: 16 pieces of 8 per row and slab
    int64_t arow[TM];
    bool alive[TM];
#pragma unroll
    for (int t = 0; t < TM; t++) {
        const int row = (tid + 256 * t) / 16;
        alive[t] = row < count;
        const int at = first + (alive[t] ? row : 0);
        arow[t] = GLU ? (int64_t)(pl.pair[at] / k) : at;
    }
    const int q8 = 8 * (tid & 15);
    uint4 xr[PL][TM];
    auto load_x = [&](int s) {
#pragma unroll
        for (int t = 0; t < TM; t++) {
            const bool in = alive[t] && s * SLAB + q8 < K;
#pragma unroll
            for (int p = 0; p < PL; p++)
                xr[p][t] = in ? *reinterpret_cast<const uint4 *>((p ? Alo : A) + arow[t] * K + s * SLAB + q8)
                              : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    auto store_x = [&](int buf) {
#pragma unroll
        for (int t = 0; t < TM; t++)
#pragma unroll
            for (int p = 0; p < PL; p++)
                *reinterpret_cast<uint4 *>(&sX[buf][p][((tid + 256 * t) / 16) * PITCH + 2 * q8]) = xr[p][t];
    };
    f32x4_t acc[NT][TM];
#pragma unroll
    for (int i = 0; i < NT; i++)
#pragma unroll
        for (int j = 0; j < TM; j++)
            acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    load_x(0);
    store_x(0);
    if (nslab > 1)
        load_x(1);
    lds_barrier();
    for (int s = 0; s < nslab; s++) {
        const int buf = s & 1;
        const int blk = min(4 * s + g, blocks - 1);  // past the row: the A operand is zero
#pragma unroll
        for (int i = 0; i < NT; i++) {
            const Mat &w = GLU && i >= NF ? w1 : w0;
#pragma unroll
            for (int t = 0; t < 4; t++) {
                float v[8];
                dequant8<FMT>(w.B, w.p, wpiece[i] + 4 * blk + t, v);
                uint32_t h[4], l[4];
#pragma unroll
                for (int e = 0; e < 4; e++)
                    split_bf16(v[2 * e], v[2 * e + 1], h[e], l[e]);
                const bf16x8_t bh = __builtin_bit_cast(bf16x8_t, make_uint4(h[0], h[1], h[2], h[3]));
                const bf16x8_t bl = __builtin_bit_cast(bf16x8_t, make_uint4(l[0], l[1], l[2], l[3]));
#pragma unroll
                for (int j = 0; j < TM; j++) {
                    const int at = (16 * j + r16) * PITCH + 64 * g + 16 * t;
                    const bf16x8_t xh = *reinterpret_cast<const bf16x8_t *>(&sX[buf][0][at]);
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bh, xh, acc[i][j], 0, 0, 0);
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bl, xh, acc[i][j], 0, 0, 0);
                    if constexpr (!GLU) {
                        const bf16x8_t xl = *reinterpret_cast<const bf16x8_t *>(&sX[buf][PL - 1][at]);
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bh, xl, acc[i][j], 0, 0, 0);
                    }
                }
            }
        }
        if (s + 1 < nslab) {
            store_x(buf ^ 1);
            if (s + 2 < nslab)
                load_x(s + 2);
        }
        lds_barrier();
    }
    // lane holds D[row 4 g + i][pair r16] of each 16 x 16 tile: four
    // consecutive outputs of one pair (N is a multiple of 32, so all or none exist)
#pragma unroll
    for (int j = 0; j < TM; j++) {
        const int m = 16 * j + r16;
        if (m >= count)
            continue;
        const int64_t at = (int64_t)(first + m) * N;
#pragma unroll
        for (int i = 0; i < NF; i++) {
            const int64_t n = n_wave + 16 * i + 4 * g;
            if (n >= N)
                continue;
            if constexpr (GLU) {
                float h[4];
#pragma unroll
                for (int e = 0; e < 4; e++)
                    h[e] = act_f32(act, acc[i][j][e]) * acc[i + NF][j][e];
                uint2 hi, lo;
                split_bf16(h[0], h[1], hi.x, lo.x);
                split_bf16(h[2], h[3], hi.y, lo.y);
                *reinterpret_cast<uint2 *>(Hhi + at + n) = hi;
                *reinterpret_cast<uint2 *>(Hlo + at + n) = lo;
            } else {
                *reinterpret_cast<float4 *>(Pd + at + n) = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Grouped products of the tuned formats (Q4K, Q6K, Q8_0) on
// v_mfma_f32_16x16x32_f16.  Weights enter as whole numbers, which fp16 holds
// exactly, and their scales multiply fp32 sums of products:
//   Q4K   sc * u <= 63 * 15 as one operand, scale d per 256; the minimums as
//         one more product per slab of 128 (bf16): m times the sums of the
//         activations over the blocks of 32;
//   Q6K   sc * q has 13 bits, so sc = 16 sh + sl and two operands, 16 sh q and
//         sl q; scale d per 256;
//   Q8_0  q as one operand, scale d per 32.
// So X costs one product per weight (Q6K two) where a bf16 pair per weight
// costs two, and only sums round.
// Activations are fp16 times a power of two per row (row maximum in [2^14,
// 2^15)): every bf16 value of X down to 2^-31 of its token's largest is exact
// (its last bit is at least fp16's 2^-24), a smaller one is off by at most 2^-25,
// 2^-39 of that largest; H is a pair of fp16, 22 significant bits, and the same
// 2^-39 of the row's largest.
//
// k order: for Q4K and Q6K lane (g, r) holds block 4 s + g of row r in slab s
// (one 16-byte load of codes) and step t multiplies octet t of the four
// blocks; for Q8_0, whose scale is per block, step t is block 4 s + t.
//
// D[m = 4 g + i][n = r]: tokens are the A operand, so that a lane's results
// belong to the row whose scales it holds.
//
// Two kernels.  moe_thin_kernel, tiles of 16 pairs, for few pairs an expert: the
// waves read X from the caches straight into operands, there is no barrier
// in the loop, and the weights stream; waves split a row and add their sums
// through LDS.  moe_wide_kernel:
// tiles of 64 pairs whose slabs are staged in LDS, double
// buffered, and shared by four waves of 64 rows each, so that a weight is
// decoded once per 64 pairs.
// ---------------------------------------------------------------------------
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pk(float a, float b) { return __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)a, (_Float16)b}); }
__device__ __forceinline__ f16x2_t h2(uint32_t v) { return __builtin_bit_cast(f16x2_t, v); }
__device__ __forceinline__ uint32_t u2(f16x2_t v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ f16x8_t h8(uint4 v) { return __builtin_bit_cast(f16x8_t, v); }
__device__ __forceinline__ uint32_t pkb(float a, float b) { return __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)a, (__bf16)b}); }

// v = h + m + l, three bf16 (24 significant bits)
__device__ __forceinline__ void split3(float v, float &h, float &m, float &l)
{
    h = (float)(__bf16)v;
    m = (float)(__bf16)(v - h);
    l = v - h - m;
}
// A block's sum of activations and its minimum's factor as the eight k of one
// MFMA step: h h m m h l 0 0 against H M H M L H 0 0, the products of three
// bf16 parts each down to 2^-24 of the whole.
__device__ __forceinline__ uint4 sum_entry(float v)
{
    float h, m, l;
    split3(v, h, m, l);
    return make_uint4(pkb(h, h), pkb(m, m), pkb(h, l), 0u);
}
__device__ __forceinline__ bf16x8_t min_entry(float v)
{
    float h, m, l;
    split3(v, h, m, l);
    return __builtin_bit_cast(bf16x8_t, make_uint4(pkb(h, m), pkb(h, m), pkb(l, h), 0u));
}

struct Acts16 {          // activations of a product
    const uint16_t *hi;  // [rows][pitch] fp16
    const uint16_t *lo;  // H only
    const uint4 *sums;   // [rows][pitch / 32]: sum_entry of the blocks
    const float *unit;   // [rows]: 2^-e
    int64_t pitch;       // a multiple of 256, zeros past the row's end
};

// What a lane loads of one row tile: the codes of a slab, and what a group of
// 256 (two slabs) shares.
template <int FMT> struct Codes16;
template <> struct Codes16<FMT_Q4K> { uint4 c; };
template <> struct Codes16<FMT_Q6K> { uint4 c; uint2 hi; uint32_t sc; };
template <> struct Codes16<FMT_Q8_0> { uint2 c[4]; uint32_t d[2]; };
template <int FMT> struct Head16 { };
template <> struct Head16<FMT_Q4K> { uint4 h; };
template <> struct Head16<FMT_Q6K> { uint32_t d; };

// One expert's matrix: the planes at its first row (the same for the whole
// wave) and 32-bit byte offsets of a lane's row in them, so that a slab's
// addresses are scalar additions.  launch_moe keeps an expert's planes below
// 2^31 bytes here.
struct Planes16 {
    const uint8_t *codes, *sc, *d;
    int K;
};
template <int FMT>
__device__ __forceinline__ Planes16 expert_planes(const Mat &w, int64_t row)
{
    Planes16 p;
    p.K = (int)w.K;
    if constexpr (FMT == FMT_Q4K) {
        p.codes = w.B + row * (w.K / 2);
        p.sc = w.B + w.p.scales + row * (w.K / 16);
        p.d = nullptr;
    } else if constexpr (FMT == FMT_Q6K) {
        p.codes = w.B + row * (w.K / 256 * 192);
        p.sc = w.B + w.p.scales + row * (w.K / 16);
        p.d = w.B + w.p.d + row * (w.K / 128);
    } else {
        p.codes = w.B + row * w.K;
        p.sc = nullptr;
        p.d = w.B + w.p.scales + row * (w.K / 16);
    }
    return p;
}
struct Row16 {
    uint32_t codes, sc, d;
};
template <int FMT>
__device__ __forceinline__ Row16 row_offsets(int K, int row, int g)
{
    const uint32_t r = (uint32_t)row, k = (uint32_t)K;
    if constexpr (FMT == FMT_Q4K)
        return Row16{r * (k / 2) + 16u * g, r * (k / 16), 0u};
    else if constexpr (FMT == FMT_Q6K)
        return Row16{r * (k / 256 * 192), r * (k / 16) + 2u * g, r * (k / 128)};
    else
        return Row16{r * k + 8u * g, 0u, r * (k / 16)};
}

// slab 2 G + u.  Q8_0 rows may end before a whole group: the last slab again
// past it, or, TAIL, where they end inside a slab, the last block (X is zero there)
// STREAM: read once (non-temporal), so that the lines of the scale planes, which
// serve many groups, stay in the caches
template <bool STREAM>
__device__ __forceinline__ uint4 codes16(const uint8_t *p)
{
    if constexpr (STREAM)
        return stream16(p);
    else
        return *reinterpret_cast<const uint4 *>(p);
}
template <int FMT, bool TAIL, bool STREAM>
__device__ __forceinline__ void load_codes(const Planes16 &w, const Row16 &r, int G, int u, int g, Codes16<FMT> &t)
{
    if constexpr (FMT == FMT_Q4K) {
        t.c = codes16<STREAM>(w.codes + 128 * G + 64 * u + r.codes);
    } else if constexpr (FMT == FMT_Q6K) {
        const uint8_t *c = w.codes + 192 * G + 64 * u, *h = w.codes + 192 * G + 128 + 32 * u;
        t.c = codes16<STREAM>(c + (r.codes + 16u * g));
        t.hi = *reinterpret_cast<const uint2 *>(h + (r.codes + 8u * g));
        t.sc = *reinterpret_cast<const uint16_t *>(w.sc + 16 * G + 8 * u + r.sc);
    } else if constexpr (!TAIL) {
        const int s = min(2 * G + u, w.K / 128 - 1);
#pragma unroll
        for (int i = 0; i < 4; i++)
            t.c[i] = *reinterpret_cast<const uint2 *>(w.codes + 128 * s + 32 * i + r.codes);
        const uint2 d = *reinterpret_cast<const uint2 *>(w.d + 8 * s + r.d);
        t.d[0] = d.x, t.d[1] = d.y;
    } else {
        uint32_t d[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int b = min(8 * G + 4 * u + i, w.K / 32 - 1);
            t.c[i] = *reinterpret_cast<const uint2 *>(w.codes + 32 * b + r.codes);
            d[i] = *reinterpret_cast<const uint16_t *>(w.d + 2 * b + r.d);
        }
        t.d[0] = d[0] | d[1] << 16, t.d[1] = d[2] | d[3] << 16;
    }
}
template <int FMT>
__device__ __forceinline__ void load_head(const Planes16 &w, const Row16 &r, int G, Head16<FMT> &t)
{
    if constexpr (FMT == FMT_Q4K)
        t.h = *reinterpret_cast<const uint4 *>(w.sc + 16 * G + r.sc);
    else if constexpr (FMT == FMT_Q6K)
        t.d = *reinterpret_cast<const uint16_t *>(w.d + 2 * G + r.d);
}

// (a & mask) | 0x64006400 in one instruction: the mask in a register, the
// constant in a scalar one (the compiler would use an and and an or with
// literals)
struct Nibbles {
    uint32_t low, next;  // 0x000F000F, 0x00F000F0
};
__device__ __forceinline__ Nibbles make_nibbles()
{
    Nibbles n;
    asm volatile("v_mov_b32 %0, 0x000f000f" : "=v"(n.low));
    asm volatile("v_mov_b32 %0, 0x00f000f0" : "=v"(n.next));
    return n;
}
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t c)
{
    uint32_t r;
    asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(mask), "s"(c));
    return r;
}

// The fp16 operands of steps 2 h, 2 h + 1 of a slab (h = 0, 1).  DROP (Q4K): where
// the group's scale is 0 its sub-scales count as 0 too, whatever they and the
// codes hold: the wide kernel's sums are multiplied by the last scale that is
// not 0.  2048 tokens, two of 8 experts of 14336 x 4096, whole layer: 2.68 ms
// with and without (boxes in turn, to 2 %); done in the head's dwords, once per
// group, 2.82 (spills), behind a branch 2.75.
template <int FMT> constexpr int PER = FMT == FMT_Q6K ? 2 : 1;  // operands per step
template <int FMT, bool DROP>
__device__ __forceinline__ void decode_half(const Nibbles &nb, const Codes16<FMT> &t, const Head16<FMT> &hd, int u, int g,
                                            int h, f16x8_t (&o)[2][PER<FMT>])
{
    if constexpr (FMT == FMT_Q4K) {
        const int j = 4 * u + g;
        uint32_t sc = __builtin_amdgcn_ubfe(hd.h.y, 4 * j, 4) | (__builtin_amdgcn_ubfe(hd.h.w, 2 * j, 2) << 4);
        if constexpr (DROP)
            sc = (hd.h.x & 0x7FFFu) ? sc : 0u;
        const _Float16 sh = (_Float16)(float)sc;
        const f16x2_t S = {sh, sh}, S16 = S * (_Float16)0.0625f, N = S * (_Float16)-1024.0f, N16 = S * (_Float16)-64.0f;
        const uint32_t cw[2] = {h ? t.c.z : t.c.x, h ? t.c.w : t.c.y};
#pragma unroll
        for (int q = 0; q < 2; q++) {
            // 1024 + u in the low nibbles' pairs, 1024 + 16 u in the next ones';
            // the fused multiply-adds leave sc u exactly
            const uint32_t a = cw[q], b = cw[q] >> 8;
            const f16x2_t p0 = __builtin_elementwise_fma(h2(and_or(a, nb.low, 0x64006400u)), S, N);
            const f16x2_t p1 = __builtin_elementwise_fma(h2(and_or(a, nb.next, 0x64006400u)), S16, N16);
            const f16x2_t p2 = __builtin_elementwise_fma(h2(and_or(b, nb.low, 0x64006400u)), S, N);
            const f16x2_t p3 = __builtin_elementwise_fma(h2(and_or(b, nb.next, 0x64006400u)), S16, N16);
            o[q][0] = h8(make_uint4(u2(p0), u2(p1), u2(p2), u2(p3)));
        }
    } else if constexpr (FMT == FMT_Q6K) {
        // one sub-scale per half: sc = 16 sh + sl; pairs 0, 2 hold q, pairs 1, 3 hold 16 q
        const int sc = (int)(int8_t)(h ? t.sc >> 8 : t.sc);
        const _Float16 hi16 = (_Float16)(float)(sc & ~15), lo16 = (_Float16)(float)(sc & 15);
        const f16x2_t Hs = {hi16, hi16}, Ls = {lo16, lo16}, Hs16 = Hs * (_Float16)0.0625f, Ls16 = Ls * (_Float16)0.0625f;
        const f16x2_t off1 = {(_Float16)-1056.0f, (_Float16)-1056.0f}, off16 = {(_Float16)-1536.0f, (_Float16)-1536.0f};
        const uint32_t cw[2] = {h ? t.c.z : t.c.x, h ? t.c.w : t.c.y}, hw = h ? t.hi.y : t.hi.x;
#pragma unroll
        for (int q = 0; q < 2; q++) {
            const uint32_t a = cw[q], b = cw[q] >> 8, H = hw >> (8 * q);
            const f16x2_t q0 = h2((a & 0x000F000Fu) | ((H << 4) & 0x00300030u) | 0x64006400u) + off1;
            const f16x2_t q1 = h2((a & 0x00F000F0u) | ((H << 6) & 0x03000300u) | 0x64006400u) + off16;
            const f16x2_t q2 = h2((b & 0x000F000Fu) | (H & 0x00300030u) | 0x64006400u) + off1;
            const f16x2_t q3 = h2((b & 0x00F000F0u) | ((H << 2) & 0x03000300u) | 0x64006400u) + off16;
            o[q][0] = h8(make_uint4(u2(q0 * Hs), u2(q1 * Hs16), u2(q2 * Hs), u2(q3 * Hs16)));
            o[q][1] = h8(make_uint4(u2(q0 * Ls), u2(q1 * Ls16), u2(q2 * Ls), u2(q3 * Ls16)));
        }
    } else {
        const f16x2_t off = {(_Float16)-1152.0f, (_Float16)-1152.0f};  // 1024 + 128 + q -> q
#pragma unroll
        for (int q = 0; q < 2; q++) {
            const uint32_t x = t.c[2 * h + q].x ^ 0x80808080u, y = t.c[2 * h + q].y ^ 0x80808080u;
            o[q][0] = h8(make_uint4(u2(h2(__builtin_amdgcn_perm(0x64646464u, x, 0x04010400u)) + off),
                                    u2(h2(__builtin_amdgcn_perm(0x64646464u, x, 0x04030402u)) + off),
                                    u2(h2(__builtin_amdgcn_perm(0x64646464u, y, 0x04010400u)) + off),
                                    u2(h2(__builtin_amdgcn_perm(0x64646464u, y, 0x04030402u)) + off)));
        }
    }
}

// scale of the group (Q4K, Q6K) or of the slab's block i (Q8_0)
template <int FMT>
__device__ __forceinline__ float scale_of(const Codes16<FMT> &t, const Head16<FMT> &hd, int i)
{
    if constexpr (FMT == FMT_Q4K)
        return f16_bits_to_f32(hd.h.x);
    else if constexpr (FMT == FMT_Q6K)
        return f16_bits_to_f32(hd.d);
    else
        return f16_bits_to_f32(t.d[i >> 1] >> (16 * (i & 1)));
}
// min_entry of a number that one bf16 holds
__device__ __forceinline__ bf16x8_t min_entry1(float v)
{
    const uint32_t h = __float_as_uint(v) >> 16;
    return __builtin_bit_cast(bf16x8_t, make_uint4(h, h, h << 16, 0u));
}
// Q4K: the 6-bit minimum of the lane's block of slab u
__device__ __forceinline__ float min_code(const Head16<FMT_Q4K> &t, int u, int g)
{
    const int j = 4 * u + g;
    return (float)(__builtin_amdgcn_ubfe(t.h.z, 4 * j, 4) | (__builtin_amdgcn_ubfe(t.h.w, 16 + 2 * j, 2) << 4));
}

// byte offset in a 256-byte slab of a row of activations: step t, lane group g
template <int FMT>
__device__ __forceinline__ int slab_at(int t, int g)
{
    return FMT == FMT_Q8_0 ? 64 * t + 16 * g : 64 * g + 16 * t;
}

// Direct global -> LDS loads: lane i's 16 bytes at base + off_i land at LDS
// address lds + 16 i (base and lds the same for the whole wave).  They write
// no register; every read of what they bring comes after an explicit wait for
// vmcnt 0 and a barrier.
typedef __attribute__((address_space(3))) void *lds_ptr_t;
__device__ __forceinline__ uint32_t lds_addr(const uint8_t *p) { return (uint32_t)(uintptr_t)(lds_ptr_t)p; }
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is a reserved name on a clobber list
__device__ __forceinline__ void dma16(const void *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds)
                 : "memory", "m0");
}
#pragma clang diagnostic pop
// This wave's direct loads are in -- all its loads but the last AFTER, which
// were issued after them (loads return in order) -- then the workgroup's.  The
// caller answers for those AFTER loads: they stand between the direct ones, which
// the compiler takes to change memory, and the barrier, and something uses their
// results, so that they are not dropped.  tests/test_moe_waits.py counts them in
// every instance of the built library.
template <int AFTER>
__device__ __forceinline__ void loads_barrier()
{
    static_assert(AFTER < 16, "low bits of vmcnt");
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0x0070 | AFTER);  // vmcnt AFTER, lgkmcnt 0
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

__device__ __forceinline__ f32x4_t mfma16(f16x8_t a, f16x8_t b, f32x4_t c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// Work order: the tiles of one expert share its weights and the blocks of one
// tile its activations, so each XCD (workgroup id modulo 8) takes a contiguous
// part of an order that walks `band` tiles across all blocks (2048 tokens, gate
// and up in Q4K, bands of 2, 8, 32 tiles: 1.54, 1.46, 1.51 ms).
struct Order {
    int nblk, band;
};
__device__ __forceinline__ bool place_of_block(int ntiles, const Order &o, int &tile, int &blk)
{
    const int64_t total = (int64_t)ntiles * o.nblk, per = (total + 7) / 8;
    const int64_t bid = blockIdx.x, at = (bid & 7) * per + (bid >> 3);
    if ((bid >> 3) >= per || at >= total)
        return false;
    const int band = (int)(at / ((int64_t)o.nblk * o.band));
    const int tiles = min(o.band, ntiles - o.band * band);
    const int in = (int)(at - (int64_t)band * o.nblk * o.band);
    blk = in / tiles;
    tile = o.band * band + in % tiles;
    return true;
}

// What the two kernels share: the tile, the rows, the results.
// GLU: row tiles i < NT / 2 are gate rows, the others the same rows of up;
// H[place][column] = act(gate) * up in fp32.
template <bool GLU, int NT, int TM>
__device__ __forceinline__ void store_results(const f32x4_t (&acc)[NT][TM], const Acts16 &x, const Plan &pl, int k, int first,
                                              int count, int64_t n_wave, int64_t N, int64_t pitch, int act,
                                              float *__restrict__ out)
{
    constexpr int NF = GLU ? NT / 2 : NT;
    const int lane = threadIdx.x & 63, g = lane >> 4, r16 = lane & 15;
#pragma unroll
    for (int j = 0; j < TM; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int m = 16 * j + 4 * g + e;
            if (m >= count)
                continue;
            const int at = first + m;
            const float u = x.unit[GLU ? pl.pair[at] / k : at];
#pragma unroll
            for (int i = 0; i < NF; i++) {
                const int64_t n = n_wave + 16 * i + r16;
                if constexpr (GLU) {
                    if (n < N)
                        out[at * pitch + n] = act_f32(act, acc[i][j][e] * u) * (acc[i + NF][j][e] * u);
                } else {
                    if (n < N)
                        out[at * pitch + n] = acc[i][j][e] * u;
                }
            }
        }
}

// Four waves: in the gate and up product two along a row times two of 16 NT / 2
// rows of gate and of up each, in the down product, whose rows are few and long,
// four along a row of the same 16 NT; their sums meet in LDS.  Bound by the
// weights' loads, which the decode of one slab only partly covers: 21 tokens,
// two of 8 experts of 14336 x 4096, gate and up in Q4K (528 MB) 176 us, 3.0
// TB/s; down in Q6K (385 MB) 163 us, 2.4 TB/s, where each weight also takes four
// products (two operands, H a pair).  Eight waves along a row of down: 182 us (a
// CU then holds one workgroup, and its start and end lie bare).  Gate and up with
// one, two, four waves along a row, 8 of 4096 x 4096 Q8_0, 48 tokens, whole
// layer: 244, 215, 207 us; 8 of 14336 x 4096 Q4K, 24 tokens: 293, 289, 306 us.
// The down product in Q4K, 21 tokens of the same (264 MB): 111 us, 2.4 TB/s; it
// takes 264 registers, so a CU holds one workgroup of it (Q6K: 220, two).
constexpr int thin_kw(bool glu) { return glu ? 2 : 4; }
template <int FMT, int TM, int NT, bool GLU, bool TAIL>
__global__ __launch_bounds__(256) void moe_thin_kernel(Mat w0, Mat w1, Acts16 x, Plan pl, int k, int64_t N,
                                                                  Order order, int act, float *__restrict__ out,
                                                                  int64_t out_pitch)
{
    constexpr int KW = thin_kw(GLU), RW = 4 / KW, NF = GLU ? NT / 2 : NT;
    // X a slab ahead; Q8_0's down product keeps its registers for the weights (8
    // experts of 4096 x 4096, 24 tokens: 168 -> 160 us without)
    constexpr bool AHEAD = GLU || FMT != FMT_Q8_0;
    __shared__ f32x4_t red[4 * NT * TM * 64];
    int ti, blk;
    if (!place_of_block(pl.tiles[0], order, ti, blk))
        return;
    const int4 tile = reinterpret_cast<const int4 *>(pl.tiles + 4)[ti];
    const int expert = tile.x, first = tile.y, count = tile.z;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, r16 = lane & 15;
    const int64_t K = w0.K, n_wave = ((int64_t)blk * RW + wave / KW) * (16 * NF);
    const int groups = (int)((K + 255) / 256);
    const int g0 = groups * (wave % KW) / KW, g1 = groups * (wave % KW + 1) / KW;
    const Planes16 e0 = expert_planes<FMT>(w0, expert * N), e1 = expert_planes<FMT>(w1, expert * N);
    Row16 wrow[NF];
#pragma unroll
    for (int i = 0; i < NF; i++)
        wrow[i] = row_offsets<FMT>((int)K, (int)min(n_wave + 16 * i + r16, N - 1), g);
    f32x4_t acc[NT][TM];
#pragma unroll
    for (int i = 0; i < NT; i++)
#pragma unroll
        for (int j = 0; j < TM; j++)
            acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const Nibbles nb = make_nibbles();
    // Q4K, Q6K: both slabs of a group at once, since only together are they whole
    // cache lines of the codes, which are gone from the caches a slab later
    // (fetching them one by one, and with the scale planes' lines evicted by
    // them, read twice the bytes).  A slab of Q8_0 is whole lines by itself.
    constexpr int RAWS = FMT == FMT_Q8_0 ? 1 : 2;
    Codes16<FMT> raw[RAWS][NT];
    Head16<FMT> rawh[NT];
    // after slab u of group G has been decoded: what takes its registers
    auto load_w = [&](int G, int next, int u, int i) {
        const Planes16 &e = GLU && i >= NF ? e1 : e0;
        if constexpr (RAWS == 1) {
            load_codes<FMT, TAIL, true>(e, wrow[i % NF], u == 0 ? G : next, 1 - u, g, raw[0][i]);
        } else if (u == 1) {
            load_codes<FMT, TAIL, true>(e, wrow[i % NF], next, 0, g, raw[0][i]);
            load_codes<FMT, TAIL, true>(e, wrow[i % NF], next, 1, g, raw[1][i]);
            load_head<FMT>(e, wrow[i % NF], next, rawh[i]);
        }
    };
    // the lane's token of each tile (past the end: the last one)
    const uint16_t *ahi[TM], *alo[TM];
    const uint4 *asum[TM];
#pragma unroll
    for (int j = 0; j < TM; j++) {
        const int at = first + min(16 * j + r16, count - 1);
        const int64_t row = GLU ? pl.pair[at] / k : at;
        ahi[j] = x.hi + row * x.pitch + slab_at<FMT>(0, g) / 2;
        alo[j] = x.lo + row * x.pitch + slab_at<FMT>(0, g) / 2;
        asum[j] = x.sums + row * (x.pitch / 32) + g;
    }
    struct Piece {
        f16x8_t h[TM][4], l[TM][4];
        bf16x8_t s[TM];
    };
    auto load_x = [&](int s, Piece &x16) {
#pragma unroll
        for (int j = 0; j < TM; j++) {
#pragma unroll
            for (int t = 0; t < 4; t++) {
                const int at = 128 * s + (slab_at<FMT>(t, 0) - slab_at<FMT>(0, 0)) / 2;
                x16.h[j][t] = *reinterpret_cast<const f16x8_t *>(ahi[j] + at);
                if constexpr (!GLU)
                    x16.l[j][t] = *reinterpret_cast<const f16x8_t *>(alo[j] + at);
            }
            if constexpr (FMT == FMT_Q4K)
                x16.s[j] = *reinterpret_cast<const bf16x8_t *>(asum[j] + 4 * s);
        }
    };
    Piece x16;
    if (g0 < g1) {
        load_x(2 * g0, x16);
#pragma unroll
        for (int i = 0; i < NT; i++)
            load_w(g0, g0, 1, i);
    }
    for (int G = g0; G < g1; G++) {
        const int next = min(G + 1, g1 - 1);
#pragma unroll
        for (int u = 0; u < 2; u++) {
            Piece nx;
            if constexpr (AHEAD) {
                load_x(u == 0 ? 2 * G + 1 : 2 * next, nx);
                __builtin_amdgcn_sched_barrier(0x81);  // loads stay before what follows
            }
            const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < NT; i++) {
                f16x8_t o[2][2][PER<FMT>];
                float d[4];
                decode_half<FMT, false>(nb, raw[u % RAWS][i], rawh[i], u, g, 0, o[0]);
                decode_half<FMT, false>(nb, raw[u % RAWS][i], rawh[i], u, g, 1, o[1]);
#pragma unroll
                for (int q = 0; q < (FMT == FMT_Q8_0 ? 4 : 1); q++)
                    d[q] = scale_of<FMT>(raw[u % RAWS][i], rawh[i], q);
                float dm = 0.0f;
                bf16x8_t mo;
                if constexpr (FMT == FMT_Q4K) {
                    dm = f16_bits_to_f32(rawh[i].h.x >> 16);
                    mo = min_entry1(min_code(rawh[i], u, g));
                }
                // a tile's codes are spent once decoded: the next ones have the
                // time of a slab or two to arrive
                load_w(G, next, u, i);
                __builtin_amdgcn_sched_barrier(0x81);
                f32x4_t p[TM];
#pragma unroll
                for (int j = 0; j < TM; j++) {
                    p[j] = zero;
#pragma unroll
                    for (int q = 0; q < 4; q++) {
#pragma unroll
                        for (int c = 0; c < PER<FMT>; c++) {
                            p[j] = mfma16(x16.h[j][q], o[q >> 1][q & 1][c], p[j]);
                            if constexpr (!GLU)
                                p[j] = mfma16(x16.l[j][q], o[q >> 1][q & 1][c], p[j]);
                        }
                        if constexpr (FMT == FMT_Q8_0) {
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                acc[i][j][e] = fmaf(d[q], p[j][e], acc[i][j][e]);
                            p[j] = zero;
                        }
                    }
                    if constexpr (FMT != FMT_Q8_0) {
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            acc[i][j][e] = fmaf(d[0], p[j][e], acc[i][j][e]);
                    }
                    if constexpr (FMT == FMT_Q4K) {
                        const f32x4_t q = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x16.s[j], mo, zero, 0, 0, 0);
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            acc[i][j][e] = fmaf(-dm, q[e], acc[i][j][e]);
                    }
                }
            }
            if constexpr (AHEAD)
                x16 = nx;
            else
                load_x(u == 0 ? 2 * G + 1 : 2 * next, x16);
        }
    }
    // the sums of the waves along a row, in order
#pragma unroll
    for (int i = 0; i < NT; i++)
#pragma unroll
        for (int j = 0; j < TM; j++)
            red[((wave * NT + i) * TM + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    if constexpr (!GLU) {  // wave w takes the result's w-th tile
        static_assert(KW == 4 && NT * TM == 4, "a tile per wave");
        f32x4_t v[1][1] = {{red[wave * 64 + lane]}};
#pragma unroll
        for (int w = 1; w < KW; w++)
            v[0][0] += red[(w * NT * TM + wave) * 64 + lane];
        const int i = wave / TM, j = wave % TM;
        store_results<false, 1, 1>(v, x, pl, k, first + 16 * j, count - 16 * j, n_wave + 16 * i, N, out_pitch, act, out);
    } else if (wave % KW == 0) {
#pragma unroll
        for (int w = 1; w < KW; w++)
#pragma unroll
            for (int i = 0; i < NT; i++)
#pragma unroll
                for (int j = 0; j < TM; j++)
                    acc[i][j] += red[(((wave + w) * NT + i) * TM + j) * 64 + lane];
        store_results<GLU, NT, TM>(acc, x, pl, k, first, count, n_wave, N, out_pitch, act, out);
    }
}

// Four waves of 16 NT rows over a tile of 16 TM pairs.  The accumulators hold
// the sum in units of the current scale D of each row (Q4K, Q6K): at a new
// group of 256 they are multiplied by D_old / D_new, which needs no second set
// of accumulators; a group of scale 0 keeps D, and its sub-scales count as 0.
// Q4K's minimums enter as -(dmin / D) m.  Q8_0 adds each block's products times
// its scale.
// Bound by the decode and the products sharing the SIMDs' issue: 2048 tokens,
// two of 8 experts of 14336 x 4096 Q4K: gate and up 1.41 ms (0.68 PFLOP/s), down
// 1.09 ms (two products per weight, H being a pair: 0.88 PFLOP/s of them).  515
// tokens, six of 64 experts of 1408 x 2048 Q8_0 (48 pairs an expert): 221 and 132
// us, half of it waits for weights and barriers.  Rows of Q8_0 that end inside a
// slab of 128 take the TAIL form, whose down product spills 220 bytes a lane and
// waits for them in the loop: the same with 1376 columns of H, 264 us (219 us
// gate and up, as with 1408).  Measured and not kept: tiles
// of 32 and of 128 pairs, 32 rows a wave, three buffers of X, streaming weight
// loads (the tiles of an expert share them in the caches).
template <int FMT, int TM, int NT, bool GLU, bool TAIL>
__global__ __launch_bounds__(256, 2) void moe_wide_kernel(Mat w0, Mat w1, Acts16 x, Plan pl, int k, int64_t N, Order order,
                                                          int act, float *__restrict__ out, int64_t out_pitch)
{
    constexpr int BM = 16 * TM, PL = GLU ? 1 : 2, NF = GLU ? NT / 2 : NT;
    constexpr bool SUMS = FMT == FMT_Q4K, RUN = FMT != FMT_Q8_0;
    // A buffer: per plane BM rows of 256 bytes, 16-byte piece c of row m at
    // place c ^ (m & 15), then the sums, BM rows of 64 bytes, piece c at c ^
    // ((m >> 2) & 3): the 16 rows that a read touches together lie in
    // different banks, and rows need no padding, which direct loads to LDS
    // could not write.
    constexpr int PLANE = BM * 256, BUF = PL * PLANE + (SUMS ? BM * 64 : 0);
    __shared__ __attribute__((aligned(16))) uint8_t smem[2 * BUF];
    int ti, blk;
    if (!place_of_block(pl.tiles[0], order, ti, blk))
        return;
    const int4 tile = reinterpret_cast<const int4 *>(pl.tiles + 4)[ti];
    const int expert = tile.x, first = tile.y, count = tile.z;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, r16 = lane & 15;
    const int64_t K = w0.K, n_wave = (int64_t)blk * (64 * NF) + wave * 16 * NF;
    const int groups = (int)((K + 255) / 256);
    const Planes16 e0 = expert_planes<FMT>(w0, expert * N), e1 = expert_planes<FMT>(w1, expert * N);
    Row16 wrow[NF];
#pragma unroll
    for (int i = 0; i < NF; i++)
        wrow[i] = row_offsets<FMT>((int)K, (int)min(n_wave + 16 * i + r16, N - 1), g);
    f32x4_t acc[NT][TM];
#pragma unroll
    for (int i = 0; i < NT; i++)
#pragma unroll
        for (int j = 0; j < TM; j++)
            acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    float D[NT];
#pragma unroll
    for (int i = 0; i < NT; i++)
        D[i] = 1.0f;
    const Nibbles nb = make_nibbles();
    // two slabs of codes in flight where they fit the registers
    constexpr int RAWS = FMT == FMT_Q4K ? 2 : 1;
    Codes16<FMT> raw[RAWS][NT];
    Head16<FMT> hd[NT], nhd[NT];
    auto load_c = [&](int G, int u) {
#pragma unroll
        for (int i = 0; i < NT; i++)
            load_codes<FMT, TAIL, false>(GLU && i >= NF ? e1 : e0, wrow[i % NF], G, u, g, raw[u % RAWS][i]);
    };
    auto load_h = [&](int G) {
#pragma unroll
        for (int i = 0; i < NT; i++)
            load_head<FMT>(GLU && i >= NF ? e1 : e0, wrow[i % NF], G, nhd[i]);
    };
    // Wave w stages rows 16 w TM / 4 .., four rows of 256 bytes a load, and
    // the sums of as many rows, 16 rows a load.
    const uint16_t *xb0 = GLU ? x.hi : x.hi + (int64_t)first * x.pitch, *xb1 = GLU ? nullptr : x.lo + (int64_t)first * x.pitch;
    const uint4 *xbs = GLU ? x.sums : x.sums + (int64_t)first * (x.pitch / 32);
    auto row_of = [&](int m) -> uint32_t {  // GLU: the token; otherwise the place in the tile
        const int in = min(m, count - 1);
        return (uint32_t)(GLU ? pl.pair[first + in] / k : in);
    };
    uint32_t xo[TM], so[TM / 4];
#pragma unroll
    for (int t = 0; t < TM; t++) {
        const int m = 4 * (TM * wave + t) + (lane >> 4);
        xo[t] = row_of(m) * (uint32_t)(2 * x.pitch) + 16u * ((lane & 15) ^ (m & 15));
    }
    static_assert(TM % 4 == 0, "a wave stages the sums of 4 TM rows, 16 a load");
    if constexpr (SUMS) {
#pragma unroll
        for (int t = 0; t < TM / 4; t++) {
            const int m = 16 * (TM / 4 * wave + t) + (lane >> 2);
            so[t] = row_of(m) * (uint32_t)(x.pitch / 2) + 16u * ((lane & 3) ^ ((m >> 2) & 3));
        }
    }
    auto load_x = [&](int s, int buf) {
        const uint32_t at = lds_addr(smem + buf * BUF) + 1024 * TM * wave;
#pragma unroll
        for (int t = 0; t < TM; t++) {
            dma16(xb0 + 128 * s, xo[t], at + 1024 * t);
            if constexpr (!GLU)
                dma16(xb1 + 128 * s, xo[t], at + PLANE + 1024 * t);
        }
        if constexpr (SUMS) {
#pragma unroll
            for (int t = 0; t < TM / 4; t++)
                dma16(xbs + 4 * s, so[t], lds_addr(smem + buf * BUF + PL * PLANE) + 1024 * (TM / 4 * wave + t));
        }
    };
    // operand pieces of the activations: step 2 h + q, tile j of the slab in sx
    struct Piece {
        f16x8_t h[2], l[2];
    };
    auto load_piece = [&](const uint8_t *sx, int h, int j, Piece &f) {
#pragma unroll
        for (int q = 0; q < 2; q++) {
            const uint8_t *p = sx + 256 * (16 * j + r16) + (slab_at<FMT>(2 * h + q, g) ^ (16 * r16));
            f.h[q] = *reinterpret_cast<const f16x8_t *>(p);
            if constexpr (!GLU)
                f.l[q] = *reinterpret_cast<const f16x8_t *>(p + PLANE);
        }
    };
    load_x(0, 0);
    load_c(0, 0);
    if constexpr (RAWS == 2)
        load_c(0, 1);
    load_h(0);
    loads_barrier<0>();
    // At least this many of a slab's weight loads are issued after its direct
    // loads and may still be on the way at its end (Q4K: a 16-byte load a row
    // tile, and the heads' in the first slab; the others have more).
    constexpr int AFTER0 = 2 * NT, AFTER1 = FMT == FMT_Q4K ? NT : 2 * NT;
    // (Not peeled: the last group's loads ahead count in its waits, and they are
    // there because the same code runs for every group, where the next one uses
    // them.  A use of them behind the loop instead: 2.67 -> 3.19 ms, spills.)
#pragma clang loop unroll(disable)
    for (int G = 0; G < groups; G++) {
        const int next = min(G + 1, groups - 1);
        float rD[NT];  // 1 / D
        if constexpr (RUN) {
#pragma unroll
            for (int i = 0; i < NT; i++) {
                hd[i] = nhd[i];
                const float d = scale_of<FMT>(raw[0][i], hd[i], 0), dn = d != 0.0f ? d : D[i];
                // D / dn to half a step: quotient and one correction
                rD[i] = __builtin_amdgcn_rcpf(dn);
                const float q0 = D[i] * rD[i], rho = fmaf(fmaf(-dn, q0, D[i]), rD[i], q0);
                D[i] = dn;
#pragma unroll
                for (int j = 0; j < TM; j++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        acc[i][j][e] *= rho;
            }
        }
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const uint8_t *sx = smem + u * BUF;
            // the next slab of X into the other buffer, whose readers are behind the
            // last barrier (past the end the last one again)
            load_x(min(2 * G + u + 1, 2 * groups - 1), 1 - u);
            Piece f[2];
            load_piece(sx, 0, 0, f[0]);
#pragma unroll
            for (int h = 0; h < 2; h++) {
                f16x8_t o[NT][2][PER<FMT>];
                float sc[NT][2];
#pragma unroll
                for (int i = 0; i < NT; i++) {
                    if constexpr (FMT == FMT_Q6K) {  // (as DROP, once per slab)
                        if (h == 0)
                            raw[0][i].sc = (hd[i].d & 0x7FFFu) ? raw[0][i].sc : 0u;
                    }
                    decode_half<FMT, FMT == FMT_Q4K>(nb, raw[u % RAWS][i], hd[i], u, g, h, o[i]);
                    if constexpr (!RUN) {
                        sc[i][0] = scale_of<FMT>(raw[u % RAWS][i], hd[i], 2 * h);
                        sc[i][1] = scale_of<FMT>(raw[u % RAWS][i], hd[i], 2 * h + 1);
                    }
                }
                if (h == 1) {  // these codes are spent: later ones take their registers
                    load_c(RAWS == 2 || u == 1 ? next : G, RAWS == 2 ? u : 1 - u);
                    if (u == 0)
                        load_h(next);
                }
#pragma unroll
                for (int j = 0; j < TM; j++) {
                    // the next piece is read before this one's products
                    const int at = h * TM + j;
                    if (at + 1 < 2 * TM)
                        load_piece(sx, (at + 1) / TM, (at + 1) % TM, f[(at + 1) & 1]);
                    if constexpr (!GLU)  // (GLU: fewer registers without it, 1.49 -> 1.41 ms at 2048 tokens)
                        __builtin_amdgcn_sched_barrier(0x16);  // VALU, SALU and VMEM may move across
                    const Piece &x16 = f[at & 1];
                    if constexpr (RUN) {
#pragma unroll
                        for (int q = 0; q < 2; q++)
#pragma unroll
                            for (int c = 0; c < PER<FMT>; c++) {
#pragma unroll
                                for (int i = 0; i < NT; i++)
                                    acc[i][j] = mfma16(x16.h[q], o[i][q][c], acc[i][j]);
                                if constexpr (!GLU) {
#pragma unroll
                                    for (int i = 0; i < NT; i++)
                                        acc[i][j] = mfma16(x16.l[q], o[i][q][c], acc[i][j]);
                                }
                            }
                    } else {
#pragma unroll
                        for (int q = 0; q < 2; q++) {
                            f32x4_t v[NT];
#pragma unroll
                            for (int i = 0; i < NT; i++)
                                v[i] = mfma16(x16.h[q], o[i][q][0], f32x4_t{0.0f, 0.0f, 0.0f, 0.0f});
                            if constexpr (!GLU) {
#pragma unroll
                                for (int i = 0; i < NT; i++)
                                    v[i] = mfma16(x16.l[q], o[i][q][0], v[i]);
                            }
#pragma unroll
                            for (int i = 0; i < NT; i++)
#pragma unroll
                                for (int e = 0; e < 4; e++)
                                    acc[i][j][e] = fmaf(sc[i][q], v[i][e], acc[i][j][e]);
                        }
                    }
                }
            }
            if constexpr (SUMS) {
                bf16x8_t mo[NT];
#pragma unroll
                for (int i = 0; i < NT; i++)
                    mo[i] = min_entry(-f16_bits_to_f32(hd[i].h.x >> 16) * min_code(hd[i], u, g) * rD[i]);
#pragma unroll
                for (int j = 0; j < TM; j++) {
                    const bf16x8_t xs = *reinterpret_cast<const bf16x8_t *>(sx + PL * PLANE + 64 * (16 * j + r16) + 16 * (g ^ ((r16 >> 2) & 3)));
#pragma unroll
                    for (int i = 0; i < NT; i++)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xs, mo[i], acc[i][j], 0, 0, 0);
                }
            }
            if (u == 0)
                loads_barrier<AFTER0>();
            else
                loads_barrier<AFTER1>();
        }
    }
    if constexpr (RUN) {
#pragma unroll
        for (int i = 0; i < NT; i++)
#pragma unroll
            for (int j = 0; j < TM; j++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    acc[i][j][e] *= D[i];
    }
    store_results<GLU, NT, TM>(acc, x, pl, k, first, count, n_wave, N, out_pitch, act, out);
}

// A row of `n` values as fp16 times 2^e (and, for fp32 rows, the rest of each
// value as a second fp16), its block sums, zeros up to `pitch`.  One workgroup.
template <bool F32>
__device__ void row_to_f16(const void *__restrict__ src, int n, int64_t pitch, uint16_t *__restrict__ hi,
                           uint16_t *__restrict__ lo, uint4 *__restrict__ sums, float *__restrict__ unit)
{
    __shared__ float wm[16];
    const int tid = threadIdx.x, n8 = n / 8, p8 = (int)(pitch / 8);
    auto read = [&](int i, float (&v)[8]) {
        if constexpr (F32) {
            const float4 a = static_cast<const float4 *>(src)[2 * i], b = static_cast<const float4 *>(src)[2 * i + 1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 a = static_cast<const uint4 *>(src)[i];
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; j++)
                v[2 * j] = bf16_lo(w[j]), v[2 * j + 1] = bf16_hi(w[j]);
        }
    };
    float m = 0.0f;
    for (int i = tid; i < n8; i += blockDim.x) {
        float v[8];
        read(i, v);
#pragma unroll
        for (int j = 0; j < 8; j++)
            m = fmaxf(m, fabsf(v[j]));
    }
#pragma unroll
    for (int s = 1; s < 64; s <<= 1)
        m = fmaxf(m, __shfl_xor(m, s));
    if ((tid & 63) == 0)
        wm[tid >> 6] = m;
    __syncthreads();
    for (int w = 0; w < (int)blockDim.x / 64; w++)
        m = fmaxf(m, wm[w]);
    int ex = m > 0.0f ? 15 - __builtin_amdgcn_frexp_expf(m) : 0;  // m 2^ex in [2^14, 2^15)
    ex = min(ex, 126);
    if (tid == 0)
        *unit = __builtin_amdgcn_ldexpf(1.0f, -ex);
    for (int i = tid; i < p8; i += blockDim.x) {
        float v[8], s = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++)
            v[j] = 0.0f;
        if (i < n8)
            read(i, v);
        uint32_t h[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float a = __builtin_amdgcn_ldexpf(v[2 * j], ex), b = __builtin_amdgcn_ldexpf(v[2 * j + 1], ex);
            const f16x2_t q = {(_Float16)a, (_Float16)b};
            h[j] = u2(q);
            if constexpr (F32)
                l[j] = pk(a - (float)q.x, b - (float)q.y);
            s += a + b;
        }
        *reinterpret_cast<uint4 *>(hi + 8 * (int64_t)i) = make_uint4(h[0], h[1], h[2], h[3]);
        if constexpr (F32)
            *reinterpret_cast<uint4 *>(lo + 8 * (int64_t)i) = make_uint4(l[0], l[1], l[2], l[3]);
        s += dpp<0xB1>(s);  // four threads a block of 32 (p8 is a multiple of 16: all four are here)
        s += dpp<0x4E>(s);
        if ((i & 3) == 0)
            sums[i >> 2] = sum_entry(s);
    }
}

// Block T sorts the pairs; block t < T prepares X[t].  2048 tokens of 4096: 18 us,
// the sort of their 4096 pairs.
__global__ __launch_bounds__(1024) void moe_prep_kernel(const int32_t *__restrict__ ids, int P, int E, int BM, Plan pl,
                                                        const uint16_t *__restrict__ X, int T, int64_t K,
                                                        uint16_t *__restrict__ xh, uint4 *__restrict__ sums,
                                                        float *__restrict__ unit, int64_t pitch)
{
    const int64_t t = blockIdx.x;
    if (t == T)
        plan_block(ids, P, E, BM, pl);
    else
        row_to_f16<false>(X + t * K, (int)K, pitch, xh + t * pitch, nullptr, sums + t * (pitch / 32), unit + t);
}

// H of the sorted pairs for the down product.  Bytes: 4096 pairs of 14336 (235 MB
// in, 264 MB out) 108 us, 4.6 TB/s.  (The gate and up product cannot write this
// form itself: the unit needs the maximum over the whole row.)
__global__ __launch_bounds__(512) void moe_h_kernel(const float *__restrict__ H, Plan pl, int F, uint16_t *__restrict__ hi,
                                                    uint16_t *__restrict__ lo, uint4 *__restrict__ sums,
                                                    float *__restrict__ unit, int64_t pitch)
{
    const int64_t at = blockIdx.x;
    if (at < pl.tiles[1])
        row_to_f16<true>(H + at * pitch, F, pitch, hi + at * pitch, lo + at * pitch, sums + at * (pitch / 32), unit + at);
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
// The form for few tokens reads an expert's weights once per pair, the other
// once per tile of pairs.  Measured (us, few against more): 8 experts of 14336 x
// 4096 Q4K, two a token: 8 tokens 247 / 260, 12 tokens 356 / 276; 128 of 768 x
// 2048 Q4K, eight a token: 32 tokens 118 / 152, 48 tokens 168 / 156; the same in
// Q8_0: 32 tokens 231 / 251, 48 tokens 334 / 254.  So: up to two pairs an
// expert; and up to four tokens always, whose products then stay in fp32.  (The
// host knows T k, not how many of the ids stand for an expert or how evenly they
// fall: a call most of whose ids stand for none is taken for a larger one.)
bool few(int T, int E, int k) { return T <= 4 || (int64_t)T * k <= 2 * (int64_t)E; }

// Workspace, few tokens: H [T k][F] in 4 bytes a value (fp32; the digits take
// 3.5).  Otherwise, P = T k pairs: the plan, Pd fp32 [P][K], and H: two planes
// [P][F], and for the tuned formats F padded to 256, its sums and units, its
// fp32 form, and X in fp16 with its sums and units.  One layout for every
// format and tile size.
struct Layout {
    int64_t hlo, hsum, hunit, h32, xh, xsum, xunit, pd, tiles, pair, place, total;
    int64_t fp, kp;
};
Layout layout_of(int T, int E, int k, int64_t F, int64_t K)
{
    const int64_t P = (int64_t)T * k;
    Layout l{};
    if (few(T, E, k)) {
        l.total = up16(4 * P * F);
        return l;
    }
    const int64_t most = P / 16 + (P < E ? P : E) + 1;
    l.fp = (F + 255) / 256 * 256;
    l.kp = (K + 255) / 256 * 256;
    l.hlo = 2 * P * l.fp;
    l.hsum = l.hlo + 2 * P * l.fp;
    l.hunit = l.hsum + P * l.fp / 2;
    l.h32 = l.hunit + up16(4 * P);
    l.xh = l.h32 + 4 * P * l.fp;
    l.xsum = l.xh + 2 * T * l.kp;
    l.xunit = l.xsum + T * l.kp / 2;
    // Pd takes the place of H's fp32 form where that is large enough
    l.pd = K <= l.fp ? l.h32 : l.xunit + up16(4 * T);
    l.tiles = K <= l.fp ? l.xunit + up16(4 * T) : l.pd + 4 * P * K;
    l.pair = l.tiles + 16 * (1 + most);
    l.place = l.pair + up16(4 * P);
    l.total = l.place + up16(4 * P);
    return l;
}

// Groups of R rows per workgroup: one while the launch has up to `want` waves,
// then as many as keep it near that, so that the activations are read once for
// more rows and the next rows' loads overlap the current ones' products.
int groups_for(int64_t rows, int R, int64_t waves_per_group, int64_t want)
{
    const int64_t g = ((rows + R - 1) / R * waves_per_group + want - 1) / want;
    return (int)(g < 1 ? 1 : g > MAXG ? MAXG : g);
}

template <int FMT, int R, int HMODE>
hipError_t glu_few(const MoeArgs &a, hipStream_t s)
{
    const Mat wg{a.gate, planes_of(FMT, a.E * a.F, a.K), a.K}, wu{a.up, wg.p, a.K};
    const int C = (int)(a.K / 32), KS = C > 7 * 64 ? 8 : (C + 63) / 64;
    int RW = 1;
    while (RW < 32 / R && 2 * RW * KS <= 8 && RW * KS * (a.F / 32) * a.T * a.k < 4096)
        RW *= 2;
    const dim3 grid((unsigned)(a.F / 32), a.T * a.k);
    moe_glu_kernel<FMT, R, HMODE><<<grid, 64 * KS * RW, 0, s>>>(wg, wu, a.X, a.ids, a.ws, a.E, a.k, a.F, a.act, KS);
    return hipGetLastError();
}

template <int FMT>
hipError_t glu_few(const MoeArgs &a, hipStream_t s)
{
    constexpr int R = 2;
    if (!digits_fmt(a.fmt_d))
        return glu_few<FMT, R, 0>(a, s);
    if (a.fmt_d == FMT_Q8_0)
        return glu_few<FMT, R, 1>(a, s);
    return glu_few<FMT, R, 2>(a, s);
}

template <int FMT>
hipError_t down_few(const MoeArgs &a, hipStream_t s)
{
    const Mat wd{a.down, planes_of(FMT, a.E * a.K, a.F), a.F};
    const int64_t items = a.k * (a.F / 32);
    const int KS = items > 7 * 64 ? 8 : (int)((items + 63) / 64);
    constexpr int R = 2;
    const int gr = groups_for(a.K, R, (int64_t)KS * a.T, 2048);
    const int64_t per = gr * R;
    const dim3 grid((unsigned)((a.K + per - 1) / per), a.T);
    moe_down_kernel<FMT, R><<<grid, 64 * KS, 0, s>>>(wd, a.ws, a.ids, a.weights, a.Y, a.E, a.k, a.K, gr);
    return hipGetLastError();
}

template <int FMT, int TM, int NT, bool GLU>
hipError_t gemm(const MoeArgs &a, const Layout &l, const Plan &pl, int max_tiles, hipStream_t s)
{
    uint16_t *hhi = reinterpret_cast<uint16_t *>(a.ws), *hlo = reinterpret_cast<uint16_t *>(a.ws + l.hlo);
    float *pd = reinterpret_cast<float *>(a.ws + l.pd);
    const int64_t N = GLU ? a.F : a.K, K = GLU ? a.K : a.F, per = 64 * (GLU ? NT / 2 : NT);
    const Planes p = planes_of(FMT, a.E * N, K);
    const Mat w0{GLU ? a.gate : a.down, p, K}, w1{GLU ? a.up : a.down, p, K};
    moe_gemm_kernel<FMT, TM, NT, GLU><<<dim3(max_tiles, (unsigned)((N + per - 1) / per)), 256, 0, s>>>(
        w0, w1, GLU ? a.X : hhi, hlo, pl, a.k, N, a.act, hhi, hlo, pd);
    return hipGetLastError();
}

template <int FMT, bool GLU>
hipError_t gemm_tm(const MoeArgs &a, const Layout &l, const Plan &pl, int tm, int max_tiles, hipStream_t s)
{
    if (tm == 1)
        return gemm<FMT, 1, 2, GLU>(a, l, pl, max_tiles, s);
    return gemm<FMT, 4, 2, GLU>(a, l, pl, max_tiles, s);
}

// Tiles of the products: 16 tm pairs.
struct Shape {
    int tm, max_tiles;
};

template <int FMT, int TM, int NT, bool GLU, bool TAIL>
hipError_t mm(const MoeArgs &a, const Layout &l, const Plan &pl, int max_tiles, hipStream_t s)
{
    constexpr bool THIN = TM == 1;
    const int64_t N = GLU ? a.F : a.K, K = GLU ? a.K : a.F, per = (THIN ? 4 / thin_kw(GLU) : 4) * 16 * (GLU ? NT / 2 : NT);
    const Planes p = planes_of(FMT, a.E * N, K);
    const Mat w0{GLU ? a.gate : a.down, p, K}, w1{GLU ? a.up : a.down, p, K};
    const auto u16 = [&](int64_t at) { return reinterpret_cast<const uint16_t *>(a.ws + at); };
    const auto u4 = [&](int64_t at) { return reinterpret_cast<const uint4 *>(a.ws + at); };
    const auto f32 = [&](int64_t at) { return reinterpret_cast<float *>(a.ws + at); };
    const Acts16 x = GLU ? Acts16{u16(l.xh), nullptr, u4(l.xsum), f32(l.xunit), l.kp}
                         : Acts16{u16(0), u16(l.hlo), u4(l.hsum), f32(l.hunit), l.fp};
    const int64_t nblk = (N + per - 1) / per, grid = (nblk * max_tiles + 7) / 8 * 8;
    const Order order{(int)nblk, 8};
    float *out = f32(GLU ? l.h32 : l.pd);
    const int64_t pitch = GLU ? l.fp : a.K;
    if constexpr (THIN)
        moe_thin_kernel<FMT, TM, NT, GLU, TAIL><<<dim3((unsigned)grid), 256, 0, s>>>(w0, w1, x, pl, a.k, N, order,
                                                                                         a.act, out, pitch);
    else
        moe_wide_kernel<FMT, TM, NT, GLU, TAIL><<<dim3((unsigned)grid), 256, 0, s>>>(w0, w1, x, pl, a.k, N, order, a.act, out,
                                                                              pitch);
    return hipGetLastError();
}

template <int FMT, bool GLU, bool TAIL>
hipError_t mm_shape(const MoeArgs &a, const Layout &l, const Plan &pl, const Shape &sh, hipStream_t s)
{
    if (sh.tm == 1)
        return mm<FMT, 1, 4, GLU, TAIL>(a, l, pl, sh.max_tiles, s);
    return mm<FMT, 4, 4, GLU, TAIL>(a, l, pl, sh.max_tiles, s);
}

template <int FMT, bool GLU>
hipError_t mm_tail(const MoeArgs &a, const Layout &l, const Plan &pl, const Shape &sh, hipStream_t s)
{
    if constexpr (FMT == FMT_Q8_0) {
        if ((GLU ? a.K : a.F) % 128 != 0)
            return mm_shape<FMT, GLU, true>(a, l, pl, sh, s);
    }
    return mm_shape<FMT, GLU, false>(a, l, pl, sh, s);
}

template <bool GLU>
hipError_t mm_fmt(const MoeArgs &a, const Layout &l, const Plan &pl, const Shape &sh, hipStream_t s)
{
    switch (GLU ? a.fmt_gu : a.fmt_d) {
    case FMT_Q4K: return mm_tail<FMT_Q4K, GLU>(a, l, pl, sh, s);
    case FMT_Q6K: return mm_tail<FMT_Q6K, GLU>(a, l, pl, sh, s);
    default: return mm_tail<FMT_Q8_0, GLU>(a, l, pl, sh, s);
    }
}

#define QL_EACH_FMT(X)                                                                                               \
    X(FMT_Q8_0) X(FMT_Q4K) X(FMT_Q6K) X(FMT_Q2K) X(FMT_Q3K) X(FMT_Q5K) X(FMT_Q4_0) X(FMT_Q4_1) X(FMT_Q5_0) X(FMT_Q5_1) \
        X(FMT_FP8)

}  // namespace

int64_t moe_workspace(int T, int E, int k, int64_t F, int64_t K) { return layout_of(T, E, k, F, K).total; }

hipError_t launch_moe(const MoeArgs &a, hipStream_t s)
{
    const Layout l = layout_of(a.T, a.E, a.k, a.F, a.K);
    hipError_t e = hipErrorNotSupported;
    if (few(a.T, a.E, a.k)) {
        switch (a.fmt_gu) {
#define X(f) case f: e = glu_few<f>(a, s); break;
            QL_EACH_FMT(X)
#undef X
        }
        if (e != hipSuccess)
            return e;
        switch (a.fmt_d) {
#define X(f) case f: return down_few<f>(a, s);
            QL_EACH_FMT(X)
#undef X
        }
        return hipErrorNotSupported;
    }
    const int P = a.T * a.k;
    // (offsets inside an expert's planes and inside X are 32 bits there; past
    // that, and for a pair of formats of which only one is tuned, bf16 pairs)
    const bool tuned =
        digits_fmt(a.fmt_gu) && digits_fmt(a.fmt_d) && a.F * a.K < (int64_t(1) << 31) && 2 * a.T * l.kp < (int64_t(1) << 32);
    // Pairs per tile, 16 or 64, from the mean number of an expert's pairs.  Tuned
    // formats (thin against wide, us): 8 experts of 14336 x 4096 Q4K, 12 pairs
    // each 336 / 443, 16 pairs 487 / 447; 8 of 4096 x 4096 Q8_0, 12 pairs 184 /
    // 263, 20 pairs 303 / 267.  The thin kernel's down product splits rows of F
    // over four waves, which short rows feed less: 16 of 2048 x 4096 Q4K, 6 pairs
    // 114 / 151, 12 pairs 159 / 154; 64 of 1536 x 2048, 6 pairs 183 / 188, 9 pairs
    // 204 / 190; 128 of 768 x 2048, 3 pairs 181 / 150.
    // Other formats (16 against 64 pairs): 8 of 4096 x 4096 Q4_0, 16 pairs 274 /
    // 310, 32 pairs 370 / 277; 32 of 768 x 2048 Q5K, 8 pairs 118 / 121, 16 pairs
    // 153 / 123.  The two cross on either side of sixteen pairs; twelve for both
    // costs the wide experts 36 us there and spares the narrow ones 30.
    const int per = P / a.E;
    const int most = !tuned || a.F >= 4096 ? 12 : a.F >= 1536 ? 8 : 0;
    Shape sh{per <= most ? 1 : 4, 0};
    const int BM = 16 * sh.tm, max_tiles = P / BM + (P < a.E ? P : a.E);
    sh.max_tiles = max_tiles;
    const Plan pl{reinterpret_cast<int32_t *>(a.ws + l.tiles), reinterpret_cast<int32_t *>(a.ws + l.pair),
                  reinterpret_cast<int32_t *>(a.ws + l.place)};
    if (tuned) {
        moe_prep_kernel<<<a.T + 1, 1024, 0, s>>>(
            a.ids, P, a.E, BM, pl, a.X, a.T, a.K, reinterpret_cast<uint16_t *>(a.ws + l.xh),
            reinterpret_cast<uint4 *>(a.ws + l.xsum), reinterpret_cast<float *>(a.ws + l.xunit), l.kp);
        if ((e = hipGetLastError()) != hipSuccess || (e = mm_fmt<true>(a, l, pl, sh, s)) != hipSuccess)
            return e;
        moe_h_kernel<<<P, 512, 0, s>>>(reinterpret_cast<const float *>(a.ws + l.h32), pl, (int)a.F, reinterpret_cast<uint16_t *>(a.ws),
                                       reinterpret_cast<uint16_t *>(a.ws + l.hlo), reinterpret_cast<uint4 *>(a.ws + l.hsum),
                                       reinterpret_cast<float *>(a.ws + l.hunit), l.fp);
        if ((e = hipGetLastError()) != hipSuccess || (e = mm_fmt<false>(a, l, pl, sh, s)) != hipSuccess)
            return e;
    } else {
        moe_plan_kernel<<<1, 1024, 0, s>>>(a.ids, P, a.E, BM, pl);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
        e = hipErrorNotSupported;
        switch (a.fmt_gu) {
#define X(f) case f: e = gemm_tm<f, true>(a, l, pl, sh.tm, max_tiles, s); break;
            QL_EACH_FMT(X)
#undef X
        }
        if (e != hipSuccess)
            return e;
        e = hipErrorNotSupported;
        switch (a.fmt_d) {
#define X(f) case f: e = gemm_tm<f, false>(a, l, pl, sh.tm, max_tiles, s); break;
            QL_EACH_FMT(X)
#undef X
        }
        if (e != hipSuccess)
            return e;
    }
    moe_join_kernel<<<dim3(a.T, (unsigned)((a.K + 1023) / 1024)), 256, 0, s>>>(
        reinterpret_cast<const float *>(a.ws + l.pd), pl.place, a.weights, a.Y, a.k, a.K);
    return hipGetLastError();
}

hipError_t launch_moe_route(const float *logits, int T, int E, int k, int score, const float *bias, int renorm,
                            float scale, int32_t *ids, float *weights, hipStream_t s)
{
    const unsigned grid = (unsigned)((T + 3) / 4);
#define ROUTE(V)                                                                                                     \
    if (E <= 64 * V) {                                                                                               \
        if (bias)                                                                                                    \
            moe_route_kernel<V, true><<<grid, 256, 0, s>>>(logits, T, E, k, score, bias, renorm, scale, ids, weights);  \
        else                                                                                                         \
            moe_route_kernel<V, false><<<grid, 256, 0, s>>>(logits, T, E, k, score, bias, renorm, scale, ids, weights); \
        return hipGetLastError();                                                                                    \
    }
    ROUTE(1) ROUTE(2) ROUTE(4) ROUTE(8) ROUTE(16)
#undef ROUTE
    return hipErrorNotSupported;
}

}  // namespace ql
