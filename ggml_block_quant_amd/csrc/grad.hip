// grad.hip -- gradients through frozen quantized weights: the input gradient of
// a quantized linear layer, the gated projection's backward pass, and the
// softmax cross entropy over a quantized head with its gradient.  The matrix
// product behind them is in product.h; here stand the passes over rows around
// it, the plans (tiles, splits, chunks of rows) and the launches.
#include "grad.h"
#include "product.h"

#include <initializer_list>
#include <type_traits>

namespace ql {

namespace {

// ---------------------------------------------------------------------------
// The A operand
// ---------------------------------------------------------------------------

// largest of a workgroup's values (all threads get it); `red` holds a float a wave
__device__ __forceinline__ float block_max(float v, float *red)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor(v, o));
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < waves; i++)
        v = fmaxf(v, red[i]);
    __syncthreads();
    return v;
}
__device__ __forceinline__ float block_sum(float v, float *red)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v += __shfl_xor(v, o);
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < waves; i++)
        v += red[i];
    __syncthreads();
    return v;
}

// The power of two that puts v into [2^14, 2^15); 0 for 0.  Infinities and NaN
// leave their row as it is (it is not finite then, and no other is).
__device__ __forceinline__ int row_exponent(float v)
{
    if (!(v > 0.0f) || v > __FLT_MAX__)
        return 0;
    return 15 - __builtin_amdgcn_frexp_expf(v);
}

// Eight neighbouring values of a row of n from i on, zeros behind its end.
// VEC: rows of whole groups of eight, 16-byte aligned.  Others are as wide
// loads and stores, at whatever address their rows start (one value at a time,
// the gated pair's pass over 2 rows of 9330 took 23 us, so 15), but for the last
// group.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
template <bool VEC> __device__ __forceinline__ void load8(const float *row, int64_t i, int64_t n, float v[8])
{
    if (VEC || i + 8 <= n) {
        const f32x4_any *const p = reinterpret_cast<const f32x4_any *>(
            VEC ? static_cast<const float *>(__builtin_assume_aligned(row + i, 16)) : row + i);
        const f32x4_any a = p[0], b = p[1];
#pragma unroll
        for (int j = 0; j < 4; j++)
            v[j] = a[j], v[4 + j] = b[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            v[j] = i + j < n ? row[i + j] : 0.0f;
    }
}
template <bool VEC> __device__ __forceinline__ void load8(const uint16_t *row, int64_t i, int64_t n, float v[8])
{
    if (VEC || i + 8 <= n) {
        const u32x4_any w = *reinterpret_cast<const u32x4_any *>(
            VEC ? static_cast<const uint16_t *>(__builtin_assume_aligned(row + i, 16)) : row + i);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            v[2 * j] = __builtin_bit_cast(float, w[j] << 16);
            v[2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            v[j] = i + j < n ? __builtin_bit_cast(float, (uint32_t)row[i + j] << 16) : 0.0f;
    }
}
template <bool VEC> __device__ __forceinline__ void store8(uint16_t *row, int64_t i, int64_t n, const float v[8])
{
    if (VEC || i + 8 <= n) {
        u32x4_any h;
#pragma unroll
        for (int j = 0; j < 4; j++)
            h[j] = bf16_bits(v[2 * j]) | (uint32_t)bf16_bits(v[2 * j + 1]) << 16;
        *reinterpret_cast<u32x4_any *>(VEC ? static_cast<uint16_t *>(__builtin_assume_aligned(row + i, 16)) : row + i) = h;
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (i + j < n)
                row[i + j] = bf16_bits(v[j]);
    }
}

// v[i] += the same of `more` further rows behind row[i], `apart` values from one
// to the next, in their order.  Four groups are asked for together (14 splits of
// 85 rows of 802 values, the gated pair: 19 us one after the other, now 10).
template <bool VEC, int ROWS>
__device__ __forceinline__ void add8(const float *const row[ROWS], int64_t apart, int more, int64_t i, int64_t n, float *const v[ROWS])
{
    int64_t at = 0;
    auto take = [&](auto count) {
        constexpr int C = decltype(count)::value;
        float t[C][ROWS][8];
#pragma unroll
        for (int s = 0; s < C; s++)
#pragma unroll
            for (int r = 0; r < ROWS; r++)
                load8<VEC>(row[r] + at + s * apart, i, n, t[s][r]);
#pragma unroll
        for (int s = 0; s < C; s++)
#pragma unroll
            for (int r = 0; r < ROWS; r++)
#pragma unroll
                for (int j = 0; j < 8; j++)
                    v[r][j] += t[s][r][j];
        at += C * apart;
    };
    constexpr int TOGETHER = 4 / ROWS;
    for (; more >= TOGETHER; more -= TOGETHER)
        take(std::integral_constant<int, TOGETHER>{});
    if (TOGETHER > 2 && more & 2)
        take(std::integral_constant<int, 2>{});
    if (more & 1)
        take(std::integral_constant<int, 1>{});
}

// largest magnitude of eight values; infinite where one is not finite
__device__ __forceinline__ float size8(const float v[8], float big)
{
#pragma unroll
    for (int j = 0; j < 8; j++)
        big = !(fabsf(v[j]) <= __FLT_MAX__) ? INFINITY : fmaxf(big, fabsf(v[j]));
    return big;
}

// chunk c (8 columns) of row m into its place
template <int PK>
__device__ __forceinline__ void store_a(uint8_t *A, int64_t Mp, int64_t m, int64_t c, const float v[8], int e)
{
    constexpr int C = PK / 8;
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; j++)
        h[j] = pack_f16(__builtin_ldexpf(v[2 * j], e), __builtin_ldexpf(v[2 * j + 1], e));
    *reinterpret_cast<uint4 *>(A + ((c / C) * Mp + m) * (2 * PK) + 16 * a_chunk<PK>((int)m, (int)(c % C))) =
        make_uint4(h[0], h[1], h[2], h[3]);
}

// The passes over rows below take one workgroup a row of up to HELD groups of
// eight a thread (16384 values with 512 threads), read once and held in
// registers between the row's largest value and its stores; longer rows are
// read twice, the second time from the cache.  One value at a time and twice,
// 2048 rows of 14336 took 83 us for the gradients and 400 us for the gated
// pair's.
constexpr int HELD = 4, HELD_LONG = 0, ROW_THREADS = 512;

// Rows of src [M][n] into panels, with zeros up to column `wide`.  scale: FP8's scales of the reduction's
// rows, or null.
template <typename V, int PK, int H, bool VEC>
__global__ __launch_bounds__(ROW_THREADS) void rows_kernel(const V *__restrict__ src, int64_t n, int64_t wide, int64_t Mp,
                                                           uint8_t *__restrict__ A, int *__restrict__ e_out,
                                                           const float *__restrict__ scale)
{
    __shared__ float red[ROW_THREADS / 64];
    const int64_t m = blockIdx.x;
    const V *row = src + m * n;
    const int64_t full = (n + 7) / 8, chunks = wide / 8;  // of eight: with values, with the zeros behind
    auto value = [&](int64_t c, float v[8]) {
        load8<VEC>(row, 8 * c, n, v);
        if (scale)
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (8 * c + j < n)
                    v[j] *= scale[8 * c + j];
    };
    float held[H > 0 ? H : 1][8];
    float big = 0.0f;
    if constexpr (H > 0) {
#pragma unroll
        for (int i = 0; i < H; i++) {
            const int64_t c = threadIdx.x + i * ROW_THREADS;
            if (c < full)
                value(c, held[i]);
            else
#pragma unroll
                for (int j = 0; j < 8; j++)
                    held[i][j] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < H; i++)
            big = size8(held[i], big);
    } else {
        for (int64_t c = threadIdx.x; c < full; c += ROW_THREADS) {
            value(c, held[0]);
            big = size8(held[0], big);
        }
    }
    big = block_max(big, red);
    const int e = row_exponent(big);
    if (threadIdx.x == 0)
        e_out[m] = e;
    if constexpr (H > 0) {
#pragma unroll
        for (int i = 0; i < H; i++) {
            const int64_t c = threadIdx.x + i * ROW_THREADS;
            if (c < chunks)
                store_a<PK>(A, Mp, m, c, held[i], e);
        }
    } else {
        for (int64_t c = threadIdx.x; c < chunks; c += ROW_THREADS) {
            float v[8] = {};
            if (c < full)
                value(c, v);
            store_a<PK>(A, Mp, m, c, v, e);
        }
    }
}

// dX = the splits' sums, scaled back by the row's power of two (e) and factor
// (w), each or null.  A workgroup takes 64 columns: 16 lanes of four, and 16
// runs of splits beside each other, whose sums meet in LDS.  (One thread a
// column over 32 splits took 11 us for one row, of which there are no more.)
__global__ __launch_bounds__(256) void join_kernel(const float *__restrict__ part, const int *__restrict__ e,
                                                   const float *__restrict__ w, int splits, int64_t M, int64_t K,
                                                   uint16_t *__restrict__ out)
{
    __shared__ float4 sum[16][16];
    const int c = threadIdx.x & 15, run = threadIdx.x >> 4;
    const int64_t m = blockIdx.y, k = 64 * (int64_t)blockIdx.x + 4 * c;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (k < K) {
        const int per = (splits + 15) / 16, s1 = min(splits, (run + 1) * per);
#pragma unroll 4
        for (int s = run * per; s < s1; s++) {
            const float4 t = *reinterpret_cast<const float4 *>(part + ((int64_t)s * M + m) * K + k);
            v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
        }
    }
    sum[run][c] = v;
    __syncthreads();
    if (run || k >= K)
        return;
    v = sum[0][c];
#pragma unroll
    for (int i = 1; i < 16; i++) {
        const float4 t = sum[i][c];
        v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
    }
    const int x = e ? -e[m] : 0;
    const float f = w ? w[m] : 1.0f;
    const uint32_t lo = bf16_bits(__builtin_ldexpf(v.x, x) * f) | (uint32_t)bf16_bits(__builtin_ldexpf(v.y, x) * f) << 16;
    const uint32_t hi = bf16_bits(__builtin_ldexpf(v.z, x) * f) | (uint32_t)bf16_bits(__builtin_ldexpf(v.w, x) * f) << 16;
    *reinterpret_cast<uint2 *>(out + m * K + k) = make_uint2(lo, hi);
}
// The same for few splits of many rows: eight columns a thread.
__global__ __launch_bounds__(256) void join_few_kernel(const float *__restrict__ part, const int *__restrict__ e,
                                                       const float *__restrict__ w, int splits, int64_t M, int64_t K,
                                                       uint16_t *__restrict__ out)
{
    const int64_t m = blockIdx.y, k = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (k >= K)
        return;
    float v[8] = {};
    const float *const row[1] = {part + m * K};
    float *const sums[1] = {v};
    add8<true, 1>(row, M * K, splits, k, K, sums);
    const int x = e ? -e[m] : 0;
    const float f = w ? w[m] : 1.0f;
#pragma unroll
    for (int j = 0; j < 8; j++)
        v[j] = __builtin_ldexpf(v[j], x) * f;
    store8<true>(out + m * K, k, K, v);
}

// ---------------------------------------------------------------------------
// The gated pair's gradients from g and u
// ---------------------------------------------------------------------------

__device__ __forceinline__ void glu_grad(int act, float g, float u, float dh, float &dg, float &du)
{
    if (act == 1) {
        const bool on = !(g <= 0.0f);  // (a NaN stays one)
        dg = on ? dh * u : 0.0f;
        du = on ? dh * g : 0.0f;
        return;
    }
    // p = sigmoid(g) and q = 1 - p without the digits that the difference would
    // lose: from e^-|g|, which cannot overflow
    const float t = expf(-fabsf(g)), z = 1.0f / (1.0f + t);
    const float p = g >= 0.0f ? z : t * z, q = g >= 0.0f ? t * z : z;
    if (act == 0) {
        dg = dh * u * (p * (1.0f + g * q));
        du = dh * (g * p);
    } else {
        dg = dh * u * (p * q);
        du = dh * p;
    }
}

struct GluRows {
    const float *g, *u;  // sums of the rows, the first split: row m at m ld
    const float *mg, *mu;  // the others, from column `from` on: row m of split s at ((s - 1) M + m) more_ld - from
    int splits, act;
    bool whole;          // whether the sums' rows have room for whole groups of eight, 16-byte aligned
    int64_t more_ld, from;
    int64_t M, F, Mp, ld;
    const int *ex;       // exponents of X's rows, or null
    const float *sg, *su;  // FP8's scales of the rows, or null
    bool raw;            // whether g and u still lack them
    const void *dH;
    uint8_t *A;
    int *e_out;
    uint16_t *dG, *dU;   // or null
};
// dg and du of row m's values 8 c .. 8 c + 7, with FP8's scales taken; keep: the
// bf16 results (without them) with them
template <typename V, bool VEC>
__device__ __forceinline__ void glu_values(const GluRows &a, int64_t m, int64_t c, float dg[8], float du[8], bool keep)
{
    const int64_t F = a.F;
    const int x = a.ex ? -a.ex[m] : 0;
    float g[8], u[8], h[8];
    load8<VEC>(static_cast<const V *>(a.dH) + m * F, 8 * c, F, h);
    const int more = 8 * c < a.from ? 0 : a.splits - 1;
    auto sums = [&](auto whole) {
        constexpr bool V8 = decltype(whole)::value;
        load8<V8>(a.g + m * a.ld, 8 * c, F, g);
        load8<V8>(a.u + m * a.ld, 8 * c, F, u);
        const float *const row[2] = {a.mg + m * a.more_ld - a.from, a.mu + m * a.more_ld - a.from};
        float *const both[2] = {g, u};
        add8<V8, 2>(row, a.M * a.more_ld, more, 8 * c, F, both);
    };
    if (VEC || a.whole)
        sums(std::true_type{});
    else
        sums(std::false_type{});
#pragma unroll
    for (int j = 0; j < 8; j++) {
        float p = __builtin_ldexpf(g[j], x), q = __builtin_ldexpf(u[j], x);
        const int64_t f = min(8 * c + j, F - 1);
        if (a.raw && a.sg)
            p *= a.sg[f], q *= a.su[f];
        glu_grad(a.act, p, q, h[j], dg[j], du[j]);
        if (8 * c + j >= F)
            dg[j] = du[j] = 0.0f;
    }
    if (keep) {
        if (a.dG)
            store8<VEC>(a.dG + m * F, 8 * c, F, dg);
        if (a.dU)
            store8<VEC>(a.dU + m * F, 8 * c, F, du);
    }
    if (a.sg)
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int64_t f = min(8 * c + j, F - 1);
            dg[j] *= a.sg[f], du[j] *= a.su[f];
        }
}

// One row, for one_kernel: both gradients in fp32, one behind the other
template <typename V, bool VEC> __global__ __launch_bounds__(64) void glu_one_kernel(GluRows a, float *__restrict__ D)
{
    const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (8 * c >= a.F)
        return;
    float dg[8], du[8];
    glu_values<V, VEC>(a, 0, c, dg, du, true);
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (8 * c + j < a.F)
            D[8 * c + j] = dg[j], D[a.F + 8 * c + j] = du[j];
}

// One workgroup a row: g and u from the splits' sums, the two gradients (bf16
// where wanted), and both as rows of A under one power of two.
template <typename V, int H, bool VEC>
__global__ __launch_bounds__(ROW_THREADS) void glu_rows_kernel(GluRows a)
{
    __shared__ float red[ROW_THREADS / 64];
    const int64_t m = blockIdx.x, F = a.F;
    const int64_t panels = (F + 63) / 64, chunks = panels * 8, full = (F + 7) / 8;
    auto value = [&](int64_t c, float dg[8], float du[8], bool keep) { glu_values<V, VEC>(a, m, c, dg, du, keep); };
    float hg[H > 0 ? H : 1][8], hu[H > 0 ? H : 1][8];
    float big = 0.0f;
    if constexpr (H > 0) {
#pragma unroll
        for (int i = 0; i < H; i++) {
            const int64_t c = threadIdx.x + i * ROW_THREADS;
            if (c < full)
                value(c, hg[i], hu[i], true);
            else
#pragma unroll
                for (int j = 0; j < 8; j++)
                    hg[i][j] = hu[i][j] = 0.0f;
            big = size8(hu[i], size8(hg[i], big));
        }
    } else {
        for (int64_t c = threadIdx.x; c < full; c += ROW_THREADS) {
            value(c, hg[0], hu[0], true);
            big = size8(hu[0], size8(hg[0], big));
        }
    }
    big = block_max(big, red);
    const int e = row_exponent(big);
    if (threadIdx.x == 0)
        a.e_out[m] = e;
    uint8_t *const A1 = a.A + panels * a.Mp * 128;
    if constexpr (H > 0) {
#pragma unroll
        for (int i = 0; i < H; i++) {
            const int64_t c = threadIdx.x + i * ROW_THREADS;
            if (c < chunks) {
                store_a<64>(a.A, a.Mp, m, c, hg[i], e);
                store_a<64>(A1, a.Mp, m, c, hu[i], e);
            }
        }
    } else {
        for (int64_t c = threadIdx.x; c < chunks; c += ROW_THREADS) {
            float dg[8] = {}, du[8] = {};
            if (c < full)
                value(c, dg, du, false);
            store_a<64>(a.A, a.Mp, m, c, dg, e);
            store_a<64>(A1, a.Mp, m, c, du, e);
        }
    }
}

// ---------------------------------------------------------------------------
// Cross entropy from the logits' sums
// ---------------------------------------------------------------------------

// The largest logit but the given token's (m), the sum of e^(z - m) of these
// (l; NaN where one of the logits is, also where none of them is a number and m
// stays -inf); FP8: the largest scale of the rows (s)
struct Stat {
    float m, l, s;
};
__device__ __forceinline__ Stat join(Stat a, Stat b)
{
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY)
        return Stat{m, a.l + b.l, fmaxf(a.s, b.s)};  // of zeros and NaN
    return Stat{m, a.l * expf(a.m - m) + b.l * expf(b.m - m), fmaxf(a.s, b.s)};
}

struct XentRows {
    const float *part;       // sums, the first split: [M][ld]
    const float *more;       // the others, from column `from` on: [splits - 1][M][more_ld]
    int splits, runs;
    int64_t ld, more_ld, from;
    int64_t M, N, run, Mp;   // runs of `run` logits (a multiple of 64), one a workgroup
    const int *ex;           // exponents of X's rows, or null
    const float *sw;         // FP8's scales of the rows, or null
    bool raw;                // whether the sums still lack them
    const int32_t *targets;
    const float *weights;    // or null
    Stat *stats;             // [M][runs]
    uint8_t *A;              // panels for the gradient, or null
    float *D;                // the gradient of one row in fp32, or null
    int *e_out;
    float *w_out, *loss, *lse;  // lse: or null
};

__device__ __forceinline__ float logit(const XentRows &a, int64_t m, int64_t n, int x)
{
    float z = a.part[m * a.ld + n];
    for (int s = 1; s < (n < a.from ? 1 : a.splits); s++)
        z += a.more[((int64_t)(s - 1) * a.M + m) * a.more_ld + n - a.from];
    z = __builtin_ldexpf(z, x);
    return a.raw && a.sw ? z * a.sw[n] : z;
}
// logits 8 c .. 8 c + 7 of row m, -inf behind the row's end.  VEC: rows 16-byte
// aligned, with room for whole groups of eight
template <bool VEC> __device__ __forceinline__ void logits8(const XentRows &a, int64_t m, int64_t c, int x, float z[8])
{
    load8<VEC>(a.part + m * a.ld, 8 * c, a.N, z);
    const float *const row[1] = {a.more + m * a.more_ld - a.from};
    float *const sums[1] = {z};
    add8<VEC, 1>(row, a.M * a.more_ld, 8 * c < a.from ? 0 : a.splits - 1, 8 * c, a.N, sums);
#pragma unroll
    for (int j = 0; j < 8; j++) {
        z[j] = __builtin_ldexpf(z[j], x);
        if (a.raw && a.sw)
            z[j] *= a.sw[min(8 * c + j, a.N - 1)];
        if (8 * c + j >= a.N)
            z[j] = -INFINITY;
    }
}

// Run blockIdx.x of row blockIdx.y: its Stat, in one pass with the running
// maximum and sum of each thread.  The given token is left out: 1 - p of it is
// the others' share, with all of its digits.
template <bool VEC> __global__ __launch_bounds__(256) void stat_kernel(XentRows a)
{
    __shared__ float red[4];
    const int64_t m = blockIdx.y, t = a.targets[m];
    const int64_t c0 = blockIdx.x * a.run / 8, c1 = min((a.N + 7) / 8, c0 + a.run / 8);
    const int x = a.ex ? -a.ex[m] : 0;
    float big = -INFINITY, l = 0.0f;
    bool odd = false;
    for (int64_t c = c0 + threadIdx.x; c < c1; c += 256) {
        float z[8];
        logits8<VEC>(a, m, c, x, z);
        float top = big;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            odd |= z[j] != z[j];
            z[j] = 8 * c + j == t ? -INFINITY : z[j];
            top = fmaxf(top, z[j]);
        }
        if (top == -INFINITY)
            continue;
        l *= expf(big - top);
#pragma unroll
        for (int j = 0; j < 8; j++)
            l += expf(z[j] - top);
        big = top;
    }
    const float top = block_max(big, red);
    l = block_sum(big == -INFINITY ? 0.0f : l * expf(big - top), red);
    odd = __syncthreads_or(odd);
    float sc = 0.0f;
    if (a.sw) {
        for (int64_t n = 8 * c0 + threadIdx.x; n < min(a.N, 8 * c1); n += 256)
            sc = fmaxf(sc, a.sw[n]);
        sc = block_max(sc, red);
    }
    if (threadIdx.x == 0)
        a.stats[m * a.runs + blockIdx.x] = Stat{top, odd ? NAN : l, sc};
}

// Row m: loss and lse, and its gradient with respect to the logits as a row of
// A (zeros for a token that is not scored and for one of weight 0, whatever
// their logits: padding may hold anything).  p_n - [n = t] is at most
// max(largest p of the others, 1 - p_t) in size, which fixes the power of two;
// the row's weight enters as a factor of its own afterwards (w_out).
template <bool VEC> __global__ __launch_bounds__(256) void xent_rows_kernel(XentRows a)
{
    const int64_t m = blockIdx.y;
    const int64_t t = a.targets[m];
    const bool given = t >= 0 && t < a.N;
    const int x = a.ex ? -a.ex[m] : 0;
    // the runs' Stats, as the threads' own first (in an order that does not change)
    __shared__ float red[4];
    Stat rest{-INFINITY, 0.0f, 0.0f};
    for (int i = threadIdx.x; i < a.runs; i += 256)
        rest = join(rest, a.stats[m * a.runs + i]);
    if (a.runs > 1) {
        const float big = block_max(rest.m, red);
        rest.l = block_sum(rest.m == -INFINITY ? rest.l : rest.l * expf(rest.m - big), red);
        rest.s = block_max(rest.s, red);
        rest.m = big;
    } else {
        rest = a.stats[m];
    }
    // the whole: the others and the given token
    const float zt = given ? logit(a, m, t, x) : -INFINITY;
    const float top = fmaxf(rest.m, zt);
    const float lr = rest.l * expf(rest.m - top), lt = given ? expf(zt - top) : 0.0f;
    const float l = lr + lt;
    const bool first = blockIdx.x == 0 && threadIdx.x == 0;
    if (first) {
        // ln(l / lt) = log1p(lr / lt) where the token is the likelier side
        a.loss[m] = !given ? 0.0f : lt > lr ? log1pf(lr / lt) : logf(l) + (top - zt);
        if (a.lse)
            a.lse[m] = logf(l) + top;
    }
    if (!a.A && !a.D)
        return;
    const float big = fmaxf(expf(rest.m - top) / l, lr / l) * (a.sw ? rest.s : 1.0f);
    const float rl = 1.0f / l;
    const float gt = -lr * rl;
    const int e = row_exponent(big);
    const float weight = given ? (a.weights ? a.weights[m] : 1.0f) : 0.0f;
    const bool counts = weight != 0.0f;
    if (first && a.A) {
        a.e_out[m] = e;
        a.w_out[m] = weight;
    }
    const int64_t full = (a.N + 7) / 8, c1 = min((a.N + 63) / 64 * 8, ((int64_t)blockIdx.x + 1) * a.run / 8);
    for (int64_t c = blockIdx.x * a.run / 8 + threadIdx.x; c < c1; c += 256) {
        float v[8] = {};
        if (counts && c < full) {
            logits8<VEC>(a, m, c, x, v);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                v[j] = 8 * c + j == t ? gt : expf(v[j] - top) * rl;
                if (a.sw)
                    v[j] *= a.sw[min(8 * c + j, a.N - 1)];
            }
        }
        if (a.A) {
            store_a<64>(a.A, a.Mp, m, c, v, e);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (8 * c + j < a.N)
                    a.D[8 * c + j] = v[j] * weight;
        }
    }
}

// ---------------------------------------------------------------------------
// Plans and launches
// ---------------------------------------------------------------------------

int tile_rows(int tile) { return tile == TILE_192 ? 192 : tile == TILE_256 ? 256 : 32 << tile; }

// A form of the product by its mode and tile: columns of C and of the
// reduction that a workgroup takes at a time, columns of a panel of A.
struct Form {
    int cols, step, panel;
};
Form form_of(int mode, int tile)
{
    if (mode == BACK)
        return Form{256, 64, 64};
    if (tile <= TILE_64)
        return Form{mode == FORE_GLU ? 32 : 64, 128, 64};
    return mode == FORE_GLU ? Form{128, 64, 64} : Form{256, 32, 32};
}

// tiles of which the first `whole` are not split, the others `splits` ways
struct Plan {
    int tile, splits, steps, per;
    int64_t Mp, tiles, whole;
    Form f;
    int64_t workgroups() const { return whole + (tiles - whole) * splits; }
    int64_t split_from() const { return splits > 1 ? whole / (Mp / rows) * f.cols : 0; }  // the first column that is split
    int64_t rows;  // of a tile
};
// Up to 64 rows a launch is split until it fills the card twice; from 65 on
// splits are chosen by time, with one workgroup a CU.  (Their LDS admits no more
// but in the pairs' form of 128 rows, of which two would fit: its 97 x 32003 of
// 2048 run as 252 workgroups of four waves, one wave a SIMD.)
constexpr int kSplitTo = 512, kTimedSplits = 64, kTimedTo = 1024;

Plan plan_with(int mode, int tile, int64_t M, int64_t cols, int64_t depth, int parts, int64_t n)
{
    Plan p;
    p.tile = tile, p.rows = tile_rows(tile), p.whole = 0;
    p.f = form_of(mode, tile);
    p.Mp = up_to(M, tile_rows(tile));
    p.tiles = p.Mp / tile_rows(tile) * ((cols + p.f.cols - 1) / p.f.cols);
    p.steps = (int)((depth + p.f.step - 1) / p.f.step) * parts;
    n = n < 1 ? 1 : n > p.steps ? p.steps : n;
    p.per = (int)((p.steps + n - 1) / n);
    p.splits = (p.steps + p.per - 1) / p.per;
    p.whole = p.splits == 1 ? p.tiles : 0;
    return p;
}
// the same with whole columns of tiles unsplit in front, as many as fill whole
// rounds of 256 workgroups
Plan with_whole(Plan p)
{
    const int64_t mt = p.Mp / p.rows;
    p.whole = p.tiles / 256 * 256 / mt * mt;
    if (p.whole == p.tiles || p.splits == 1)
        p.whole = p.tiles, p.splits = 1, p.per = p.steps;
    return p;
}
// Estimated time of a plan in us, from what its kernels reach: a workgroup's
// products in TFLOP/s (256 rows: 1.0 to 1.1 PFLOP/s of the card in the backward
// form, half for pairs), whole rounds of 256 workgroups, 4 us to start, and the
// splits' sums written and read (backward: none where there is one split; the
// cross entropy reads them twice) at 4.5 TB/s.
double plan_us(const Plan &p, int mode, int64_t M, int64_t cols)
{
    const double rate = (p.tile == TILE_256 ? 4.1 : p.tile == TILE_192 ? 3.6 : 2.6) * (mode == FORE_PAIR ? 0.5 : 1.0);
    const int64_t rounds = (p.whole + 255) / 256, parted = ((p.tiles - p.whole) * p.splits + 255) / 256;
    const double flops = 2.0 * p.rows * 256 * p.f.step;  // of a step
    const double bytes = 4.0 * M * cols * (mode == FORE_GLU ? 2 : 1), part = 1.0 - (double)p.whole / p.tiles;
    const double times = (1.0 - part) + part * p.splits;  // that a value of C is written
    const double moved = mode == BACK ? (p.splits > 1 ? 2 * times : 0) : mode == FORE_GLU ? 2 * times : 3 * times;
    return rounds * (flops * p.steps / rate * 1e-6 + 4.0) + parted * (flops * p.per / rate * 1e-6 + 4.0) + moved * bytes / 4.5e6;
}
// M rows, `cols` columns of C, a reduction over `parts` times `depth`.  Between
// one tile of 192 and of 256 rows, and between splits, the least time decides:
// 515 rows are 3 tiles of either (6144 x 4096 Q4K backward 49.7 and 41.0 us);
// 375 tiles in one round and a half leave half of the card idle in the second,
// so a forward product may split what its whole rounds leave (gate and up of
// 2048 x 14336 x 4096: 896 tiles, the last 128 in halves).
Plan plan_of(int mode, int64_t M, int64_t cols, int64_t depth, int parts)
{
    if (M <= 64) {
        const int tile = M <= 32 ? TILE_32 : TILE_64;
        const Form f = form_of(mode, tile);
        int64_t n = kSplitTo / ((cols + f.cols - 1) / f.cols);
        // (a forward split takes four steps or more: gate and up of
        // 50 x 1408 of 2048 in eighths 11.4 us, in quarters 10.1)
        if (mode != BACK && n > depth / f.step / 4)
            n = depth / f.step / 4;
        return plan_with(mode, tile, M, cols, depth, parts, n);
    }
    Plan best{};
    double least = 0.0;
    // (192 only where it pads to no more than 256 does: padded() counts on it)
    const int first = M <= 128 ? TILE_128 : up_to(M, 192) < up_to(M, 256) ? TILE_192 : TILE_256;
    for (int tile = first; tile <= (M <= 128 ? TILE_128 : TILE_256); tile++)
        for (const int n : {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 16, 20, 24, 32, 48, kTimedSplits}) {
            const Plan p = plan_with(mode, tile, M, cols, depth, parts, n);
            // (a backward product's sums are joined for all columns or none)
            const bool tail = mode != BACK && p.tiles > 256;
            if (p.tiles * n > kTimedTo && n > 1 && !tail)
                break;
            for (const Plan &t : {p, tail ? with_whole(p) : p}) {
                if (t.splits > 1 && (t.tiles - t.whole) * t.splits > kTimedTo)
                    continue;
                const double us = plan_us(t, mode, M, cols);
                if (best.steps == 0 || us < least)
                    best = t, least = us;
            }
        }
    return best;
}
// The most rows that the splits' sums of a call of up to M rows take (splits
// times rows; 0 where nothing is split).  It grows with M, so that a workspace
// for M rows serves fewer.
int64_t split_rows(int mode, int64_t M, int64_t cols)
{
    int64_t most = 0;
    for (int t = 0; t <= (M <= 32 ? TILE_32 : M <= 64 ? TILE_64 : M <= 128 ? TILE_128 : TILE_256); t++) {
        const int64_t ct = (cols + form_of(mode, t).cols - 1) / form_of(mode, t).cols;
        // splits * row tiles * ct is at most this where there is more than one
        const int64_t n = (t <= TILE_64 ? kSplitTo : kTimedTo) / ct;
        int64_t rows = n > 1 ? n * tile_rows(t) : 0;
        rows = t > TILE_64 && rows > kTimedSplits * M ? kTimedSplits * M : rows;
        most = rows > most ? rows : most;
    }
    return most;
}

// Rows of a call that go through at once: at most 2^e values of the widest
// operand, whole tiles.
int64_t chunk_rows(int64_t M, int64_t width, int e)
{
    int64_t r = ((int64_t)1 << e) / width;
    r = r >= 256 ? r / 256 * 256 : r >= 32 ? r / 32 * 32 : 32;
    r = r > 32768 ? 32768 : r;
    return r < M ? r : M;
}
// the most rows that a tile of some plan of M rows pads them to
int64_t padded(int64_t M) { return up_to(M, M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256); }

// panels of n columns (a multiple of 128: the widest step)
int64_t panels_bytes(int64_t Mp, int64_t n) { return up_to(n, 128) * Mp * 2; }

hipError_t launch_product(int fmt, int mode, const Plan &p, ProductArgs a, hipStream_t s)
{
    a.Mp = p.Mp, a.steps = p.steps, a.per = p.per, a.tiles = (uint32_t)p.tiles, a.whole = (uint32_t)p.whole;
    const unsigned grid = (unsigned)p.workgroups();
    switch (fmt) {
    case FMT_Q8_0: return launch_product_q8_0(mode, p.tile, a, grid, s);
    case FMT_Q4K: return launch_product_q4k(mode, p.tile, a, grid, s);
    case FMT_Q6K: return launch_product_q6k(mode, p.tile, a, grid, s);
    case FMT_Q5K:
    case FMT_Q3K:
    case FMT_Q2K:
    case FMT_FP8: return launch_product_kquants(fmt, mode, p.tile, a, grid, s);
    default: return launch_product_legacy(fmt, mode, p.tile, a, grid, s);
    }
}

const float *row_scales(int fmt, const uint8_t *W, const Planes &p)
{
    return fmt == FMT_FP8 ? reinterpret_cast<const float *>(W + p.scales) : nullptr;
}

// rows of src (M of n) into panels of PK columns, zeros up to `wide`
template <int PK, typename V>
hipError_t run_rows(const V *src, int64_t M, int64_t n, int64_t wide, int64_t Mp, uint8_t *A, int *e, const float *scale,
                    hipStream_t s)
{
    const bool held = wide <= 8 * HELD * ROW_THREADS, vec = n % 8 == 0;
    const auto run = [&](auto kernel) { kernel<<<(unsigned)M, ROW_THREADS, 0, s>>>(src, n, wide, Mp, A, e, scale); };
    held ? vec ? run(rows_kernel<V, PK, HELD, true>) : run(rows_kernel<V, PK, HELD, false>)
         : vec ? run(rows_kernel<V, PK, HELD_LONG, true>) : run(rows_kernel<V, PK, HELD_LONG, false>);
    return hipGetLastError();
}

// a workspace handed out piece by piece, each 256-byte aligned (from a base
// that is 16-byte aligned)
struct Pieces {
    uint8_t *base;
    int64_t used = 0;
    uint8_t *take(int64_t bytes)
    {
        uint8_t *p = base + used;
        used += up_to(bytes, 256);
        return p;
    }
};

hipError_t run_join(const float *part, const int *e, const float *w, int splits, int64_t M, int64_t K, uint16_t *dX, hipStream_t s)
{
    // (48 splits of one row: 4 us against 11)
    if (splits >= 16)
        join_kernel<<<dim3((unsigned)((K + 63) / 64), (unsigned)M), 256, 0, s>>>(part, e, w, splits, M, K, dX);
    else
        join_few_kernel<<<dim3((unsigned)((K + 2047) / 2048), (unsigned)M), 256, 0, s>>>(part, e, w, splits, M, K, dX);
    return hipGetLastError();
}

// dX = the backward product of A's rows over one weight or two, split or not
Plan back_plan(int64_t M, int64_t rows, int64_t K, int weights) { return plan_of(BACK, M, K, rows, weights); }
hipError_t run_back(int fmt, const Plan &p, const uint8_t *W0, const uint8_t *W1, const Planes &pl, const uint8_t *A, const int *e,
                    const float *w, int64_t M, int64_t rows, int64_t K, float *part, uint16_t *dX, hipStream_t s)
{
    ProductArgs a{};
    a.W0 = W0, a.W1 = W1, a.p = pl, a.A = A, a.e = e, a.w = w;
    a.part = p.splits > 1 ? part : nullptr;
    a.out = p.splits > 1 ? nullptr : dX;
    a.M = M, a.ld = a.more_ld = K, a.more = part + M * K, a.rows = rows, a.K = K;
    const hipError_t err = launch_product(fmt, BACK, p, a, s);
    if (err != hipSuccess || p.splits == 1)
        return err;
    return run_join(part, e, w, p.splits, M, K, dX, s);
}
// the same of one row in fp32 or bf16 (of two weights, one behind the other)
constexpr int kOneSplitTo = 1024;
hipError_t run_one(int fmt, const uint8_t *W0, const uint8_t *W1, const Planes &pl, const void *D, bool bf16, const float *scale,
                   int64_t rows, int64_t K, float *part, uint16_t *dX, hipStream_t s)
{
    const int64_t groups = (K + 255) / 256, all = (W1 ? 2 * rows : rows), runs = (all + 31) / 32;
    int64_t n = kOneSplitTo / groups;
    // (at least eight runs of 32 rows: a split ends in 32 KiB of LDS summed)
    n = n > runs / 8 ? runs / 8 : n;
    n = n < 1 ? 1 : n;
    OneArgs a{};
    a.W0 = W0, a.W1 = W1, a.p = pl, a.D = D, a.scale = scale, a.part = part, a.rows = rows, a.K = K;
    a.per = (int)((runs + n - 1) / n);
    const int splits = (int)((runs + a.per - 1) / a.per);
    const unsigned grid = (unsigned)(groups * splits);
    hipError_t err;
    switch (fmt) {
    case FMT_Q8_0: err = launch_one_q8_0(bf16, a, grid, s); break;
    case FMT_Q4K: err = launch_one_q4k(bf16, a, grid, s); break;
    case FMT_Q6K: err = launch_one_q6k(bf16, a, grid, s); break;
    case FMT_Q5K:
    case FMT_Q3K:
    case FMT_Q2K:
    case FMT_FP8: err = launch_one_kquants(fmt, bf16, a, grid, s); break;
    default: err = launch_one_legacy(fmt, bf16, a, grid, s); break;
    }
    return err != hipSuccess ? err : run_join(part, nullptr, nullptr, splits, 1, K, dX, s);
}
// the splits' sums of either
int64_t back_part_bytes(int64_t M, int64_t K)
{
    const int64_t one = kOneSplitTo / ((K + 255) / 256), tiles = split_rows(BACK, M, K);
    return 4 * K * (tiles > one ? tiles : one > 1 ? one : 1);
}
// Sums of a forward product: rows of `width` values, and what the other splits
// of split columns take: at most the tiles they are split into (64 x 64 values
// up to 64 rows, 256 x 256 from 65), and so many times the rows.  (256 bytes to
// start a second half on a boundary.)
int64_t fore_part_bytes(int64_t M, int64_t width)
{
    const auto least = [](int64_t a, int64_t b) { return a < b ? a : b; };
    const int64_t few = least((int64_t)kSplitTo * 64 * 64, kSplitTo * (M < 64 ? M : 64) * width);
    const int64_t many = M > 64 ? least((int64_t)kTimedTo * 256 * 256, kTimedSplits * M * width) : 0;
    return 4 * (M * width + (few > many ? few : many)) + 256;
}

// Up to two rows the forward products are matrix-vector products: the GEMV
// takes the weights exactly and sums in fp32 (131072 x 5120 Q6K, one and two
// rows: 93 and 141 us, tiles of 32 rows 237).  So are three rows, and four of
// the cross entropy's pairs, where its one-shot kernel takes them (32000 x 4096,
// pairs, tiles against GEMV: Q4K 43 and 23, four 43 and 31; Q6K 51 and 39, four
// 51 and 48; Q8_0 43 and 31, four 43 and 37; the gated pair's three 57 and 45,
// 85 and 79, 87 and 62, but Q6K's four 85 and 96), but for Q6K and Q8_0 at three
// chunks of 64 units a row, where it is slow (32000 x 5120, three rows: Q6K 58
// and 96, Q8_0 52 and 71).
bool gemv_takes(int fmt, int64_t M, int64_t K, int64_t most)
{
    return M <= 2 || (M <= most && gemv_one_shot_fits(fmt, (int)M, K) && (fmt == FMT_Q4K || (K / 32 + 63) / 64 != 3));
}

}  // namespace

// ---- dX = dY . deq(W)

constexpr int kGradChunk = 27;  // log2 of the values of dY that go through at once (256 MiB of A)

int64_t grad_workspace(int fmt, int64_t M, int64_t N, int64_t K)
{
    const int64_t R = chunk_rows(M, up_to(N, 64), kGradChunk);
    Pieces w{nullptr};
    w.take(panels_bytes(padded(R), N));
    w.take(4 * R);
    w.take(back_part_bytes(R, K));
    return w.used;
}

hipError_t launch_grad(const GradArgs &a, hipStream_t s)
{
    const Planes p = planes_of(a.fmt, a.N, a.K);
    const int64_t R = chunk_rows(a.M, up_to(a.N, 64), kGradChunk);
    Pieces w{a.ws};
    uint8_t *A = w.take(panels_bytes(padded(R), a.N));
    int *e = reinterpret_cast<int *>(w.take(4 * R));
    float *part = reinterpret_cast<float *>(w.take(back_part_bytes(R, a.K)));
    const float *sw = row_scales(a.fmt, a.W, p);
    if (a.M == 1)
        return run_one(a.fmt, a.W, nullptr, p, a.dY, a.dy_bf16, sw, a.N, a.K, part, a.dX, s);
    for (int64_t m = 0; m < a.M; m += R) {
        const int64_t n = a.M - m < R ? a.M - m : R, wide = up_to(a.N, 64);
        const Plan b = back_plan(n, a.N, a.K, 1);
        hipError_t err = a.dy_bf16 ? run_rows<64>(static_cast<const uint16_t *>(a.dY) + m * a.N, n, a.N, wide, b.Mp, A, e, sw, s)
                                   : run_rows<64>(static_cast<const float *>(a.dY) + m * a.N, n, a.N, wide, b.Mp, A, e, sw, s);
        if (err == hipSuccess)
            err = run_back(a.fmt, b, a.W, nullptr, p, A, e, nullptr, n, a.N, a.K, part, a.dX + m * a.K, s);
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

// ---- the gated pair

constexpr int kGluChunk = 26;  // log2 of the values of G (and of U) at once

int64_t glu_grad_workspace(int fmt, int64_t M, int64_t F, int64_t K)
{
    const int64_t R = chunk_rows(M, up_to(F, 64), kGluChunk);
    Pieces w{nullptr};
    w.take(panels_bytes(padded(R), K));
    w.take(2 * panels_bytes(padded(R), F));
    w.take(4 * R);
    w.take(4 * R);
    w.take(fore_part_bytes(R, 2 * up_to(F, 8)));
    w.take(back_part_bytes(R, K));
    return w.used;
}

hipError_t launch_glu_grad(const GluGradArgs &a, hipStream_t s)
{
    const Planes pl = planes_of(a.fmt, a.F, a.K);
    const int64_t R = chunk_rows(a.M, up_to(a.F, 64), kGluChunk);
    Pieces w{a.ws};
    uint8_t *AX = w.take(panels_bytes(padded(R), a.K));
    uint8_t *AD = w.take(2 * panels_bytes(padded(R), a.F));
    int *ex = reinterpret_cast<int *>(w.take(4 * R)), *ed = reinterpret_cast<int *>(w.take(4 * R));
    float *gu = reinterpret_cast<float *>(w.take(fore_part_bytes(R, 2 * up_to(a.F, 8))));
    float *part = reinterpret_cast<float *>(w.take(back_part_bytes(R, a.K)));
    for (int64_t m = 0; m < a.M; m += R) {
        const int64_t n = a.M - m < R ? a.M - m : R;
        const Plan b = back_plan(n, a.F, a.K, 2);
        GluRows r{};
        r.splits = 1, r.act = a.act, r.M = n, r.F = a.F, r.Mp = b.Mp;
        r.sg = row_scales(a.fmt, a.gate, pl), r.su = row_scales(a.fmt, a.up, pl);
        r.dH = a.dh_bf16 ? (const void *)(static_cast<const uint16_t *>(a.dH) + m * a.F)
                         : (const void *)(static_cast<const float *>(a.dH) + m * a.F);
        r.A = AD, r.e_out = ed, r.dG = a.dG ? a.dG + m * a.F : nullptr, r.dU = a.dU ? a.dU + m * a.F : nullptr;
        hipError_t err = hipErrorNotSupported;
        if (gemv_takes(a.fmt, n, a.K, 3)) {
            float *u = gu + up_to(n * a.F, 64);
            r.g = gu, r.u = u, r.ld = a.F;
            err = launch_gemv(a.fmt, a.gate, a.X + m * a.K, gu, (int)n, a.F, a.K, s);
            if (err == hipSuccess)
                err = launch_gemv(a.fmt, a.up, a.X + m * a.K, u, (int)n, a.F, a.K, s);
        }
        if (err == hipErrorNotSupported) {
            const Plan p = plan_of(FORE_GLU, n, a.F, a.K, 1);
            err = run_rows<64>(a.X + m * a.K, n, a.K, up_to(a.K, p.f.step), p.Mp, AX, ex, nullptr, s);
            if (err != hipSuccess)
                return err;
            const int64_t wide = up_to(a.F, 8);
            ProductArgs g{};
            g.W0 = a.gate, g.W1 = a.up, g.p = pl, g.A = AX, g.part = gu, g.M = n, g.ld = 2 * wide, g.rows = a.F, g.K = a.K;
            r.from = g.from = p.split_from(), r.more_ld = g.more_ld = 2 * (wide - g.from), g.more = gu + n * g.ld;
            err = launch_product(a.fmt, FORE_GLU, p, g, s);
            r.g = gu, r.u = gu + wide, r.ld = 2 * wide, r.whole = true, r.mg = g.more, r.mu = g.more + g.more_ld / 2;
            r.splits = p.splits, r.ex = ex, r.raw = true;
        }
        if (err != hipSuccess)
            return err;
        const bool held = a.F <= 8 * HELD * ROW_THREADS, vec = a.F % 8 == 0;
        if (n == 1) {
            float *D = reinterpret_cast<float *>(AD);
            const unsigned grid = (unsigned)((a.F + 511) / 512);
            const auto run = [&](auto kernel) { kernel<<<grid, 64, 0, s>>>(r, D); };
            if (a.dh_bf16)
                vec ? run(glu_one_kernel<uint16_t, true>) : run(glu_one_kernel<uint16_t, false>);
            else
                vec ? run(glu_one_kernel<float, true>) : run(glu_one_kernel<float, false>);
            err = hipGetLastError();
            if (err == hipSuccess)
                err = run_one(a.fmt, a.gate, a.up, pl, D, false, nullptr, a.F, a.K, part, a.dX + m * a.K, s);
        } else {
            const auto run = [&](auto kernel) { kernel<<<(unsigned)n, ROW_THREADS, 0, s>>>(r); };
            if (a.dh_bf16)
                held ? vec ? run(glu_rows_kernel<uint16_t, HELD, true>) : run(glu_rows_kernel<uint16_t, HELD, false>)
                     : vec ? run(glu_rows_kernel<uint16_t, HELD_LONG, true>) : run(glu_rows_kernel<uint16_t, HELD_LONG, false>);
            else
                held ? vec ? run(glu_rows_kernel<float, HELD, true>) : run(glu_rows_kernel<float, HELD, false>)
                     : vec ? run(glu_rows_kernel<float, HELD_LONG, true>) : run(glu_rows_kernel<float, HELD_LONG, false>);
            err = hipGetLastError();
            if (err == hipSuccess)
                err = run_back(a.fmt, b, a.gate, a.up, pl, AD, ed, nullptr, n, a.F, a.K, part, a.dX + m * a.K, s);
        }
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

// ---- the head's cross entropy

constexpr int kXentChunk = 26;  // log2 of the logits at once

namespace {
// runs of a row that workgroups of their own pass over: enough for the card
int64_t xent_run(int64_t M, int64_t N)
{
    int64_t runs = (2048 + M - 1) / M;
    const int64_t most = (N + 2047) / 2048;
    runs = runs > most ? most : runs;
    return up_to((N + runs - 1) / runs, 64);
}
// runs * rows: at most 2048 + rows, and at most a run of 2048 logits each
int64_t stats_bytes(int64_t R, int64_t N)
{
    const int64_t a = 2048 + R, b = R * ((N + 2047) / 2048);
    return (a < b ? a : b) * (int64_t)sizeof(Stat);
}
}  // namespace

int64_t xent_workspace(int fmt, int64_t M, int64_t N, int64_t K, bool grad)
{
    const int64_t R = chunk_rows(M, up_to(N, 64), kXentChunk);
    Pieces w{nullptr};
    w.take(panels_bytes(padded(R), K));
    w.take(4 * R);
    w.take(fore_part_bytes(R, up_to(N, 8)));
    w.take(stats_bytes(R, N));
    if (grad) {
        w.take(panels_bytes(padded(R), N));
        w.take(4 * R);
        w.take(4 * R);
        w.take(back_part_bytes(R, K));
    }
    return w.used;
}

hipError_t launch_xent(const XentArgs &a, hipStream_t s)
{
    const Planes pl = planes_of(a.fmt, a.N, a.K);
    const int64_t R = chunk_rows(a.M, up_to(a.N, 64), kXentChunk);
    Pieces w{a.ws};
    uint8_t *AX = w.take(panels_bytes(padded(R), a.K));
    int *ex = reinterpret_cast<int *>(w.take(4 * R));
    float *z = reinterpret_cast<float *>(w.take(fore_part_bytes(R, up_to(a.N, 8))));
    Stat *stats = reinterpret_cast<Stat *>(w.take(stats_bytes(R, a.N)));
    uint8_t *AD = nullptr;
    int *ed = nullptr;
    float *wd = nullptr, *part = nullptr;
    if (a.dX) {
        AD = w.take(panels_bytes(padded(R), a.N));
        ed = reinterpret_cast<int *>(w.take(4 * R));
        wd = reinterpret_cast<float *>(w.take(4 * R));
        part = reinterpret_cast<float *>(w.take(back_part_bytes(R, a.K)));
    }
    for (int64_t m = 0; m < a.M; m += R) {
        const int64_t n = a.M - m < R ? a.M - m : R;
        const uint16_t *X = a.X + m * a.K;
        const Plan b = back_plan(n, a.N, a.K, 1);
        XentRows r{};
        r.run = xent_run(n, a.N), r.runs = (int)((a.N + r.run - 1) / r.run);
        r.part = z, r.splits = 1, r.ld = a.N, r.M = n, r.N = a.N, r.Mp = b.Mp, r.sw = row_scales(a.fmt, a.W, pl), r.targets = a.targets + m;
        r.weights = a.weights ? a.weights + m : nullptr, r.stats = stats, r.e_out = ed, r.w_out = wd;
        if (n == 1)
            r.D = reinterpret_cast<float *>(AD);
        else
            r.A = AD;
        r.loss = a.loss + m, r.lse = a.lse ? a.lse + m : nullptr;
        hipError_t err = hipErrorNotSupported;
        if (gemv_takes(a.fmt, n, a.K, 4))
            err = launch_gemv(a.fmt, a.W, X, z, (int)n, a.N, a.K, s);
        if (err == hipErrorNotSupported) {
            const Plan p = plan_of(FORE_PAIR, n, a.N, a.K, 1);
            err = p.f.panel == 64 ? run_rows<64>(X, n, a.K, up_to(a.K, p.f.step), p.Mp, AX, ex, nullptr, s)
                                  : run_rows<32>(X, n, a.K, up_to(a.K, p.f.step), p.Mp, AX, ex, nullptr, s);
            if (err != hipSuccess)
                return err;
            ProductArgs g{};
            // (rows of whole groups of eight, whatever N)
            r.ld = up_to(a.N, 8);
            g.W0 = a.W, g.p = pl, g.A = AX, g.part = z, g.M = n, g.ld = r.ld, g.rows = a.N, g.K = a.K;
            r.from = g.from = p.split_from(), r.more_ld = g.more_ld = r.ld - g.from, r.more = g.more = z + n * r.ld;
            err = launch_product(a.fmt, FORE_PAIR, p, g, s);
            r.splits = p.splits, r.ex = ex, r.raw = true;
        }
        if (err != hipSuccess)
            return err;
        const dim3 grid((unsigned)r.runs, (unsigned)n), rows = a.dX ? grid : dim3(1, (unsigned)n);
        if (r.ld % 8 == 0) {
            stat_kernel<true><<<grid, 256, 0, s>>>(r);
            xent_rows_kernel<true><<<rows, 256, 0, s>>>(r);
        } else {
            stat_kernel<false><<<grid, 256, 0, s>>>(r);
            xent_rows_kernel<false><<<rows, 256, 0, s>>>(r);
        }
        err = hipGetLastError();
        if (err == hipSuccess && a.dX)
            err = n == 1 ? run_one(a.fmt, a.W, nullptr, pl, r.D, false, nullptr, a.N, a.K, part, a.dX + m * a.K, s)
                         : run_back(a.fmt, b, a.W, nullptr, pl, AD, ed, wd, n, a.N, a.K, part, a.dX + m * a.K, s);
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace ql
