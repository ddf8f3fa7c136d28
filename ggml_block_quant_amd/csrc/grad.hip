// grad.hip -- gradients through frozen quantized weights: the input gradient of
// a quantized linear layer, the gated projection's backward pass, and the
// softmax cross entropy over a quantized head with its gradient.  The matrix
// product behind them is in product.h; here stand the passes over rows around
// it, the plans (tiles, splits, chunks of rows) and the launches.
#include "grad.h"
#include "product.h"

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
    if (!(v > 0.0f) || v > 3.4e38f)
        return 0;
    return 15 - __builtin_amdgcn_frexp_expf(v);
}

// Eight neighbouring values of a row of n from i on, zeros behind its end.
// VEC: rows of whole groups of eight, 16-byte aligned.
template <bool VEC> __device__ __forceinline__ void load8(const float *row, int64_t i, int64_t n, float v[8])
{
    if constexpr (VEC) {
        const float4 a = *reinterpret_cast<const float4 *>(row + i), b = *reinterpret_cast<const float4 *>(row + i + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            v[j] = i + j < n ? row[i + j] : 0.0f;
    }
}
template <bool VEC> __device__ __forceinline__ void load8(const uint16_t *row, int64_t i, int64_t n, float v[8])
{
    if constexpr (VEC) {
        const uint4 a = *reinterpret_cast<const uint4 *>(row + i);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
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
    if constexpr (VEC) {
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; j++)
            h[j] = bf16_bits(v[2 * j]) | (uint32_t)bf16_bits(v[2 * j + 1]) << 16;
        *reinterpret_cast<uint4 *>(row + i) = make_uint4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (i + j < n)
                row[i + j] = bf16_bits(v[j]);
    }
}

// largest magnitude of eight values; infinite where one is not finite
__device__ __forceinline__ float size8(const float v[8], float big)
{
#pragma unroll
    for (int j = 0; j < 8; j++)
        big = !(fabsf(v[j]) <= 3.4e38f) ? INFINITY : fmaxf(big, fabsf(v[j]));
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

// Rows of src [M][n] into panels.  scale: FP8's scales of the reduction's
// rows, or null.
template <typename V, int PK, int H, bool VEC>
__global__ __launch_bounds__(ROW_THREADS) void rows_kernel(const V *__restrict__ src, int64_t n, int64_t Mp,
                                                           uint8_t *__restrict__ A, int *__restrict__ e_out,
                                                           const float *__restrict__ scale)
{
    __shared__ float red[ROW_THREADS / 64];
    const int64_t m = blockIdx.x;
    const V *row = src + m * n;
    const int64_t full = (n + 7) / 8, chunks = (n + PK - 1) / PK * (PK / 8);  // of eight: with values, with the zeros behind
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

// dX = the splits' sums, scaled back (K is a multiple of 32)
__global__ __launch_bounds__(256) void join_kernel(const float *__restrict__ part, const int *__restrict__ e,
                                                   const float *__restrict__ w, int splits, int64_t M, int64_t K,
                                                   uint16_t *__restrict__ out)
{
    const int64_t m = blockIdx.y, k = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (k >= K)
        return;
    float v[8] = {};
    for (int s = 0; s < splits; s++) {
        const float4 *p = reinterpret_cast<const float4 *>(part + ((int64_t)s * M + m) * K + k);
        const float4 a = p[0], b = p[1];
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
    }
    const int x = -e[m];
    const float f = w ? w[m] : 1.0f;
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; j++)
        h[j] = bf16_bits(__builtin_ldexpf(v[2 * j], x) * f) | (uint32_t)bf16_bits(__builtin_ldexpf(v[2 * j + 1], x) * f) << 16;
    *reinterpret_cast<uint4 *>(out + m * K + k) = make_uint4(h[0], h[1], h[2], h[3]);
}

// ---------------------------------------------------------------------------
// The gated pair's gradients from g and u
// ---------------------------------------------------------------------------

__device__ __forceinline__ void glu_grad(int act, float g, float u, float dh, float &dg, float &du)
{
    if (act == 1) {
        dg = g > 0.0f ? dh * u : 0.0f;
        du = g > 0.0f ? dh * g : 0.0f;
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

// One workgroup a row: g and u from the splits' sums, the two gradients (bf16
// where wanted), and both as rows of A under one power of two.
struct GluRows {
    const float *part;   // [splits][M][2][F]
    int splits, act;
    int64_t M, F, Mp;
    const int *ex;       // exponents of X's rows
    const float *sg, *su;  // FP8's scales of the rows, or null
    const void *dH;
    uint8_t *A;
    int *e_out;
    uint16_t *dG, *dU;   // or null
};
template <typename V, int H, bool VEC>
__global__ __launch_bounds__(ROW_THREADS) void glu_rows_kernel(GluRows a)
{
    __shared__ float red[ROW_THREADS / 64];
    const int64_t m = blockIdx.x, F = a.F;
    const int x = -a.ex[m];
    const V *dh = static_cast<const V *>(a.dH) + m * F;
    const int64_t panels = (F + 63) / 64, chunks = panels * 8, full = (F + 7) / 8;
    // dg and du of eight values; the bf16 results with them
    auto value = [&](int64_t c, float dg[8], float du[8], bool keep) {
        float g[8] = {}, u[8] = {}, h[8], t[8];
        for (int s = 0; s < a.splits; s++) {
            const float *y = a.part + ((int64_t)s * a.M + m) * 2 * F;
            load8<VEC>(y, 8 * c, F, t);
#pragma unroll
            for (int j = 0; j < 8; j++)
                g[j] += t[j];
            load8<VEC>(y + F, 8 * c, F, t);
#pragma unroll
            for (int j = 0; j < 8; j++)
                u[j] += t[j];
        }
        load8<VEC>(dh, 8 * c, F, h);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            float p = __builtin_ldexpf(g[j], x), q = __builtin_ldexpf(u[j], x);
            const int64_t f = min(8 * c + j, F - 1);
            if (a.sg)
                p *= a.sg[f], q *= a.su[f];
            glu_grad(a.act, p, q, h[j], dg[j], du[j]);
            if (8 * c + j >= F)  // (the sigmoid's du is dh's share of 1 / 2 at g = 0)
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
    };
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
// (l); FP8: the largest scale of the rows (s)
struct Stat {
    float m, l, s;
};
__device__ __forceinline__ Stat join(Stat a, Stat b)
{
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY)
        return Stat{m, 0.0f, fmaxf(a.s, b.s)};
    return Stat{m, a.l * expf(a.m - m) + b.l * expf(b.m - m), fmaxf(a.s, b.s)};
}

struct XentRows {
    const float *part;       // [splits][M][N]
    int splits, runs;
    int64_t M, N, run, Mp;   // runs of `run` logits (a multiple of 64), one a workgroup
    const int *ex;           // exponents of X's rows
    const float *sw;         // FP8's scales of the rows, or null
    const int32_t *targets;
    const float *weights;    // or null
    Stat *stats;             // [M][runs]
    uint8_t *A;              // or null
    int *e_out;
    float *w_out, *loss, *lse;  // lse: or null
};

__device__ __forceinline__ float logit(const XentRows &a, int64_t m, int64_t n, int x)
{
    float z = 0.0f;
    for (int s = 0; s < a.splits; s++)
        z += a.part[((int64_t)s * a.M + m) * a.N + n];
    z = __builtin_ldexpf(z, x);
    return a.sw ? z * a.sw[n] : z;
}
// logits 8 c .. 8 c + 7 of row m, -inf behind the row's end
template <bool VEC> __device__ __forceinline__ void logits8(const XentRows &a, int64_t m, int64_t c, int x, float z[8])
{
#pragma unroll
    for (int j = 0; j < 8; j++)
        z[j] = 0.0f;
    for (int s = 0; s < a.splits; s++) {
        float t[8];
        load8<VEC>(a.part + ((int64_t)s * a.M + m) * a.N, 8 * c, a.N, t);
#pragma unroll
        for (int j = 0; j < 8; j++)
            z[j] += t[j];
    }
#pragma unroll
    for (int j = 0; j < 8; j++) {
        z[j] = __builtin_ldexpf(z[j], x);
        if (a.sw)
            z[j] *= a.sw[min(8 * c + j, a.N - 1)];
        if (!VEC && 8 * c + j >= a.N)
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
    const int x = -a.ex[m];
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
// A (a token that is not scored gives zeros).  p_n - [n = t] is at most
// max(largest p of the others, 1 - p_t) in size, which fixes the power of two;
// the row's weight enters as a factor of its own afterwards (w_out).
template <bool VEC> __global__ __launch_bounds__(256) void xent_rows_kernel(XentRows a)
{
    const int64_t m = blockIdx.y;
    const int64_t t = a.targets[m];
    const bool given = t >= 0 && t < a.N;
    const int x = -a.ex[m];
    Stat rest = a.stats[m * a.runs];
    for (int i = 1; i < a.runs; i++)
        rest = join(rest, a.stats[m * a.runs + i]);
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
    if (!a.A)
        return;
    const float big = fmaxf(expf(rest.m - top) / l, lr / l) * (a.sw ? rest.s : 1.0f);
    const float rl = 1.0f / l;
    const float gt = -lr * rl;
    const int e = row_exponent(big);
    if (first) {
        a.e_out[m] = e;
        a.w_out[m] = given ? (a.weights ? a.weights[m] : 1.0f) : 0.0f;
    }
    const int64_t full = (a.N + 7) / 8, c1 = min((a.N + 63) / 64 * 8, ((int64_t)blockIdx.x + 1) * a.run / 8);
    for (int64_t c = blockIdx.x * a.run / 8 + threadIdx.x; c < c1; c += 256) {
        float v[8] = {};
        if (given && c < full) {
            logits8<VEC>(a, m, c, x, v);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                v[j] = 8 * c + j == t ? gt : expf(v[j] - top) * rl;
                if (a.sw)
                    v[j] *= a.sw[min(8 * c + j, a.N - 1)];
            }
        }
        store_a<64>(a.A, a.Mp, m, c, v, e);
    }
}

// ---------------------------------------------------------------------------
// Plans and launches
// ---------------------------------------------------------------------------

int tile_rows(int tile) { return 32 << tile; }
// rows of one call -> the tile
int tile_of(int64_t M) { return M <= 32 ? TILE_32 : M <= 64 ? TILE_64 : M <= 128 ? TILE_128 : TILE_256; }

// Workgroups that a launch may split its reduction into; also the bound of
// what the splits' sums take (splits * tiles <= this where splits > 1).
int64_t split_to(int tile) { return tile == TILE_32 ? 512 : 256; }

struct Plan {
    int tile, splits, steps, per;
    int64_t Mp, tiles;
};
Plan plan_of(int64_t M, int64_t col_tiles, int64_t steps)
{
    Plan p;
    p.tile = tile_of(M);
    p.Mp = up_to(M, tile_rows(p.tile));
    p.tiles = p.Mp / tile_rows(p.tile) * col_tiles;
    p.steps = (int)steps;
    int64_t n = split_to(p.tile) / p.tiles;
    n = n < 1 ? 1 : n > steps ? steps : n;
    p.per = (int)((steps + n - 1) / n);
    p.splits = (p.steps + p.per - 1) / p.per;
    return p;
}
// The most rows that the splits' sums of a call of up to M rows take (splits
// times rows; 0 or the call's own rows where nothing is split).  It grows with
// M, so that a workspace for M rows serves fewer.
int64_t split_rows(int64_t M, int64_t col_tiles)
{
    int64_t most = 0;
    for (int t = 0; t <= tile_of(M); t++) {
        const int64_t n = split_to(t) / col_tiles;
        if (n > 1 && n * tile_rows(t) > most)
            most = n * tile_rows(t);
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
int64_t padded(int64_t M) { return up_to(M, tile_rows(tile_of(M))); }

int64_t panels_bytes(int64_t Mp, int64_t n, int pk) { return up_to(n, pk) * Mp * 2; }

hipError_t launch_product(int fmt, int mode, const Plan &p, const ProductArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)p.tiles, (unsigned)p.splits);
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

// rows of src (M of n) into panels of PK
template <int PK, typename V>
hipError_t run_rows(const V *src, int64_t M, int64_t n, int64_t Mp, uint8_t *A, int *e, const float *scale, hipStream_t s)
{
    const bool held = n <= 8 * HELD * ROW_THREADS, vec = n % 8 == 0;
    const auto run = [&](auto kernel) { kernel<<<(unsigned)M, ROW_THREADS, 0, s>>>(src, n, Mp, A, e, scale); };
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

// dX = the backward product of A's rows over one weight or two, split or not
int64_t back_steps(int64_t rows, int weights) { return (rows + 63) / 64 * weights; }
hipError_t run_back(int fmt, const uint8_t *W0, const uint8_t *W1, const Planes &pl, const uint8_t *A, const int *e,
                    const float *w, int64_t M, int64_t rows, int64_t K, float *part, uint16_t *dX, hipStream_t s)
{
    const Plan p = plan_of(M, (K + 255) / 256, back_steps(rows, W1 ? 2 : 1));
    ProductArgs a{};
    a.W0 = W0, a.W1 = W1, a.p = pl, a.A = A, a.e = e, a.w = w;
    a.part = p.splits > 1 ? part : nullptr;
    a.out = p.splits > 1 ? nullptr : dX;
    a.M = M, a.Mp = p.Mp, a.ld = K, a.rows = rows, a.K = K, a.steps = p.steps, a.per = p.per;
    hipError_t err = launch_product(fmt, BACK, p, a, s);
    if (err != hipSuccess || p.splits == 1)
        return err;
    join_kernel<<<dim3((unsigned)((K + 2047) / 2048), (unsigned)M), 256, 0, s>>>(part, e, w, p.splits, M, K, dX);
    return hipGetLastError();
}
int64_t back_part_bytes(int64_t M, int64_t K) { return split_rows(M, (K + 255) / 256) * K * 4; }

}  // namespace

// ---- dX = dY . deq(W)

constexpr int kGradChunk = 27;  // log2 of the values of dY that go through at once (256 MiB of A)

int64_t grad_workspace(int fmt, int64_t M, int64_t N, int64_t K)
{
    const int64_t R = chunk_rows(M, up_to(N, 64), kGradChunk);
    Pieces w{nullptr};
    w.take(panels_bytes(padded(R), N, 64));
    w.take(4 * R);
    w.take(back_part_bytes(R, K));
    return w.used;
}

hipError_t launch_grad(const GradArgs &a, hipStream_t s)
{
    const Planes p = planes_of(a.fmt, a.N, a.K);
    const int64_t R = chunk_rows(a.M, up_to(a.N, 64), kGradChunk);
    Pieces w{a.ws};
    uint8_t *A = w.take(panels_bytes(padded(R), a.N, 64));
    int *e = reinterpret_cast<int *>(w.take(4 * R));
    float *part = reinterpret_cast<float *>(w.take(back_part_bytes(R, a.K)));
    const float *sw = row_scales(a.fmt, a.W, p);
    for (int64_t m = 0; m < a.M; m += R) {
        const int64_t n = a.M - m < R ? a.M - m : R;
        hipError_t err = a.dy_bf16 ? run_rows<64>(static_cast<const uint16_t *>(a.dY) + m * a.N, n, a.N, padded(n), A, e, sw, s)
                                   : run_rows<64>(static_cast<const float *>(a.dY) + m * a.N, n, a.N, padded(n), A, e, sw, s);
        if (err == hipSuccess)
            err = run_back(a.fmt, a.W, nullptr, p, A, e, nullptr, n, a.N, a.K, part, a.dX + m * a.K, s);
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

// ---- the gated pair

constexpr int kGluChunk = 26;  // log2 of the values of G (and of U) at once

namespace {
// sums of a forward product: rows of `width` values, split or not
int64_t fore_part_bytes(int64_t M, int64_t col_tiles, int64_t width)
{
    const int64_t r = split_rows(M, col_tiles);
    return (r > M ? r : M) * width * 4;
}
}  // namespace

int64_t glu_grad_workspace(int fmt, int64_t M, int64_t F, int64_t K)
{
    const int64_t R = chunk_rows(M, up_to(F, 64), kGluChunk);
    Pieces w{nullptr};
    w.take(panels_bytes(padded(R), K, 64));
    w.take(2 * panels_bytes(padded(R), F, 64));
    w.take(4 * R);
    w.take(4 * R);
    w.take(fore_part_bytes(R, (F + 127) / 128, 2 * F));
    w.take(back_part_bytes(R, K));
    return w.used;
}

hipError_t launch_glu_grad(const GluGradArgs &a, hipStream_t s)
{
    const Planes pl = planes_of(a.fmt, a.F, a.K);
    const int64_t R = chunk_rows(a.M, up_to(a.F, 64), kGluChunk);
    Pieces w{a.ws};
    uint8_t *AX = w.take(panels_bytes(padded(R), a.K, 64));
    uint8_t *AD = w.take(2 * panels_bytes(padded(R), a.F, 64));
    int *ex = reinterpret_cast<int *>(w.take(4 * R)), *ed = reinterpret_cast<int *>(w.take(4 * R));
    float *gu = reinterpret_cast<float *>(w.take(fore_part_bytes(R, (a.F + 127) / 128, 2 * a.F)));
    float *part = reinterpret_cast<float *>(w.take(back_part_bytes(R, a.K)));
    const float *sg = row_scales(a.fmt, a.gate, pl), *su = row_scales(a.fmt, a.up, pl);
    for (int64_t m = 0; m < a.M; m += R) {
        const int64_t n = a.M - m < R ? a.M - m : R;
        const Plan p = plan_of(n, (a.F + 127) / 128, (a.K + 63) / 64);
        hipError_t err = run_rows<64>(a.X + m * a.K, n, a.K, p.Mp, AX, ex, nullptr, s);
        if (err != hipSuccess)
            return err;
        ProductArgs g{};
        g.W0 = a.gate, g.W1 = a.up, g.p = pl, g.A = AX, g.e = ex, g.part = gu;
        g.M = n, g.Mp = p.Mp, g.ld = 2 * a.F, g.rows = a.F, g.K = a.K, g.steps = p.steps, g.per = p.per;
        err = launch_product(a.fmt, FORE_GLU, p, g, s);
        if (err != hipSuccess)
            return err;
        GluRows r{};
        r.part = gu, r.splits = p.splits, r.act = a.act, r.M = n, r.F = a.F, r.Mp = p.Mp, r.ex = ex, r.sg = sg, r.su = su;
        r.dH = a.dh_bf16 ? (const void *)(static_cast<const uint16_t *>(a.dH) + m * a.F)
                         : (const void *)(static_cast<const float *>(a.dH) + m * a.F);
        r.A = AD, r.e_out = ed, r.dG = a.dG ? a.dG + m * a.F : nullptr, r.dU = a.dU ? a.dU + m * a.F : nullptr;
        const bool held = a.F <= 8 * HELD * ROW_THREADS, vec = a.F % 8 == 0;
        const auto run = [&](auto kernel) { kernel<<<(unsigned)n, ROW_THREADS, 0, s>>>(r); };
        if (a.dh_bf16)
            held ? vec ? run(glu_rows_kernel<uint16_t, HELD, true>) : run(glu_rows_kernel<uint16_t, HELD, false>)
                 : vec ? run(glu_rows_kernel<uint16_t, HELD_LONG, true>) : run(glu_rows_kernel<uint16_t, HELD_LONG, false>);
        else
            held ? vec ? run(glu_rows_kernel<float, HELD, true>) : run(glu_rows_kernel<float, HELD, false>)
                 : vec ? run(glu_rows_kernel<float, HELD_LONG, true>) : run(glu_rows_kernel<float, HELD_LONG, false>);
        err = hipGetLastError();
        if (err == hipSuccess)
            err = run_back(a.fmt, a.gate, a.up, pl, AD, ed, nullptr, n, a.F, a.K, part, a.dX + m * a.K, s);
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
int64_t xent_most_runs(int64_t N) { return (N + 2047) / 2048; }
}  // namespace

int64_t xent_workspace(int fmt, int64_t M, int64_t N, int64_t K, bool grad)
{
    const int64_t R = chunk_rows(M, up_to(N, 64), kXentChunk);
    Pieces w{nullptr};
    w.take(panels_bytes(padded(R), K, 32));
    w.take(4 * R);
    w.take(fore_part_bytes(R, (N + 255) / 256, N));
    // runs * rows: at most 2048 + rows, and at most a run of 2048 logits each
    const int64_t a = 2048 + R, b = R * xent_most_runs(N);
    w.take((a < b ? a : b) * (int64_t)sizeof(Stat));
    if (grad) {
        w.take(panels_bytes(padded(R), N, 64));
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
    uint8_t *AX = w.take(panels_bytes(padded(R), a.K, 32));
    int *ex = reinterpret_cast<int *>(w.take(4 * R));
    float *z = reinterpret_cast<float *>(w.take(fore_part_bytes(R, (a.N + 255) / 256, a.N)));
    const int64_t sa = 2048 + R, sb = R * xent_most_runs(a.N);
    Stat *stats = reinterpret_cast<Stat *>(w.take((sa < sb ? sa : sb) * (int64_t)sizeof(Stat)));
    uint8_t *AD = nullptr;
    int *ed = nullptr;
    float *wd = nullptr, *part = nullptr;
    if (a.dX) {
        AD = w.take(panels_bytes(padded(R), a.N, 64));
        ed = reinterpret_cast<int *>(w.take(4 * R));
        wd = reinterpret_cast<float *>(w.take(4 * R));
        part = reinterpret_cast<float *>(w.take(back_part_bytes(R, a.K)));
    }
    const float *sw = row_scales(a.fmt, a.W, pl);
    for (int64_t m = 0; m < a.M; m += R) {
        const int64_t n = a.M - m < R ? a.M - m : R;
        const Plan p = plan_of(n, (a.N + 255) / 256, (a.K + 31) / 32);
        hipError_t err = run_rows<32>(a.X + m * a.K, n, a.K, p.Mp, AX, ex, nullptr, s);
        if (err != hipSuccess)
            return err;
        ProductArgs g{};
        g.W0 = a.W, g.p = pl, g.A = AX, g.e = ex, g.part = z;
        g.M = n, g.Mp = p.Mp, g.ld = a.N, g.rows = a.N, g.K = a.K, g.steps = p.steps, g.per = p.per;
        err = launch_product(a.fmt, FORE_PAIR, p, g, s);
        if (err != hipSuccess)
            return err;
        XentRows r{};
        r.run = xent_run(n, a.N), r.runs = (int)((a.N + r.run - 1) / r.run);
        r.part = z, r.splits = p.splits, r.M = n, r.N = a.N, r.Mp = p.Mp, r.ex = ex, r.sw = sw, r.targets = a.targets + m;
        r.weights = a.weights ? a.weights + m : nullptr, r.stats = stats, r.A = AD, r.e_out = ed, r.w_out = wd;
        r.loss = a.loss + m, r.lse = a.lse ? a.lse + m : nullptr;
        const dim3 grid((unsigned)r.runs, (unsigned)n), rows = a.dX ? grid : dim3(1, (unsigned)n);
        if (a.N % 8 == 0) {
            stat_kernel<true><<<grid, 256, 0, s>>>(r);
            xent_rows_kernel<true><<<rows, 256, 0, s>>>(r);
        } else {
            stat_kernel<false><<<grid, 256, 0, s>>>(r);
            xent_rows_kernel<false><<<rows, 256, 0, s>>>(r);
        }
        err = hipGetLastError();
        if (err == hipSuccess && a.dX)
            err = run_back(a.fmt, a.W, nullptr, pl, AD, ed, wd, n, a.N, a.K, part, a.dX + m * a.K, s);
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace ql
