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

__device__ __forceinline__ float load_value(const float *p) { return *p; }
__device__ __forceinline__ float load_value(const uint16_t *p) { return __builtin_bit_cast(float, (uint32_t)*p << 16); }

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

// Rows of src [M][n] into panels.  One workgroup a row; the row is read twice
// (its largest value, then the values), the second time from the cache.
// scale: FP8's scales of the reduction's rows, or null.
template <typename V, int PK>
__global__ __launch_bounds__(256) void rows_kernel(const V *__restrict__ src, int64_t n, int64_t Mp, uint8_t *__restrict__ A,
                                                   int *__restrict__ e_out, const float *__restrict__ scale)
{
    __shared__ float red[4];
    const int64_t m = blockIdx.x;
    const V *row = src + m * n;
    float big = 0.0f;
    bool odd = false;
    for (int64_t i = threadIdx.x; i < n; i += 256) {
        const float v = fabsf(scale ? load_value(row + i) * scale[i] : load_value(row + i));
        odd |= !(v <= 3.4e38f);
        big = fmaxf(big, v);
    }
    big = block_max(odd ? INFINITY : big, red);
    const int e = row_exponent(big);
    if (threadIdx.x == 0)
        e_out[m] = e;
    const int64_t chunks = (n + PK - 1) / PK * (PK / 8);
    for (int64_t c = threadIdx.x; c < chunks; c += 256) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int64_t i = 8 * c + j;
            v[j] = i < n ? (scale ? load_value(row + i) * scale[i] : load_value(row + i)) : 0.0f;
        }
        store_a<PK>(A, Mp, m, c, v, e);
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
template <typename V>
__global__ __launch_bounds__(1024) void glu_rows_kernel(const float *__restrict__ part, int splits, int64_t M, int64_t F,
                                                        const int *__restrict__ ex, const float *__restrict__ sg,
                                                        const float *__restrict__ su, const V *__restrict__ dH, int act,
                                                        int64_t Mp, uint8_t *__restrict__ A, int *__restrict__ e_out,
                                                        uint16_t *__restrict__ dG, uint16_t *__restrict__ dU)
{
    __shared__ float red[16];
    const int64_t m = blockIdx.x;
    const int x = -ex[m];
    const int nt = blockDim.x;
    auto value = [&](int64_t f, float &dg, float &du) {
        float g = 0.0f, u = 0.0f;
        for (int s = 0; s < splits; s++) {
            const float *y = part + ((int64_t)s * M + m) * 2 * F;
            g += y[f], u += y[F + f];
        }
        g = __builtin_ldexpf(g, x), u = __builtin_ldexpf(u, x);
        if (sg)  // FP8: the rows' scales
            g *= sg[f], u *= su[f];
        glu_grad(act, g, u, load_value(dH + m * F + f), dg, du);
    };
    float big = 0.0f;
    bool odd = false;
    for (int64_t f = threadIdx.x; f < F; f += nt) {
        float dg, du;
        value(f, dg, du);
        if (dG)
            dG[m * F + f] = bf16_bits(dg);
        if (dU)
            dU[m * F + f] = bf16_bits(du);
        if (sg)
            dg *= sg[f], du *= su[f];
        const float v = fmaxf(fabsf(dg), fabsf(du));
        odd |= !(fabsf(dg) <= 3.4e38f) || !(fabsf(du) <= 3.4e38f);
        big = fmaxf(big, v);
    }
    big = block_max(odd ? INFINITY : big, red);
    const int e = row_exponent(big);
    if (threadIdx.x == 0)
        e_out[m] = e;
    const int64_t panels = (F + 63) / 64;
    for (int64_t c = threadIdx.x; c < panels * 8; c += nt) {
        float a[8], b[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int64_t f = 8 * c + j;
            a[j] = b[j] = 0.0f;
            if (f < F) {
                value(f, a[j], b[j]);
                if (sg)
                    a[j] *= sg[f], b[j] *= su[f];
            }
        }
        store_a<64>(A, Mp, m, c, a, e);
        store_a<64>(A + panels * Mp * 128, Mp, m, c, b, e);
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

__device__ __forceinline__ float logit(const float *part, int splits, int64_t stride, int64_t n, int x, const float *sw)
{
    float z = 0.0f;
    for (int s = 0; s < splits; s++)
        z += part[s * stride + n];
    z = __builtin_ldexpf(z, x);
    return sw ? z * sw[n] : z;
}

// part of row m (blockIdx.y), run blockIdx.x of it: its Stat.  The given token
// is left out: 1 - p of it is the others' share, with all of its digits.
__global__ __launch_bounds__(256) void stat_kernel(const float *__restrict__ part, int splits, int64_t M, int64_t N, int64_t run,
                                                   const int *__restrict__ ex, const float *__restrict__ sw,
                                                   const int32_t *__restrict__ targets, Stat *__restrict__ out)
{
    __shared__ float red[4];
    const int64_t m = blockIdx.y, n0 = blockIdx.x * run, n1 = min(N, n0 + run);
    const int64_t t = targets[m];
    const float *row = part + m * N;
    const int x = -ex[m];
    float big = -INFINITY;
    for (int64_t n = n0 + threadIdx.x; n < n1; n += 256)
        if (n != t)
            big = fmaxf(big, logit(row, splits, M * N, n, x, sw));
    big = block_max(big, red);
    float l = 0.0f;
    for (int64_t n = n0 + threadIdx.x; n < n1; n += 256)
        if (n != t)
            l += expf(logit(row, splits, M * N, n, x, sw) - big);
    l = block_sum(l, red);
    float sc = 0.0f;
    if (sw) {
        for (int64_t n = n0 + threadIdx.x; n < n1; n += 256)
            sc = fmaxf(sc, sw[n]);
        sc = block_max(sc, red);
    }
    if (threadIdx.x == 0)
        out[m * gridDim.x + blockIdx.x] = Stat{big, l, sc};
}

// Row m: loss and lse, and its gradient with respect to the logits as a row of
// A (a token that is not scored gives zeros).  p_n - [n = t] is at most
// max(largest p of the others, 1 - p_t) in size, which fixes the power of two;
// the row's weight enters as a factor of its own afterwards (w_out).
__global__ __launch_bounds__(256) void xent_rows_kernel(const float *__restrict__ part, int splits, int64_t M, int64_t N,
                                                        const int *__restrict__ ex, const float *__restrict__ sw,
                                                        const int32_t *__restrict__ targets, const float *__restrict__ weights,
                                                        const Stat *__restrict__ stats, int runs, int64_t run, int64_t Mp,
                                                        uint8_t *__restrict__ A, int *__restrict__ e_out, float *__restrict__ w_out,
                                                        float *__restrict__ loss, float *__restrict__ lse)
{
    const int64_t m = blockIdx.y;
    const int64_t t = targets[m];
    const bool given = t >= 0 && t < N;
    const float *row = part + m * N;
    const int x = -ex[m];
    Stat rest = stats[m * runs];
    for (int i = 1; i < runs; i++)
        rest = join(rest, stats[m * runs + i]);
    // the whole: the others and the given token
    const float zt = given ? logit(row, splits, M * N, t, x, sw) : -INFINITY;
    const float top = fmaxf(rest.m, zt);
    const float lr = rest.l * expf(rest.m - top), lt = given ? expf(zt - top) : 0.0f;
    const float l = lr + lt;
    const bool first = blockIdx.x == 0 && threadIdx.x == 0;
    if (first) {
        // ln(l / lt) = log1p(lr / lt) where the token is the likelier side
        loss[m] = !given ? 0.0f : lt > lr ? log1pf(lr / lt) : logf(l) + (top - zt);
        if (lse)
            lse[m] = logf(l) + top;
    }
    if (!A)
        return;
    const float big = fmaxf(expf(rest.m - top) / l, lr / l) * (sw ? rest.s : 1.0f);
    const float rl = 1.0f / l;
    const float gt = -lr * rl;
    const float w = given ? (weights ? weights[m] : 1.0f) : 0.0f;
    const int e = row_exponent(big);
    if (first) {
        e_out[m] = e;
        w_out[m] = w;
    }
    const int64_t c1 = min((N + 63) / 64 * 8, ((int64_t)blockIdx.x + 1) * run / 8);
    for (int64_t c = blockIdx.x * run / 8 + threadIdx.x; c < c1; c += 256) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int64_t n = 8 * c + j;
            v[j] = 0.0f;
            if (n < N && given) {
                v[j] = n == t ? gt : expf(logit(row, splits, M * N, n, x, sw) - top) * rl;
                if (sw)
                    v[j] *= sw[n];
            }
        }
        store_a<64>(A, Mp, m, c, v, e);
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
    int tile, splits;
    int64_t Mp, tiles, steps, per;
};
Plan plan_of(int64_t M, int64_t col_tiles, int64_t steps)
{
    Plan p;
    p.tile = tile_of(M);
    p.Mp = up_to(M, tile_rows(p.tile));
    p.tiles = p.Mp / tile_rows(p.tile) * col_tiles;
    p.steps = steps;
    int64_t n = split_to(p.tile) / p.tiles;
    n = n < 1 ? 1 : n > steps ? steps : n;
    p.per = (steps + n - 1) / n;
    p.splits = (int)((steps + p.per - 1) / p.per);
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
        if (a.dy_bf16)
            rows_kernel<uint16_t, 64><<<(unsigned)n, 256, 0, s>>>(static_cast<const uint16_t *>(a.dY) + m * a.N, a.N, padded(n), A, e, sw);
        else
            rows_kernel<float, 64><<<(unsigned)n, 256, 0, s>>>(static_cast<const float *>(a.dY) + m * a.N, a.N, padded(n), A, e, sw);
        hipError_t err = hipGetLastError();
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
        rows_kernel<uint16_t, 64><<<(unsigned)n, 256, 0, s>>>(a.X + m * a.K, a.K, p.Mp, AX, ex, nullptr);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
        ProductArgs g{};
        g.W0 = a.gate, g.W1 = a.up, g.p = pl, g.A = AX, g.e = ex, g.part = gu;
        g.M = n, g.Mp = p.Mp, g.ld = 2 * a.F, g.rows = a.F, g.K = a.K, g.steps = p.steps, g.per = p.per;
        err = launch_product(a.fmt, FORE_GLU, p, g, s);
        if (err != hipSuccess)
            return err;
        uint16_t *dG = a.dG ? a.dG + m * a.F : nullptr, *dU = a.dU ? a.dU + m * a.F : nullptr;
        const int nt = n <= 64 ? 1024 : 256;
        if (a.dh_bf16)
            glu_rows_kernel<uint16_t><<<(unsigned)n, nt, 0, s>>>(gu, p.splits, n, a.F, ex, sg, su,
                                                                 static_cast<const uint16_t *>(a.dH) + m * a.F, a.act, p.Mp, AD, ed,
                                                                 dG, dU);
        else
            glu_rows_kernel<float><<<(unsigned)n, nt, 0, s>>>(gu, p.splits, n, a.F, ex, sg, su,
                                                              static_cast<const float *>(a.dH) + m * a.F, a.act, p.Mp, AD, ed, dG,
                                                              dU);
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
        rows_kernel<uint16_t, 32><<<(unsigned)n, 256, 0, s>>>(a.X + m * a.K, a.K, p.Mp, AX, ex, nullptr);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
        ProductArgs g{};
        g.W0 = a.W, g.p = pl, g.A = AX, g.e = ex, g.part = z;
        g.M = n, g.Mp = p.Mp, g.ld = a.N, g.rows = a.N, g.K = a.K, g.steps = p.steps, g.per = p.per;
        err = launch_product(a.fmt, FORE_PAIR, p, g, s);
        if (err != hipSuccess)
            return err;
        const int64_t run = xent_run(n, a.N), runs = (a.N + run - 1) / run;
        const dim3 grid((unsigned)runs, (unsigned)n);
        stat_kernel<<<grid, 256, 0, s>>>(z, p.splits, n, a.N, run, ex, sw, a.targets + m, stats);
        err = hipGetLastError();
        if (err != hipSuccess)
            return err;
        xent_rows_kernel<<<a.dX ? grid : dim3(1, (unsigned)n), 256, 0, s>>>(
            z, p.splits, n, a.N, ex, sw, a.targets + m, a.weights ? a.weights + m : nullptr, stats, (int)runs, run, p.Mp, AD, ed, wd,
            a.loss + m, a.lse ? a.lse + m : nullptr);
        err = hipGetLastError();
        if (err == hipSuccess && a.dX)
            err = run_back(a.fmt, a.W, nullptr, pl, AD, ed, wd, n, a.N, a.K, part, a.dX + m * a.K, s);
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace ql
