// logprobs.hip -- log probabilities of given tokens from fp32 logits, with the
// entropy of each row, the given token's rank and the top alternatives, in
// one pass over the logits.
//
// For a row x of V logits, m = max x, z = sum e^(x - m), lse = m + ln z:
//   logprob  = x[t] - lse
//   rank     = 1 + #{x > x[t]}
//   entropy  = ln z - (sum e^(x - m) (x - m)) / z
//   top      = the `top` largest x - lse, ties to the lower index.
// The sums run online: a thread keeps (m, z, w) of the elements it has seen,
// w = sum e^(x - m) (x - m); when its maximum moves by delta = m_old - m_new,
// z <- z e^delta and w <- (w + delta z) e^delta.  Every logit is read once.
//
// x = -inf is a masked token: e^(x - m) = 0 and it is never an alternative.
// x - m is clamped at -200 (e^-200 is 0 in fp32), which keeps (x - m) e^(x - m)
// from becoming inf * 0 at masked places.  e^(x - m) is v_exp_f32 of (x - m) log2 e
// rounded once to fp32: with the constant's own rounding less than 2 |x - m| 2^-24
// of the term, which is below 2^-24 of the largest one for every x.
//
// Alternatives.  A workgroup walks its part of a row in tiles of 4096 (16
// logits per thread, the next tile's on the way).  From the first tile it
// takes a threshold: the tile is cut into 64 groups of 64, and the top-th
// largest of the 64 group maxima is a value that at least `top` logits reach,
// so no logit below it can be an alternative.  Logits at or above it are
// appended to a list in LDS, as 64-bit keys whose order is the value's and
// then the lower index's; a key's position among the list's keys is its rank.
// A list past 4 top + 16 keys is cut to its `top` best, whose last value is
// the new threshold, so that later tiles add ever fewer; a tile that would
// overflow the list (a rising row, a row of ties) is taken again after such a
// cut and with a threshold of its own, and if even that overflows (thousands
// of equal logits), by `top` rounds of a maximum over the tile, read again.
//
// Bound by the logits' bytes where there are many rows: 2048 of 131072 with eight
// alternatives, a pass of 194 to 205 us from box to box, 5.2 to 5.5 TB/s (a plain
// read reaches 6.9; the exponentials and the comparisons of 16 logits a thread run
// beside the next tile's loads).  One row is cut into 11 parts and is all latency:
// 10 us and 4 us for the join.
// Measured and not kept: 512 threads with two tiles on their way (136 registers, slower).
#include "logprobs.h"

namespace ql {
namespace {

constexpr int NT = 256;            // threads of a workgroup
constexpr int NW = NT / 64;
constexpr int QPT = 4;             // 16-byte quads per thread and tile
constexpr int TILE = NT * QPT * 4; // logits per tile
constexpr int CAP = 2048;          // keys in the list
constexpr float LOWEST = -3.4028234663852886e38f;
constexpr float CLAMP = -200.0f;
constexpr float LOG2E = 1.4426950408889634f;

// The order of fp32 values as unsigned numbers (-0 counted as +0), and back.
__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t u)
{
    return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}
// larger value first, then the lower index; 0 is below every key
__device__ __forceinline__ uint64_t key_of(float x, uint32_t i)
{
    return ((uint64_t)order_of(x) << 32) | (0xFFFFFFFFu - i);
}

// (m, z, w) of the union of two sets of logits
struct Stat {
    float m, z, w;
};
__device__ __forceinline__ void rebase(Stat &a, float m)
{
    const float d = fmaxf(a.m - m, CLAMP), c = __builtin_amdgcn_exp2f(d * LOG2E);
    a.w = fmaf(d, a.z, a.w) * c;
    a.z *= c;
    a.m = m;
}
__device__ __forceinline__ Stat join(Stat a, Stat b)
{
    const float m = fmaxf(a.m, b.m);
    rebase(a, m);
    rebase(b, m);
    return Stat{m, a.z + b.z, a.w + b.w};
}
// in a fixed order, so that a row's sums do not change from run to run
__device__ __forceinline__ Stat wave_join(Stat a)
{
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const Stat b{__shfl_xor(a.m, s), __shfl_xor(a.z, s), __shfl_xor(a.w, s)};
        a = (threadIdx.x & s) ? join(b, a) : join(a, b);
    }
    return a;
}
__device__ __forceinline__ int wave_sum(int v)
{
#pragma unroll
    for (int s = 1; s < 64; s <<= 1)
        v += __shfl_xor(v, s);
    return v;
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v)
{
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const uint64_t o = __shfl_xor(v, s);
        v = o > v ? o : v;
    }
    return v;
}

// the partner's value, lane ^ 1 (0xB1) or lane ^ 2 (0x4E)
template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}

struct Shared {
    uint64_t key[CAP];
    uint64_t best[64];     // the `top` best after a cut
    float group[64];
    float stat[NW][3];
    int cnt[NW];
    uint64_t wmax[NW];
    int count;
};

// The `top` best of the first n keys of the list, in order, to sh.best (0
// where there are fewer).  All threads; ends with a barrier.
__device__ void select_best(Shared &sh, int n, int top)
{
    if (threadIdx.x < 64)
        sh.best[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += NT) {
        const uint64_t k = sh.key[i];
        int r = 0;
        for (int j = 0; j < n; j++)
            r += sh.key[j] > k;
        if (r < top)
            sh.best[r] = k;
    }
    __syncthreads();
}

// One workgroup: part `seg` of row `row` (tiles t0 .. t1 of the row).
template <bool TOP>
__global__ __launch_bounds__(NT) void logprobs_kernel(LogprobArgs a, int segs, int tiles_per_seg, float4 *__restrict__ pstat,
                                                      uint64_t *__restrict__ pkeys)
{
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.y + (int64_t)blockIdx.z * 32768;
    if (row >= a.M)
        return;
    const int seg = blockIdx.x;
    const float *xr = a.logits + row * a.ld;
    // quads are counted from the 16-byte boundary at or below the row's
    // start: element i of the row is element i + lead of that grid
    const int lead = (int)((reinterpret_cast<uintptr_t>(xr) >> 2) & 3);
    const float *base = xr - lead;
    const int64_t t0 = (int64_t)seg * tiles_per_seg, tiles = (a.V + lead + TILE - 1) / TILE;
    const int64_t t1 = t0 + tiles_per_seg < tiles ? t0 + tiles_per_seg : tiles;

    const int32_t tgt = a.targets ? a.targets[row] : -1;
    const bool given = tgt >= 0 && tgt < a.V;
    const float xt = given ? xr[tgt] : 0.0f;

    if (tid == 0)
        sh.count = 0;
    auto load = [&](int64_t tile, float (&x)[4 * QPT]) {
        const float4 *q4 = reinterpret_cast<const float4 *>(base + tile * TILE);  // uniform
        if (tile * TILE >= lead && (tile + 1) * TILE - lead <= a.V) {             // all of the tile is in the row
#pragma unroll
            for (int q = 0; q < QPT; q++) {
                const float4 v = q4[(uint32_t)(tid + NT * q)];
                x[4 * q] = v.x, x[4 * q + 1] = v.y, x[4 * q + 2] = v.z, x[4 * q + 3] = v.w;
            }
            return;
        }
        const int left = (int)(a.V + lead - tile * TILE), skip = tile == 0 ? lead : 0;  // of the tile: its end, its start
#pragma unroll
        for (int q = 0; q < QPT; q++) {
            const int f = 4 * (tid + NT * q);
            if (f >= skip && f + 4 <= left) {
                const float4 v = q4[(uint32_t)(tid + NT * q)];
                x[4 * q] = v.x, x[4 * q + 1] = v.y, x[4 * q + 2] = v.z, x[4 * q + 3] = v.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    x[4 * q + i] = f + i >= skip && f + i < left ? base[tile * TILE + f + i] : -INFINITY;
            }
        }
    };

    Stat st{LOWEST, 0.0f, 0.0f};
    int above = 0;
    float thr = LOWEST;  // logits below it are no alternatives (inclusive)
    const int full = 4 * a.top + 16;
    float x[4 * QPT], nx[4 * QPT];
    if (t0 < t1)
        load(t0, x);
    __syncthreads();
    for (int64_t t = t0; t < t1; t++) {
        if (t + 1 < t1)
            load(t + 1, nx);
        float tm = x[0];
#pragma unroll
        for (int i = 1; i < 4 * QPT; i++)
            tm = fmaxf(tm, x[i]);
        if (tm > st.m)
            rebase(st, tm);
#pragma unroll
        for (int i = 0; i < 4 * QPT; i++) {
            const float d = fmaxf(x[i] - st.m, CLAMP), e = __builtin_amdgcn_exp2f(d * LOG2E);
            st.z += e;
            st.w = fmaf(d, e, st.w);
            above += x[i] > xt;
        }
        if constexpr (TOP) {
            // this thread's i-th logit of the tile, from memory, and its index
            auto again = [&](int i, uint32_t &e) {
                const int64_t at = t * TILE + 4 * (tid + NT * (i >> 2)) - lead + (i & 3);
                e = (uint32_t)at;
                return at >= 0 && at < a.V ? xr[at] : -INFINITY;
            };
            auto threshold = [&]() {  // from the tile's 64 group maxima
                float g = fmaxf(tm, dpp<0xB1>(tm));
                g = fmaxf(g, dpp<0x4E>(g));
                if ((lane & 3) == 0)
                    sh.group[wave * 16 + (lane >> 2)] = g;
                __syncthreads();
                // the top-th largest: the largest number that at least `top` of
                // them reach, bit by bit
                const uint32_t u = order_of(sh.group[lane]);
                uint32_t v = 0;
#pragma unroll
                for (int b = 31; b >= 0; b--) {
                    const uint32_t c = v | 1u << b;
                    if (__popcll(__ballot(u >= c)) >= a.top)
                        v = c;
                }
                thr = fmaxf(thr, value_of(v));
            };
            const uint32_t e0 = (uint32_t)(t * TILE + 4 * tid - lead);  // (V is below 2^25)
            auto push = [&]() {
                if (tm < thr)
                    return;
#pragma unroll
                for (int i = 0; i < 4 * QPT; i++) {
                    if (x[i] >= thr) {
                        const int at = atomicAdd(&sh.count, 1);
                        if (at < CAP)
                            sh.key[at] = key_of(x[i], e0 + 4 * NT * (i / 4) + i % 4);
                    }
                }
            };
            // cut the list to its best; the last of them is the threshold of
            // what follows (later elements lose ties, so strictly above it)
            auto cut = [&](int n) {
                select_best(sh, n, a.top);
                const int kept = n < a.top ? n : a.top;
                if (tid < kept)
                    sh.key[tid] = sh.best[tid];
                if (kept == a.top)
                    thr = fmaxf(thr, value_of((uint32_t)(sh.best[a.top - 1] >> 32) + 1));
                if (tid == 0)
                    sh.count = kept;
                __syncthreads();
                return kept;
            };
            const int before = sh.count;  // the last barrier is behind every change of it
            if (t == t0)
                threshold();
            else
                lds_barrier();
            push();
            lds_barrier();
            int n = sh.count;
            if (n > CAP) {  // the tile does not fit: again, with a tighter threshold
                __syncthreads();
                const int kept = cut(before);
                threshold();
                push();
                __syncthreads();
                n = sh.count;
                if (n > CAP) {
                    // thousands of equal logits: the best keys one by one, from
                    // the tile and the kept keys (in key[0 .. kept))
                    __syncthreads();
                    const uint64_t mine = tid < kept ? sh.key[tid] : 0;
                    uint64_t last = ~0ull;
                    for (int j = 0; j < a.top; j++) {
                        uint64_t b = mine < last ? mine : 0;
#pragma unroll 1
                        for (int i = 0; i < 4 * QPT; i++) {
                            uint32_t e;
                            const float v = again(i, e);
                            const uint64_t k = v >= LOWEST ? key_of(v, e) : 0;
                            b = k < last && k > b ? k : b;
                        }
                        b = wave_max(b);
                        if (lane == 0)
                            sh.wmax[wave] = b;
                        __syncthreads();
                        b = sh.wmax[0];
#pragma unroll
                        for (int w = 1; w < NW; w++)
                            b = sh.wmax[w] > b ? sh.wmax[w] : b;
                        if (tid == 0)
                            sh.best[j] = b;
                        last = b;
                        __syncthreads();
                    }
                    // at least CAP logits were there, so every best[j] is a key
                    if (tid < a.top)
                        sh.key[tid] = sh.best[tid];
                    thr = fmaxf(thr, value_of((uint32_t)(last >> 32) + 1));
                    if (tid == 0)
                        sh.count = a.top;
                    __syncthreads();
                } else if (n > full) {
                    __syncthreads();
                    cut(n);
                }
            } else if (n > full) {
                __syncthreads();
                cut(n);
            }
        }
#pragma unroll
        for (int i = 0; i < 4 * QPT; i++)
            x[i] = nx[i];
    }

    st = wave_join(st);
    above = wave_sum(above);
    if (lane == 0) {
        sh.stat[wave][0] = st.m, sh.stat[wave][1] = st.z, sh.stat[wave][2] = st.w;
        sh.cnt[wave] = above;
    }
    __syncthreads();
    if (TOP)
        select_best(sh, sh.count, a.top);
    Stat all{sh.stat[0][0], sh.stat[0][1], sh.stat[0][2]};
    int n = sh.cnt[0];
#pragma unroll
    for (int w = 1; w < NW; w++) {
        all = join(all, Stat{sh.stat[w][0], sh.stat[w][1], sh.stat[w][2]});
        n += sh.cnt[w];
    }
    if (segs > 1) {
        if (tid == 0)
            pstat[row * segs + seg] = make_float4(all.m, all.z, all.w, __int_as_float(n));
        if (TOP && tid < a.top)
            pkeys[(row * segs + seg) * a.top + tid] = sh.best[tid];
        return;
    }
    const bool some = all.z > 0.0f;
    const float lz = logf(all.z);
    if (tid == 0) {
        if (a.logprob)
            a.logprob[row] = given ? (some && xt != -INFINITY ? (xt - all.m) - lz : -INFINITY) : 0.0f;
        if (a.rank)
            a.rank[row] = given ? n + 1 : 0;
        if (a.entropy)
            a.entropy[row] = some ? lz - all.w / all.z : 0.0f;
    }
    if (TOP && tid < a.top) {
        const uint64_t k = sh.best[tid];
        const float v = value_of((uint32_t)(k >> 32));
        a.top_ids[row * a.top + tid] = k ? (int32_t)(0xFFFFFFFFu - (uint32_t)k) : -1;
        a.top_logprobs[row * a.top + tid] = k ? (v - all.m) - lz : -INFINITY;
    }
}

// Joins the parts of a row (a workgroup per row): 4 to 6 us, a launch, the parts'
// (m, z, w) in order and the rank of every part's keys among all.
__global__ __launch_bounds__(256) void logprobs_join_kernel(LogprobArgs a, int segs, const float4 *__restrict__ pstat,
                                                            const uint64_t *__restrict__ pkeys)
{
    __shared__ uint64_t key[1024], best[64];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const float *xr = a.logits + row * a.ld;
    const int nk = segs * a.top;
    for (int i = tid; i < nk; i += 256)
        key[i] = pkeys[row * nk + i];
    if (tid < 64)
        best[tid] = 0;
    Stat all{LOWEST, 0.0f, 0.0f};
    int n = 0;
    for (int s = 0; s < segs; s++) {
        const float4 p = pstat[row * segs + s];
        all = join(all, Stat{p.x, p.y, p.z});
        n += __float_as_int(p.w);
    }
    __syncthreads();
    for (int i = tid; i < nk; i += 256) {
        const uint64_t k = key[i];
        int r = 0;
        for (int j = 0; j < nk; j++)
            r += key[j] > k;
        if (k && r < a.top)
            best[r] = k;
    }
    __syncthreads();
    const int32_t tgt = a.targets ? a.targets[row] : -1;
    const bool given = tgt >= 0 && tgt < a.V, some = all.z > 0.0f;
    const float xt = given ? xr[tgt] : 0.0f, lz = logf(all.z);
    if (tid == 0) {
        if (a.logprob)
            a.logprob[row] = given ? (some && xt != -INFINITY ? (xt - all.m) - lz : -INFINITY) : 0.0f;
        if (a.rank)
            a.rank[row] = given ? n + 1 : 0;
        if (a.entropy)
            a.entropy[row] = some ? lz - all.w / all.z : 0.0f;
    }
    if (tid < a.top) {
        const uint64_t k = best[tid];
        a.top_ids[row * a.top + tid] = k ? (int32_t)(0xFFFFFFFFu - (uint32_t)k) : -1;
        a.top_logprobs[row * a.top + tid] = k ? (value_of((uint32_t)(k >> 32)) - all.m) - lz : -INFINITY;
    }
}

// Parts per row: enough workgroups for the chip (two per CU), and, where a part
// keeps at least 16 tiles, enough to even out the last round of them (six fit
// a CU: 2048 rows of 131072 are 1.3 rounds whole and 2.7 in halves, a pass of 217
// and 205 us on one box); at most 16 (more make the join longer than the pass)
// and 1024 keys to join.
struct Split {
    int segs, per;
};
Split split_of(int64_t M, int64_t V, int top)
{
    const int64_t tiles = (V + 3 + TILE - 1) / TILE;  // whatever the row's alignment
    int64_t want = (512 + M - 1) / M;
    want = want < tiles ? want : tiles;
    int64_t even = (4096 + M - 1) / M;
    even = even < tiles / 16 ? even : tiles / 16;
    want = want > even ? want : even;
    const int64_t most = top > 0 ? 1024 / top : 64;
    want = want < most ? want : most;
    want = want < 16 ? want : 16;
    const int64_t per = (tiles + want - 1) / want;
    return Split{(int)((tiles + per - 1) / per), (int)per};
}

}  // namespace

int64_t logprobs_need(int64_t M, int64_t V, int top)
{
    const Split s = split_of(M, V, top);
    return s.segs > 1 ? M * s.segs * (16 + 8 * (int64_t)top) : 0;
}

// More rows take fewer parts each, so the bytes of a call fall again as M grows;
// this is the most that any of 1 .. M rows needs.  split_of wants at least w
// parts a row up to ceil(512 / M) >= w, M <= 511 / (w - 1), or likewise with 4096
// where w parts keep 16 tiles; w parts wanted are ceil(tiles / ceil(tiles / w)).
int64_t logprobs_workspace(int64_t M, int64_t V, int top)
{
    const int64_t tiles = (V + 3 + TILE - 1) / TILE;
    int64_t parts = 0;
    for (int64_t w = 2; w <= 16 && w <= tiles; w++) {
        const int64_t rows = (w <= tiles / 16 ? 4095 : 511) / (w - 1), per = (tiles + w - 1) / w;
        const int64_t p = (M < rows ? M : rows) * ((tiles + per - 1) / per);
        parts = parts > p ? parts : p;
    }
    return parts * (16 + 8 * (int64_t)top);
}

hipError_t launch_logprobs(const LogprobArgs &a, hipStream_t s)
{
    const Split sp = split_of(a.M, a.V, a.top);
    float4 *pstat = reinterpret_cast<float4 *>(a.ws);
    uint64_t *pkeys = reinterpret_cast<uint64_t *>(a.ws + 16 * a.M * sp.segs);
    const unsigned gy = (unsigned)(a.M < 32768 ? a.M : 32768), gz = (unsigned)((a.M + 32767) / 32768);
    const dim3 grid((unsigned)sp.segs, gy, gz);
    if (a.top > 0)
        logprobs_kernel<true><<<grid, NT, 0, s>>>(a, sp.segs, sp.per, pstat, pkeys);
    else
        logprobs_kernel<false><<<grid, NT, 0, s>>>(a, sp.segs, sp.per, pstat, pkeys);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || sp.segs == 1)
        return e;
    logprobs_join_kernel<<<dim3((unsigned)a.M), 256, 0, s>>>(a, sp.segs, pstat, pkeys);
    return hipGetLastError();
}

}  // namespace ql
