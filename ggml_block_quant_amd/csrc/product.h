// product.h -- the matrix product behind the gradients and the cross entropy
// (grad.hip), instantiated per format in product_*.hip.
//
// One product serves all of them, in two directions:
//   forward   C[m][n] = sum_k A[m][k] w[n][k]   (logits, gate and up)
//   backward  C[m][k] = sum_n A[m][n] w[n][k]   (input gradients)
// on v_mfma_f32_32x32x16_f16 with fp32 sums.
//
// Fewer bits than fp32, and why:
// - A (gradients, or X) is held as fp16 times a power of two per row that puts
//   the row's largest value into [2^14, 2^15): bf16 values are then exact down
//   to 2^-31 of the row's largest; fp32 gradients keep 11 bits (2^-11 of the
//   value, down to 2^-28 of the largest).  The results are bf16 (2^-8), so
//   their own rounding is the larger part.  fp16 instead of bf16 operands: the
//   same matrix rate, an eighth of the rounding.
// - Weights are decoded to fp32 and rounded once to fp16 (2^-11).  Every block
//   format's weights are whole multiples of 2^-24, fp16's smallest step, so
//   none is lost for being small; weights above 65504 are not finite here.
// - The cross entropy's logits take each weight as an fp16 pair, w = hi + lo
//   within 2^-22: its loss is fp32.
#pragma once

#include "units.h"

namespace ql {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int64_t up_to(int64_t v, int64_t q) { return (v + q - 1) / q * q; }

// The A operand's layout: panels of PK columns, [panel][Mp rows][PK], so that
// the rows of one tile of one step are one run of bytes and reach LDS by
// direct loads as they are; the 16-byte chunks of a row stand in an order of
// the row's own.  LDS serves a 16-byte read of 16 lanes in one clock where they
// fall on all 64 banks: 16 rows' same chunk has to take each of the 256 bytes'
// 16 places once (2 rows of 128 bytes, or 4 of 64, stand beside each other).
// With chunk c at c ^ (row & 7) every such read took twice its clocks.
template <int PK> __host__ __device__ __forceinline__ int a_chunk(int row, int c)
{
    return PK == 64 ? c ^ ((row >> 1) & 7) : c ^ ((row >> 2) & 3);
}
// Backward tiles of W, 64 rows of 512 bytes: chunk i (of 4) of unit T (of 8).
// A transposing read of 32 lanes takes 64 bytes of 4 neighbouring rows, a write
// of 8 lanes the same chunk of 8 units: both fall on banks of their own.
__device__ __forceinline__ int w_chunk(int row, int T, int i) { return 4 * (T ^ (row & 3)) + (i ^ (T >> 2)); }

__device__ __forceinline__ uint16_t bf16_bits(float v)
{
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Direct global -> LDS load: lane i's 16 bytes at base + off land at lds + 16 i
// (lds uniform).  It writes no register; an explicit vmcnt wait and a barrier
// come before the bytes are read.
__device__ __forceinline__ void load_to_lds(const uint8_t *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds)
                 : "memory");
}
__device__ __forceinline__ void wait_loads()
{
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt 0, expcnt 7, lgkmcnt 15
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// ---------------------------------------------------------------------------
// The product
// ---------------------------------------------------------------------------

struct ProductArgs {
    const uint8_t *W0, *W1;  // blocks; W1: the second weight (gate and up)
    Planes p;
    const uint8_t *A;        // panels (backward of two weights: the second's behind the first's)
    const int *e;            // [M] exponents: A holds values times 2^e
    const float *w;          // [M] factors of the rows of C, or null (backward, one split)
    float *part;             // [splits][M][ld] unscaled sums, or null
    uint16_t *out;           // bf16 [M][ld] (backward, one split)
    int64_t M, Mp, ld;
    int64_t rows;            // rows of one weight (N or F)
    int64_t K;
    int steps, per;          // steps along the reduction, steps per split
};

enum { BACK = 0, FORE_PAIR = 1, FORE_GLU = 2 };


// WM x WN waves, each MI x NI tiles of 32 x 32: TM = 32 MI WM rows of A, 256
// columns of C.
//   BACK       the reduction runs over the weights' rows (first weight, then
//              the second); a tile of W is 64 rows x 256 columns
//   FORE_PAIR  over K, 32 at a time, 256 rows of W, each weight as hi + lo
//   FORE_GLU   over K, 64 at a time, 128 rows of the gate and the same 128 of
//              the up projection: a lane's tiles ni and ni + NI / 2 are the two
//              of one value
template <int FMT, int MODE, int WM, int WN, int MI, int NI>
struct Tile {
    static constexpr int TM = 32 * MI * WM, TN = 256, NT = 64 * WM * WN;
    static constexpr int BK = MODE == FORE_PAIR ? 32 : 64;
    static constexpr int WPITCH = MODE == BACK ? 512 : 2 * BK;    // bytes of a row of W in LDS
    static constexpr int WROWS = MODE == BACK ? 64 : 256;
    static constexpr int WBYTES = WROWS * WPITCH * (MODE == FORE_PAIR ? 2 : 1);
    static constexpr int ABYTES = TM * BK * 2;
    static constexpr int BUF = ABYTES + WBYTES;
    static constexpr int UNITS = MODE == BACK ? 64 * 8 : 256 * BK / 32;
    static constexpr int UPT = (UNITS + NT - 1) / NT;
    static_assert(WN * NI * 32 == TN && UNITS % NT == 0, "256 columns, whole units");
};

template <int FMT, int MODE, int WM, int WN, int MI, int NI>
__global__ __launch_bounds__(64 * WM *WN) void product_kernel(ProductArgs a)
{
    using T = Tile<FMT, MODE, WM, WN, MI, NI>;
    constexpr int BK = T::BK, KK = BK / 16;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * T::BUF];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int r32 = lane & 31, half = lane >> 5;

    // consecutive workgroups go to the 8 XCDs in turn: each XCD gets a run of
    // tiles that walks the row tiles of one column tile, whose weights then
    // stay in its L2
    const uint32_t mt = (uint32_t)(a.Mp / T::TM), ntiles = gridDim.x;
    const uint32_t xcd = blockIdx.x % 8, q = ntiles / 8, rem = ntiles % 8;
    const uint32_t tile = xcd * q + min(xcd, rem) + blockIdx.x / 8;
    const uint32_t ct = tile / mt;
    const int64_t m0 = (int64_t)(tile % mt) * T::TM;
    const int s0 = blockIdx.y * a.per, s1 = min(a.steps, s0 + a.per);

    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8 *)smem;

    // A: the tile's run of TM * BK * 2 bytes, 1024 a wave and load
    const uint8_t *const Abase = a.A + m0 * (BK * 2);
    const int64_t Astep = a.Mp * (BK * 2);
    auto issue_a = [&](int s, int buf) {
        const uint8_t *src = Abase + s * Astep;
#pragma unroll
        for (int i = 0; i < T::ABYTES / 1024; i += WM * WN)
            if (T::ABYTES / 1024 % (WM * WN) == 0 || i + wave < T::ABYTES / 1024)
                load_to_lds(src, (uint32_t)((i + wave) * 1024 + 16 * lane), lds0 + buf * T::BUF + (i + wave) * 1024);
    };

    // W: this thread's units of a step, registers between load and decode
    // (rows are below 2^24, units of a row below 2^15: 32 x 32 -> 64 bits)
    const uint32_t upr = (uint32_t)(a.K / 32);  // units in a row of W
    const int rows = (int)a.rows, halfsteps = (rows + 63) / 64;
    // (two sets: a step's bytes are asked for while the step two before it runs)
    Unit<FMT> un[2][T::UPT];
    auto load_w = [&](int s, Unit<FMT>(&u)[T::UPT]) {
#pragma unroll
        for (int i = 0; i < T::UPT; i++) {
            const int x = tid + i * T::NT;
            if constexpr (MODE == BACK) {
                // row x / 8 of the step, unit x % 8 of the tile's columns
                // (rows past the end meet zeros of A, columns past it are not
                // stored: both read the last one instead)
                const bool second = s >= halfsteps;
                const uint32_t row = min((second ? s - halfsteps : s) * 64 + (x >> 3), rows - 1);
                const uint32_t c = min(ct * 8 + (x & 7), upr - 1);
                u[i].load(second ? a.W1 : a.W0, a.p, (int64_t)((uint64_t)row * upr + c));
            } else {
                constexpr int UR = BK / 32;  // units of a row in a step
                const int r = x / UR;
                const uint32_t c = min((uint32_t)(s * UR + x % UR), upr - 1);  // past the row's end: zeros of A
                const int first = MODE == FORE_GLU ? (int)ct * 128 + (r & 127) : (int)ct * 256 + r;
                const uint32_t row = min(first, rows - 1);
                u[i].load(MODE == FORE_GLU && r >= 128 ? a.W1 : a.W0, a.p, (int64_t)((uint64_t)row * upr + c));
            }
        }
    };
    // task t (8 elements) of unit i into LDS
    auto store_w = [&](Unit<FMT>(&u)[T::UPT], int i, int t, int buf) {
        if (t == 0)
            u[i].begin();
        const int x = tid + i * T::NT;
        uint8_t *const w = smem + buf * T::BUF + T::ABYTES;
        uint32_t h[4];
        [[maybe_unused]] float v[8];
        if constexpr (MODE == FORE_PAIR) {
            u[i].decode(t, v);
#pragma unroll
            for (int j = 0; j < 4; j++)
                h[j] = pack_f16(v[2 * j], v[2 * j + 1]);
        } else {
            u[i].halves(t, h);
        }
        if constexpr (MODE == BACK) {
            *reinterpret_cast<uint4 *>(w + (x >> 3) * T::WPITCH + 16 * w_chunk(x >> 3, x & 7, t)) = make_uint4(h[0], h[1], h[2], h[3]);
        } else {
            constexpr int UR = BK / 32;
            const int r = x / UR, c = (x % UR) * 4 + t;
            uint8_t *const at = w + r * T::WPITCH + 16 * a_chunk<BK>(r, c);
            *reinterpret_cast<uint4 *>(at) = make_uint4(h[0], h[1], h[2], h[3]);
            if constexpr (MODE == FORE_PAIR) {
                uint32_t l[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const f16x2 p = __builtin_bit_cast(f16x2, h[j]);
                    l[j] = pack_f16(v[2 * j] - (float)p.x, v[2 * j + 1] - (float)p.y);
                }
                *reinterpret_cast<uint4 *>(at + T::WBYTES / 2) = make_uint4(l[0], l[1], l[2], l[3]);
            }
        }
    };

    f32x16 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
        for (int j = 0; j < NI; j++)
#pragma unroll
            for (int r = 0; r < 16; r++)
                acc[i][j][r] = 0.0f;

    auto read_a = [&](int i, int kk, int buf) {
        const int row = (wm * MI + i) * 32 + r32;
        return *reinterpret_cast<const f16x8 *>(smem + buf * T::BUF + row * (BK * 2) + 16 * a_chunk<BK>(row, 2 * kk + half));
    };
    auto read_w = [&](int j, int kk, int buf, int plane) {
        const uint8_t *w = smem + buf * T::BUF + T::ABYTES;
        if constexpr (MODE == BACK) {
            // 8 rows of W at this lane's column: two transposing reads, each of
            // which gives lane i of 16 the column i of 4 rows x 16 columns
            // whose pieces of 4 the lanes 4 row + column / 4 point at
            // (row and row + 4 share their chunks' order)
            const int row = kk * 16 + 8 * half + ((lane >> 2) & 3);
            const uint8_t *at = w + row * T::WPITCH + 8 * (lane & 1) +
                                16 * w_chunk(row, wn * NI + j, 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1));
            union {
                s16x4 q[2];
                f16x8 v;
            } r;
            r.q[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(lds_u8 *)at);
            r.q[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(lds_u8 *)(at + 4 * T::WPITCH));
            return r.v;
        } else {
            // FORE_GLU: the wave's first tiles from the gate's rows, the others
            // from the up projection's
            const int row = MODE == FORE_GLU ? (j / (NI / 2)) * 128 + (wn * (NI / 2) + j % (NI / 2)) * 32 + r32
                                             : (wn * NI + j) * 32 + r32;
            return *reinterpret_cast<const f16x8 *>(w + plane * (T::WBYTES / 2) + row * T::WPITCH +
                                                    16 * a_chunk<BK>(row, 2 * kk + half));
        }
    };

    // A step's products.  Each leaves the next one's fragments behind it: A's
    // in the registers of those it is done with, W's in the other set.  The
    // workgroup's one barrier a step stands before the last product, whose
    // fragments are in registers by then: behind it nobody reads this step's
    // buffer any more, the next step's is filled, and the last product runs
    // while the next step's first fragments are read and the loads of the step
    // after it are asked for.
    constexpr int P = MODE == FORE_PAIR ? 2 : 1, NP = KK * P;  // kk, of it hi and lo
    static_assert(NP % 2 == 0, "a step's first fragments stand in the first registers");
    f16x8 af[MI], wf[2][NI];
    auto read_ws = [&](int x, int from) {
#pragma unroll
        for (int j = 0; j < NI; j++)
            wf[x & 1][j] = read_w(j, x / P % KK, from, x % P);
    };
    auto product = [&](int x, int from, bool next) {
        if (next)
            read_ws(x + 1, from);
#pragma unroll
        for (int i = 0; i < MI; i++) {
#pragma unroll
            for (int j = 0; j < NI; j++)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[i], wf[x & 1][j], acc[i][j], 0, 0, 0);
            if (next && x % P == P - 1)
                af[i] = read_a(i, (x + 1) / P % KK, from);
        }
    };
    int buf = 0;
    const int last = s1 - 1;
    // step s with the next one's weights in `u`, which it refills for s + 3
    auto step = [&](int s, Unit<FMT>(&u)[T::UPT]) {
        constexpr int tasks = 4 * T::UPT;
#pragma unroll
        for (int x = 0; x + 1 < NP; x++) {
            product(x, buf, true);
#pragma unroll
            for (int t = x * tasks / (NP - 1); t < (x + 1) * tasks / (NP - 1); t++)
                store_w(u, t / 4, t % 4, buf ^ 1);
            // a product of the matrix cores, then decode beside it
#pragma unroll
            for (int g = 0; g < MI * NI; g++) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
            }
        }
        wait_loads();
        lds_barrier();
        load_w(min(s + 3, last), u);
        issue_a(min(s + 2, last), buf);
        product(NP - 1, buf ^ 1, true);
        buf ^= 1;
    };
    if (s0 < s1) {
        load_w(s0, un[1]);
        issue_a(s0, 0);
        load_w(min(s0 + 1, last), un[0]);
#pragma unroll
        for (int i = 0; i < T::UPT; i++)
#pragma unroll
            for (int t = 0; t < 4; t++)
                store_w(un[1], i, t, 0);
        load_w(min(s0 + 2, last), un[1]);
        issue_a(min(s0 + 1, last), 1);
        wait_loads();
        lds_barrier();
        read_ws(0, 0);
#pragma unroll
        for (int i = 0; i < MI; i++)
            af[i] = read_a(i, 0, 0);
        // Two steps a turn, each with registers of its own for the weights on
        // their way, and no branch in it: loads are asked for whatever step
        // they are for (behind the last, the last again) and waited for a step
        // later, so no wait stands before their use.  (With the loads under
        // conditions, or handed from one set of registers to the other, the
        // compiler waits for them where they are asked for.)
        int s = s0;
        for (; s + 1 < last; s += 2) {
            step(s, un[0]);
            step(s + 1, un[1]);
        }
        if (s < last)
            step(s, un[0]);
#pragma unroll
        for (int x = 0; x < NP; x++)
            product(x, buf, x + 1 < NP);
        wait_loads();  // none may land in LDS after the workgroup's end
    }

    // register r of a lane: row 8 (r / 4) + 4 half + r % 4, column r32 of its tile
    const int64_t ncol = MODE == BACK ? a.K : a.rows;
#pragma unroll
    for (int i = 0; i < MI; i++) {
        const int64_t mr = m0 + (wm * MI + i) * 32 + 4 * half;
#pragma unroll
        for (int r = 0; r < 16; r++) {
            const int64_t m = mr + 8 * (r / 4) + r % 4;
            if (m >= a.M)
                continue;
            if constexpr (MODE == BACK) {
                if (a.out) {
                    const int e = -a.e[m];
                    const float f = a.w ? a.w[m] : 1.0f;
#pragma unroll
                    for (int j = 0; j < NI; j++) {
                        const int64_t c = (int64_t)ct * 256 + (wn * NI + j) * 32 + r32;
                        if (c < ncol)
                            a.out[m * a.ld + c] = bf16_bits(__builtin_ldexpf(acc[i][j][r], e) * f);
                    }
                    continue;
                }
            }
            float *const y = a.part + ((int64_t)blockIdx.y * a.M + m) * a.ld;
#pragma unroll
            for (int j = 0; j < NI; j++) {
                if constexpr (MODE == FORE_GLU) {
                    const int64_t c = (int64_t)ct * 128 + (wn * (NI / 2) + j % (NI / 2)) * 32 + r32;
                    if (c < ncol)
                        y[(j / (NI / 2)) * ncol + c] = acc[i][j][r];
                } else {
                    const int64_t c = (int64_t)ct * 256 + (wn * NI + j) * 32 + r32;
                    if (c < ncol)
                        y[c] = acc[i][j][r];
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The forward product of few rows
// ---------------------------------------------------------------------------

// Up to 128 rows of A: the weights' bytes are what it costs, so a workgroup
// takes 64 rows of W (FORE_GLU: 32 of the gate, 32 of the up projection) and
// 128 of K a step, which its lanes read as runs of a row (in the tiles above
// every lane reads another row, 32 or 64 elements at a time: at one row of A
// that fetched each line of the head several times, 1090 us).  Four waves: two
// column tiles times the two halves of a step's K, whose sums meet in LDS at
// the end.  The steps run as in product_kernel.
template <int MODE, int MI> struct Thin {
    static constexpr int TM = 32 * MI, BK = 128, NT = 256;
    static constexpr int P = MODE == FORE_PAIR ? 2 : 1;
    static constexpr int ABYTES = TM * BK * 2, WPLANE = 64 * BK * 2, BUF = ABYTES + P * WPLANE;
};

template <int FMT, int MODE, int MI>
__global__ __launch_bounds__(256) void thin_kernel(ProductArgs a)
{
    using T = Thin<MODE, MI>;
    constexpr int P = T::P, NP = 4 * P;  // a wave's products of a step: four of 16, of each hi and lo
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * T::BUF];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = wave & 1, kh = wave >> 1;
    const int r32 = lane & 31, half = lane >> 5;
    const uint32_t mt = (uint32_t)(a.Mp / T::TM), ntiles = gridDim.x;
    const uint32_t xcd = blockIdx.x % 8, q = ntiles / 8, rem = ntiles % 8;
    const uint32_t tile = xcd * q + min(xcd, rem) + blockIdx.x / 8;
    const uint32_t ct = tile / mt;
    const int64_t m0 = (int64_t)(tile % mt) * T::TM;
    const int s0 = blockIdx.y * a.per, s1 = min(a.steps, s0 + a.per);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8 *)smem;

    // A: two panels of 64 columns a step
    auto issue_a = [&](int s, int buf) {
#pragma unroll
        for (int i = 0; i < T::ABYTES / 1024; i += 4) {
            const int at = (i + wave) * 1024;  // of the step's bytes
            const int panel = at / (T::TM * 128);
            load_to_lds(a.A + (((int64_t)2 * s + panel) * a.Mp + m0) * 128, (uint32_t)(at % (T::TM * 128) + 16 * lane),
                        lds0 + buf * T::BUF + at);
        }
    };
    // W: unit tid % 4 of the step, row tid / 4 of the tile
    const uint32_t upr = (uint32_t)(a.K / 32);
    const int rows = (int)a.rows, wr = tid >> 2, wc = tid & 3;
    const int first = MODE == FORE_GLU ? (int)ct * 32 + (wr & 31) : (int)ct * 64 + wr;
    const uint64_t row0 = (uint64_t)(uint32_t)min(first, rows - 1) * upr;
    const uint8_t *const W = MODE == FORE_GLU && wr >= 32 ? a.W1 : a.W0;
    Unit<FMT> un[2];
    auto load_w = [&](int s, Unit<FMT> &u) { u.load(W, a.p, (int64_t)(row0 + min((uint32_t)(s * 4 + wc), upr - 1))); };
    // chunk c of row r of a tile of W: 16 rows' same chunk on all banks, and a
    // row's units' same task on banks of their own
    auto w_at = [&](int r, int c) { return r * 256 + 16 * ((4 * (c >> 2) + ((c & 3) ^ (c >> 2))) ^ (r & 15)); };
    auto store_w = [&](Unit<FMT> &u, int t, int buf) {
        if (t == 0)
            u.begin();
        uint8_t *const at = smem + buf * T::BUF + T::ABYTES + w_at(wr, 4 * wc + t);
        uint32_t h[4];
        if constexpr (MODE == FORE_PAIR) {
            float v[8];
            uint32_t l[4];
            u.decode(t, v);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                h[j] = pack_f16(v[2 * j], v[2 * j + 1]);
                const f16x2 p = __builtin_bit_cast(f16x2, h[j]);
                l[j] = pack_f16(v[2 * j] - (float)p.x, v[2 * j + 1] - (float)p.y);
            }
            *reinterpret_cast<uint4 *>(at + T::WPLANE) = make_uint4(l[0], l[1], l[2], l[3]);
        } else {
            u.halves(t, h);
        }
        *reinterpret_cast<uint4 *>(at) = make_uint4(h[0], h[1], h[2], h[3]);
    };

    f32x16 acc[MI];
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
        for (int r = 0; r < 16; r++)
            acc[i][r] = 0.0f;
    // product x of buffer `from`: columns 16 (x / P) of the wave's half
    auto product = [&](int x, int from) {
        const int kk = x / P % 4;
        const uint8_t *const b = smem + from * T::BUF;
        const f16x8 w = *reinterpret_cast<const f16x8 *>(b + T::ABYTES + (x % P) * T::WPLANE +
                                                         w_at(col * 32 + r32, 8 * kh + 2 * kk + half));
#pragma unroll
        for (int i = 0; i < MI; i++) {
            const int row = 32 * i + r32;
            const f16x8 x8 = *reinterpret_cast<const f16x8 *>(b + kh * (T::TM * 128) + row * 128 + 16 * a_chunk<64>(row, 2 * kk + half));
            acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x8, w, acc[i], 0, 0, 0);
        }
    };
    int buf = 0;
    const int last = s1 - 1;
    auto step = [&](int s, Unit<FMT> &u) {
#pragma unroll
        for (int x = 0; x < NP; x++) {
            product(x, buf);
            if (x < 4)
                store_w(u, x, buf ^ 1);
        }
        wait_loads();
        lds_barrier();
        load_w(min(s + 3, last), u);
        issue_a(min(s + 2, last), buf);
        buf ^= 1;
    };
    if (s0 < s1) {
        load_w(s0, un[1]);
        issue_a(s0, 0);
        load_w(min(s0 + 1, last), un[0]);
#pragma unroll
        for (int t = 0; t < 4; t++)
            store_w(un[1], t, 0);
        load_w(min(s0 + 2, last), un[1]);
        issue_a(min(s0 + 1, last), 1);
        wait_loads();
        lds_barrier();
        int s = s0;
        for (; s + 1 < last; s += 2) {
            step(s, un[0]);
            step(s + 1, un[1]);
        }
        if (s < last)
            step(s, un[0]);
#pragma unroll
        for (int x = 0; x < NP; x++)
            product(x, buf);
        wait_loads();  // none may land in LDS after this
    }
    // the halves of K meet: 64 lanes' values of a register stand together
    __syncthreads();
    float *const sum = reinterpret_cast<float *>(smem) + col * (MI * 16 * 64) + lane;
    static_assert(2 * MI * 16 * 64 * 4 <= 2 * T::BUF, "room for the halves' sums");
    if (kh == 1)
#pragma unroll
        for (int i = 0; i < MI; i++)
#pragma unroll
            for (int r = 0; r < 16; r++)
                sum[(i * 16 + r) * 64] = acc[i][r];
    __syncthreads();
    if (kh == 1)
        return;
    const int64_t c = MODE == FORE_GLU ? (int64_t)ct * 32 + r32 : (int64_t)ct * 64 + col * 32 + r32;
    if (c >= a.rows)
        return;
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
        for (int r = 0; r < 16; r++) {
            const int64_t m = m0 + 32 * i + 8 * (r / 4) + 4 * half + r % 4;
            if (m < a.M)
                a.part[((int64_t)blockIdx.y * a.M + m) * a.ld + (MODE == FORE_GLU ? col * a.rows : 0) + c] =
                    acc[i][r] + sum[(i * 16 + r) * 64];
        }
}

// The shapes of a product's workgroups, by the rows of A they take.
enum { TILE_32 = 0, TILE_64 = 1, TILE_128 = 2, TILE_256 = 3 };

template <int FMT, int MODE>
hipError_t launch_mode(int tile, const ProductArgs &a, dim3 grid, hipStream_t s)
{
    switch (tile) {
    case TILE_32: product_kernel<FMT, MODE, 1, 4, 1, 2><<<grid, 256, 0, s>>>(a); break;
    case TILE_64: product_kernel<FMT, MODE, 1, 4, 2, 2><<<grid, 256, 0, s>>>(a); break;
    case TILE_128: product_kernel<FMT, MODE, 2, 2, 2, 4><<<grid, 256, 0, s>>>(a); break;
    default:
        // (a pair's step is 256 units: four waves)
        if constexpr (MODE == FORE_PAIR)
            product_kernel<FMT, MODE, 2, 2, 4, 4><<<grid, 256, 0, s>>>(a);
        else
            product_kernel<FMT, MODE, 2, 4, 4, 2><<<grid, 512, 0, s>>>(a);
        break;
    }
    return hipGetLastError();
}
template <int FMT>
hipError_t launch_fmt(int mode, int tile, const ProductArgs &a, dim3 grid, hipStream_t s)
{
    switch (mode) {
    case BACK: return launch_mode<FMT, BACK>(tile, a, grid, s);
    case FORE_GLU: return launch_mode<FMT, FORE_GLU>(tile, a, grid, s);
    default: return launch_mode<FMT, FORE_PAIR>(tile, a, grid, s);
    }
}

// one instance a source file (product_*.hip)
hipError_t launch_product_q8_0(int mode, int tile, const ProductArgs &a, dim3 grid, hipStream_t s);
hipError_t launch_product_q4k(int mode, int tile, const ProductArgs &a, dim3 grid, hipStream_t s);
hipError_t launch_product_q6k(int mode, int tile, const ProductArgs &a, dim3 grid, hipStream_t s);
hipError_t launch_product_kquants(int fmt, int mode, int tile, const ProductArgs &a, dim3 grid, hipStream_t s);
hipError_t launch_product_legacy(int fmt, int mode, int tile, const ProductArgs &a, dim3 grid, hipStream_t s);

}  // namespace ql
