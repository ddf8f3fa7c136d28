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
//   within 2^-22: its loss is fp32.  (FP8's codes are whole in hi: their lo is
//   zero, and the products with it, half of its logits' work, add nothing.)
#pragma once

#include "units.h"

namespace ql {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
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
    // unscaled sums: of the first split [M][ld], of the others [splits - 1][M]
    // [more_ld], columns from `from` on (what comes before is not split);
    // FORE_GLU: the second weight's half a row on.  Or null
    float *part, *more;
    int64_t more_ld, from;
    uint16_t *out;           // bf16 [M][ld] (backward, one split)
    int64_t M, Mp, ld;
    int64_t rows;            // rows of one weight (N or F)
    int64_t K;
    int steps, per;          // steps along the reduction, steps per split
    uint32_t tiles;          // row tiles times column tiles
    uint32_t whole;          // of them (the first, whole columns of tiles) those that are not split
};

// Consecutive workgroups go to the 8 XCDs in turn: each XCD gets a run of
// places, row tiles first, column tiles next, splits last.  The row tiles share
// their weights in its L2, the column tiles their rows of A and the lines that
// hold a row's scales: a column tile uses 16 of a line's 128 bytes of Q4K's
// headers and 2 or 3 values of Q6K's.  (Column tiles in turn over the XCDs made
// each fetch those lines: one row backward, 14336 x 4096 Q4K, 16.4 -> 14.6 us.)
__device__ __forceinline__ uint32_t xcd_run(uint32_t i, uint32_t n)
{
    const uint32_t xcd = i % 8;
    return xcd * (n / 8) + min(xcd, n % 8) + i / 8;
}
struct Place {
    uint32_t ct;
    int split, s0, s1;
    int64_t m0;
};
__device__ __forceinline__ Place place(const ProductArgs &a, int tm)
{
    const uint32_t mt = (uint32_t)(a.Mp / tm);
    // (the whole tiles and the split ones each spread evenly over the XCDs)
    uint32_t tile = xcd_run(blockIdx.x, a.whole), split = 0;
    int s0 = 0, s1 = a.steps;
    if (blockIdx.x >= a.whole) {
        const uint32_t i = xcd_run(blockIdx.x - a.whole, gridDim.x - a.whole), n = a.tiles - a.whole;
        tile = a.whole + i % n, split = i / n;
        s0 = split * a.per, s1 = min(a.steps, s0 + a.per);
    }
    return Place{tile / mt, (int)split, s0, s1, (int64_t)(tile % mt) * tm};
}

// row m of the sums of a place's split, by column
__device__ __forceinline__ float *sums_row(const ProductArgs &a, const Place &at, int64_t m)
{
    return at.split ? a.more + ((int64_t)(at.split - 1) * a.M + m) * a.more_ld - a.from : a.part + m * a.ld;
}

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
    static constexpr int UPT = UNITS / NT, TASKS = 4 * UPT;  // units a thread, tasks of eight weights
    // Up to 32 rows of A, A comes through registers as W does: the compiler's
    // own waits then let every set but the one it needs stay on its way (a wait
    // for direct loads to LDS is one for everything asked for before it).  131072
    // x 5120 Q6K, 32 rows: 170 -> 149 us; with 64 rows it makes no difference.
    // Two sets: 30 rows of 14336 x 4096 Q8_0 21.5 us, one 22.0, four 23.1.
    static constexpr bool AREG = TM <= 32;
    static constexpr int DEPTH = 2;
    // 16-byte pieces of A a thread (where there are fewer than threads, two
    // threads bring the same one)
    static constexpr int PIECES = ABYTES / 16, APT = AREG ? (PIECES + NT - 1) / NT : 1;
    static_assert(!AREG || PIECES % NT == 0 || NT % PIECES == 0, "every piece has a thread");
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

    const Place at = place(a, T::TM);
    const uint32_t ct = at.ct;
    const int64_t m0 = at.m0;
    const int s0 = at.s0, s1 = at.s1;

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
    // (a set holds a step's bytes on their way, DEPTH sets DEPTH steps')
    struct Set {
        Unit<FMT> u[T::UPT];
        u32x4 a[T::APT];
    };
    Set set[T::DEPTH];
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
    // task k of this thread (8 weights: task t of unit i) into LDS
    auto store_w = [&](Unit<FMT>(&u)[T::UPT], int k, int buf) {
        const int i = k / 4, t = k % 4;
        if (t == 0)
            u[i].begin();
        const int x = tid + i * T::NT;
        uint8_t *const w = smem + buf * T::BUF + T::ABYTES;
        uint32_t h[4];
        [[maybe_unused]] uint32_t l[4];
        if constexpr (MODE == FORE_PAIR)
            u[i].pairs(t, h, l);
        else
            u[i].halves(t, h);
        if constexpr (MODE == BACK) {
            *reinterpret_cast<uint4 *>(w + (x >> 3) * T::WPITCH + 16 * w_chunk(x >> 3, x & 7, t)) = make_uint4(h[0], h[1], h[2], h[3]);
        } else {
            constexpr int UR = BK / 32;
            const int r = x / UR, c = (x % UR) * 4 + t;
            uint8_t *const at = w + r * T::WPITCH + 16 * a_chunk<BK>(r, c);
            *reinterpret_cast<uint4 *>(at) = make_uint4(h[0], h[1], h[2], h[3]);
            if constexpr (MODE == FORE_PAIR)
                *reinterpret_cast<uint4 *>(at + T::WBYTES / 2) = make_uint4(l[0], l[1], l[2], l[3]);
        }
    };

    auto load_set = [&](int s, Set &t) {
        if constexpr (T::AREG)
#pragma unroll
            for (int i = 0; i < T::APT; i++)
                t.a[i] = *reinterpret_cast<const u32x4 *>(Abase + s * Astep + 16 * ((tid + i * T::NT) % T::PIECES));
        load_w(s, t.u);
    };
    auto store_a_regs = [&](const Set &t, int buf) {
        if constexpr (T::AREG)
#pragma unroll
            for (int i = 0; i < T::APT; i++)
                *reinterpret_cast<u32x4 *>(smem + buf * T::BUF + 16 * ((tid + i * T::NT) % T::PIECES)) = t.a[i];
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
    // step s with the next one's bytes in `t`, which it refills for DEPTH later
    auto step = [&](int s, Set &t) {
        constexpr int tasks = T::TASKS;
        store_a_regs(t, buf ^ 1);
#pragma unroll
        for (int x = 0; x + 1 < NP; x++) {
            product(x, buf, true);
#pragma unroll
            for (int k = x * tasks / (NP - 1); k < (x + 1) * tasks / (NP - 1); k++)
                store_w(t.u, k, buf ^ 1);
            // a product of the matrix cores, then decode beside it
#pragma unroll
            for (int g = 0; g < MI * NI; g++) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
            }
        }
        if constexpr (!T::AREG)
            wait_loads();
        lds_barrier();
        load_set(min(s + 1 + T::DEPTH, last), t);
        if constexpr (!T::AREG)
            issue_a(min(s + 2, last), buf);
        product(NP - 1, buf ^ 1, true);
        buf ^= 1;
        __builtin_amdgcn_sched_barrier(0);  // each step's products and decode are ordered by themselves
    };
    if (s0 < s1) {
        Set head;
        load_set(s0, head);
        if constexpr (!T::AREG) {
            issue_a(s0, 0);
            issue_a(min(s0 + 1, last), 1);
        }
#pragma unroll
        for (int i = 0; i < T::DEPTH; i++) {
            __builtin_amdgcn_sched_barrier(0);  // in this order, which the loop's waits count on
            load_set(min(s0 + 1 + i, last), set[i]);
        }
        __builtin_amdgcn_sched_barrier(0);
        store_a_regs(head, 0);
#pragma unroll
        for (int k = 0; k < T::TASKS; k++)
            store_w(head.u, k, 0);
        if constexpr (!T::AREG)
            wait_loads();
        lds_barrier();
        read_ws(0, 0);
#pragma unroll
        for (int i = 0; i < MI; i++)
            af[i] = read_a(i, 0, 0);
        // DEPTH steps a turn, each with registers of its own for the bytes on
        // their way, and no condition on a load: they are asked for whatever
        // step they are for (behind the last, the last again), so no wait
        // stands before their use.  (With the loads under conditions, or handed
        // from one set of registers to the other, the compiler waits for them
        // where they are asked for.)
        int s = s0;
        for (; s + T::DEPTH <= last; s += T::DEPTH)
#pragma unroll
            for (int i = 0; i < T::DEPTH; i++)
                step(s + i, set[i]);
#pragma unroll
        for (int i = 0; i + 1 < T::DEPTH; i++)
            if (s + i < last)
                step(s + i, set[i]);
#pragma unroll
        for (int x = 0; x < NP; x++)
            product(x, buf, x + 1 < NP);
        if constexpr (!T::AREG)
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
            float *const y = sums_row(a, at, m);
#pragma unroll
            for (int j = 0; j < NI; j++) {
                if constexpr (MODE == FORE_GLU) {
                    const int64_t c = (int64_t)ct * 128 + (wn * (NI / 2) + j % (NI / 2)) * 32 + r32;
                    if (c < ncol)
                        y[(j / (NI / 2)) * ((at.split ? a.more_ld : a.ld) / 2) + c] = acc[i][j][r];
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

// Up to 64 rows of A: the weights' bytes are what it costs, so a workgroup
// takes 64 rows of W (FORE_GLU: 32 of the gate, 32 of the up projection) and
// 128 of K a step.  Four waves: two column tiles times the two halves of a
// step's K, whose sums meet in LDS at the end.  A lane decodes a unit of its own
// row of W, eight weights a product, straight into the product's operand: the
// order of K within a step is free as long as A's is the same, so the lanes
// 0 .. 31 of a wave take one unit of the row and 32 .. 63 the next, and W never
// passes through LDS.  131072 x 5120 Q6K pairs of 3 rows take 237 us (2.3 TB/s)
// and of 64 rows 285, with W through LDS 267 and 399.  Of these 111 and 117 are
// vector instructions (416 and 440 for two steps, four clocks each); the rest
// are waits at the barrier of every step and for the memory: Q4K's loop, for
// one, waits for its second set's header in the first one's step, which nothing
// in begin() holds back.  Two steps on their way, so that three workgroups fit a
// CU (two of 64 rows); with four, 40 x 32000 of 4096 Q4K took 63 us against 47.
template <int MODE, int MI> struct Thin {
    static constexpr int TM = 32 * MI, BK = 128, NT = 256;
    static constexpr int P = MODE == FORE_PAIR ? 2 : 1;
    static constexpr int ABYTES = TM * BK * 2, SUMS = 2 * MI * 16 * 64 * 4;
    static constexpr int LDS = 2 * ABYTES > SUMS ? 2 * ABYTES : SUMS;
    static constexpr int DEPTH = 2, APT = ABYTES / 16 / NT;
};

template <int FMT, int MODE, int MI>
__global__ __launch_bounds__(256, MI == 1 ? 3 : 2) void thin_kernel(ProductArgs a)
{
    using T = Thin<MODE, MI>;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = wave & 1, kh = wave >> 1;
    const int r32 = lane & 31, half = lane >> 5;
    const Place at = place(a, T::TM);
    const uint32_t ct = at.ct;
    const int64_t m0 = at.m0;
    const int s0 = at.s0, s1 = at.s1;

    // W: unit 2 kh + half of the step, row r32 of the wave's tile
    const uint32_t upr = (uint32_t)(a.K / 32);
    const int rows = (int)a.rows, wc = 2 * kh + half;
    const int first = (MODE == FORE_GLU ? (int)ct * 32 : (int)ct * 64 + col * 32) + r32;
    const uint64_t row0 = (uint64_t)(uint32_t)min(first, rows - 1) * upr;
    const uint8_t *const W = MODE == FORE_GLU && col ? a.W1 : a.W0;
    // bytes on their way: the unit of a step, and this thread's pieces of A's
    // two panels of 64 columns for the step behind it
    struct Set {
        Unit<FMT> u;
        u32x4 a[T::APT];
    };
    Set set[T::DEPTH];
    const int64_t panel = a.Mp * 128;
    const uint8_t *const Abase = a.A + m0 * 128;
    auto load_a = [&](int s, Set &t) {
#pragma unroll
        for (int i = 0; i < T::APT; i++) {
            const int at = 16 * (tid + i * T::NT);
            t.a[i] = *reinterpret_cast<const u32x4 *>(Abase + (2 * s + at / (T::TM * 128)) * panel + at % (T::TM * 128));
        }
    };
    auto store_a_regs = [&](const Set &t, int buf) {
#pragma unroll
        for (int i = 0; i < T::APT; i++)
            *reinterpret_cast<u32x4 *>(smem + buf * T::ABYTES + 16 * (tid + i * T::NT)) = t.a[i];
    };
    const int last = s1 - 1;
    auto load_set = [&](int s, Set &t) {
        load_a(min(s + 1, last), t);
        t.u.load(W, a.p, (int64_t)(row0 + min((uint32_t)(min(s, last) * 4 + wc), upr - 1)));
    };

    f32x16 acc[MI];
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
        for (int r = 0; r < 16; r++)
            acc[i][r] = 0.0f;
    int buf = 0;
    auto step = [&](int s, Set &t) {
        // all of A's fragments, then the decode hides their way
        f16x8 af[4][MI];
#pragma unroll
        for (int x = 0; x < 4; x++)
#pragma unroll
            for (int i = 0; i < MI; i++) {
                const int row = 32 * i + r32;
                af[x][i] = *reinterpret_cast<const f16x8 *>(smem + buf * T::ABYTES + kh * (T::TM * 128) + row * 128 +
                                                            16 * a_chunk<64>(row, 4 * half + x));
            }
        store_a_regs(t, buf ^ 1);
        t.u.begin();
#pragma unroll
        for (int x = 0; x < 4; x++) {
            uint32_t h[4], l[4];
            if constexpr (MODE == FORE_PAIR)
                t.u.pairs(x, h, l);
            else
                t.u.halves(x, h);
#pragma unroll
            for (int i = 0; i < MI; i++) {
                acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[x][i], __builtin_bit_cast(f16x8, h), acc[i], 0, 0, 0);
                if constexpr (MODE == FORE_PAIR)
                    acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[x][i], __builtin_bit_cast(f16x8, l), acc[i], 0, 0, 0);
            }
        }
        load_set(s + T::DEPTH, t);
        lds_barrier();
        buf ^= 1;
    };
    if (s0 < s1) {
        Set head;
        load_a(s0, head);
#pragma unroll
        for (int i = 0; i < T::DEPTH; i++) {
            __builtin_amdgcn_sched_barrier(0);  // in this order, which the loop's waits count on
            load_set(s0 + i, set[i]);
        }
        __builtin_amdgcn_sched_barrier(0);
        store_a_regs(head, 0);
        lds_barrier();
        int s = s0;
        for (; s + T::DEPTH <= s1; s += T::DEPTH)
#pragma unroll
            for (int i = 0; i < T::DEPTH; i++)
                step(s + i, set[i]);
#pragma unroll
        for (int i = 0; i + 1 < T::DEPTH; i++)
            if (s + i < s1)
                step(s + i, set[i]);
    }
    // the halves of K meet: 64 lanes' values of a register stand together
    __syncthreads();
    float *const sum = reinterpret_cast<float *>(smem) + col * (MI * 16 * 64) + lane;
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
                sums_row(a, at, m)[(MODE == FORE_GLU ? col * ((at.split ? a.more_ld : a.ld) / 2) : 0) + c] =
                    acc[i][r] + sum[(i * 16 + r) * 64];
        }
}

// ---------------------------------------------------------------------------
// The backward product of one row
// ---------------------------------------------------------------------------

struct OneArgs {
    const uint8_t *W0, *W1;  // W1: the second weight, or null
    Planes p;
    const void *D;           // [rows] (of two weights: the second's behind the first's), fp32 or bf16
    const float *scale;      // FP8: the rows' scales still to be taken, or null
    float *part;             // [splits][K]
    int64_t rows, K;
    int per;                 // rows of 32 a split
};

// One row needs no matrix cores: a thread decodes units of its own 32 columns,
// row after row, and multiplies them by the rows' gradients in fp32 (nothing is
// rounded but the weights' own fp32 values and the sums); 8 lanes read a group
// of 256 weights, a wave 8 rows, nothing meets before the end.  Against the
// tiles of 32 rows, which also need the gradients as fp16 panels first (3.5
// us): 14336 x 4096 Q4K 13.4 against 14.6 us, Q8_0 16.1 against 18.1, 131072 x
// 5120 Q6K 122 against 141; two rows in this way 20 us, so they take the tiles.
// 2.4 to 4.5 TB/s of weights, bound by waits as much as by the decode: Q4K's 242
// vector instructions for 64 weights a lane are 5.6 of the 13 us, Q6K's 311 are
// 83 of the 122.  The sets are no prefetch: load() uses the row's gradient where
// it asks for it, and the compiler asks for most formats' units at the head of
// the turn that decodes them.
template <int FMT, typename V>
__global__ __launch_bounds__(256) void one_kernel(OneArgs a)
{
    constexpr int DEPTH = 2;  // rows a turn (131072 x 5120 Q6K: 122 us; 3, 4 and 6: 130, 131, 157)
    __shared__ float sum[32][256 + 4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int slot = wave * 8 + (lane >> 3), c = lane & 7;
    const uint32_t upr = (uint32_t)(a.K / 32);
    const uint32_t groups = (uint32_t)((a.K + 255) / 256), at = xcd_run(blockIdx.x, gridDim.x);
    const int col = (int)(at % groups), split = (int)(at / groups);
    const uint32_t unit = min((uint32_t)(col * 8 + c), upr - 1);  // behind the row's end: not stored
    const int rows = (int)a.rows, all = a.W1 ? 2 * rows : rows;
    const int n0 = split * a.per * 32 + slot;
    const int n1 = min(all, (split + 1) * a.per * 32);
    const V *const D = static_cast<const V *>(a.D);
    struct Set {
        Unit<FMT> u;
        float d;
    };
    Set set[DEPTH];
    auto load = [&](int n, Set &t) {
        const int r = min(n, all - 1);
        const bool second = r >= rows;
        t.u.load(second ? a.W1 : a.W0, a.p, (int64_t)((uint64_t)(uint32_t)(second ? r - rows : r) * upr + unit));
        if constexpr (sizeof(V) == 2)
            t.d = __builtin_bit_cast(float, (uint32_t)D[r] << 16);
        else
            t.d = D[r];
        if (FMT == FMT_FP8 && a.scale)
            t.d *= a.scale[r];
        t.d = n < n1 ? t.d : 0.0f;
    };
    float acc[32];
#pragma unroll
    for (int i = 0; i < 32; i++)
        acc[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < DEPTH; i++)
        load(n0 + 32 * i, set[i]);
    for (int n = n0; n < n1; n += 32 * DEPTH) {
#pragma unroll
        for (int i = 0; i < DEPTH; i++) {
            Set &t = set[i];
            t.u.begin();
#pragma unroll
            for (int k = 0; k < 4; k++) {
                float w[8];
                t.u.values(k, w);
#pragma unroll
                for (int j = 0; j < 8; j++)
                    acc[8 * k + j] = fmaf(t.d, w[j], acc[8 * k + j]);
            }
            load(n + 32 * (DEPTH + i), t);
        }
    }
    // the 32 rows' sums of a column meet in LDS, in this order
#pragma unroll
    for (int i = 0; i < 32; i += 4)
        *reinterpret_cast<float4 *>(&sum[slot][32 * c + i]) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    __syncthreads();
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; i++)
        v += sum[i][tid];
    const int64_t k = (int64_t)col * 256 + tid;
    if (k < a.K)
        a.part[(int64_t)split * a.K + k] = v;
}

// The shapes of a product's workgroups, by the rows of A they take.
enum { TILE_32 = 0, TILE_64 = 1, TILE_128 = 2, TILE_192 = 3, TILE_256 = 4 };

template <int FMT, int MODE>
hipError_t launch_mode(int tile, const ProductArgs &a, unsigned grid, hipStream_t s)
{
    if constexpr (MODE == BACK) {
        // (one token of 14336 x 4096 Q4K: eight waves 16.4 us, four 18.0)
        if (tile == TILE_32)
            product_kernel<FMT, MODE, 1, 8, 1, 1><<<grid, 512, 0, s>>>(a);
        else if (tile == TILE_64)
            product_kernel<FMT, MODE, 1, 4, 2, 2><<<grid, 256, 0, s>>>(a);
    } else {
        if (tile == TILE_32)
            thin_kernel<FMT, MODE, 1><<<grid, 256, 0, s>>>(a);
        else if (tile == TILE_64)
            thin_kernel<FMT, MODE, 2><<<grid, 256, 0, s>>>(a);
    }
    if (tile >= TILE_128) {
        // eight waves of 128 x 64 against four of 128 x 128: 2048 x 14336 x 4096
        // Q8_0 backward 222 against 238 us, gate and up Q4K 507 against 610.  A
        // pair's step is 256 units: four waves (eight that share units 1914
        // against 1461 us at 512 x 131072 x 5120 Q6K)
        if constexpr (MODE == FORE_PAIR) {
            if (tile == TILE_128)
                product_kernel<FMT, MODE, 2, 2, 2, 4><<<grid, 256, 0, s>>>(a);
            else if (tile == TILE_192)
                product_kernel<FMT, MODE, 2, 2, 3, 4><<<grid, 256, 0, s>>>(a);
            else
                product_kernel<FMT, MODE, 2, 2, 4, 4><<<grid, 256, 0, s>>>(a);
        } else {
            if (tile == TILE_128)
                product_kernel<FMT, MODE, 2, 4, 2, 2><<<grid, 512, 0, s>>>(a);
            else if (tile == TILE_192)
                product_kernel<FMT, MODE, 2, 4, 3, 2><<<grid, 512, 0, s>>>(a);
            else
                product_kernel<FMT, MODE, 2, 4, 4, 2><<<grid, 512, 0, s>>>(a);
        }
    }
    return hipGetLastError();
}
template <int FMT>
hipError_t launch_fmt(int mode, int tile, const ProductArgs &a, unsigned grid, hipStream_t s)
{
    switch (mode) {
    case BACK: return launch_mode<FMT, BACK>(tile, a, grid, s);
    case FORE_GLU: return launch_mode<FMT, FORE_GLU>(tile, a, grid, s);
    default: return launch_mode<FMT, FORE_PAIR>(tile, a, grid, s);
    }
}
template <int FMT> hipError_t launch_one_fmt(bool bf16, const OneArgs &a, unsigned grid, hipStream_t s)
{
    if (bf16)
        one_kernel<FMT, uint16_t><<<grid, 256, 0, s>>>(a);
    else
        one_kernel<FMT, float><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

// one instance a source file (product_*.hip)
hipError_t launch_product_q8_0(int mode, int tile, const ProductArgs &a, unsigned grid, hipStream_t s);
hipError_t launch_one_q8_0(bool bf16, const OneArgs &a, unsigned grid, hipStream_t s);
hipError_t launch_product_q4k(int mode, int tile, const ProductArgs &a, unsigned grid, hipStream_t s);
hipError_t launch_one_q4k(bool bf16, const OneArgs &a, unsigned grid, hipStream_t s);
hipError_t launch_product_q6k(int mode, int tile, const ProductArgs &a, unsigned grid, hipStream_t s);
hipError_t launch_one_q6k(bool bf16, const OneArgs &a, unsigned grid, hipStream_t s);
hipError_t launch_product_kquants(int fmt, int mode, int tile, const ProductArgs &a, unsigned grid, hipStream_t s);
hipError_t launch_one_kquants(int fmt, bool bf16, const OneArgs &a, unsigned grid, hipStream_t s);
hipError_t launch_product_legacy(int fmt, int mode, int tile, const ProductArgs &a, unsigned grid, hipStream_t s);
hipError_t launch_one_legacy(int fmt, bool bf16, const OneArgs &a, unsigned grid, hipStream_t s);

}  // namespace ql
