// api.hip -- the C ABI declared in include/qlinear.h: argument checks, path
// selection and launches.  Every check happens before any HIP call, so an
// argument error never launches anything.
#include "../../include/qlinear.h"
#include "gemv_fp8.h"
#include "grad.h"
#include "logprobs.h"
#include "moe.h"
#include "qlinear_internal.h"

#include <stdint.h>

#include <atomic>
#include <mutex>

namespace {

bool implemented(int fmt)
{
    return fmt == QFMT_Q8_0 || fmt == QFMT_Q4K || fmt == QFMT_Q6K || ql::generic_fmt(fmt);
}
bool known(int fmt) { return fmt >= QFMT_Q8_0 && fmt <= QFMT_FP8; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int64_t kMaxElems = int64_t(1) << 40;

// shape of a [rows][K] tensor in `fmt`: K % 256 (Q8_0: K % 32)
int check_tensor(int fmt, int64_t rows, int64_t K, int64_t max_rows)
{
    if (rows < 1 || rows > max_rows || K < 1 || K > QLINEAR_MAX_K)
        return Q_ESHAPE;
    if (K % (fmt == QFMT_Q8_0 ? 32 : 256) != 0)
        return Q_ESHAPE;
    if (rows * K > kMaxElems)
        return Q_ESHAPE;
    return Q_OK;
}

int status_of(hipError_t e)
{
    if (e == hipSuccess)
        return Q_OK;
    if (e == hipErrorNotSupported)
        return Q_ENOTSUP;
    return Q_EHIP;
}

hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

int matmul_args(int fmt, const void *blocks, const void *X, const float *Y, int64_t M, int64_t N,
                int64_t K)
{
    if (!known(fmt))
        return Q_EINVAL;
    if (!implemented(fmt))
        return Q_ENOTSUP;
    if (!blocks || !X || !Y)
        return Q_EINVAL;
    if (!aligned16(blocks) || !aligned16(X) || !aligned16(Y))
        return Q_EALIGN;
    // K % 256 (Q8_0: K % 32, the tail of whole blocks)
    const int kq = fmt == QFMT_Q8_0 ? 32 : 256;
    if (M < 1 || M > QLINEAR_MAX_M || N < 1 || N > QLINEAR_MAX_N || K < kq || K > QLINEAR_MAX_K || K % kq != 0 ||
        N * K > kMaxElems || M * K > kMaxElems || M * N > kMaxElems)
        return Q_ESHAPE;
    return Q_OK;
}

// shapes of a mixture-of-experts call: stacked [E*F][K] gate and up weights,
// stacked [E*K][F] down weights
int moe_shape(int fmt_gu, int fmt_d, int64_t T, int64_t E, int64_t k, int64_t F, int64_t K)
{
    if (!implemented(fmt_gu) || !implemented(fmt_d))
        return Q_ENOTSUP;
    if (T < 0 || T > QLINEAR_MAX_M || E < 1 || E > QLINEAR_MAX_EXPERTS || k < 1 || k > QLINEAR_MAX_TOP_K || F < 1 ||
        F > QLINEAR_MAX_K || K < 1 || K > QLINEAR_MAX_K)
        return Q_ESHAPE;
    if (check_tensor(fmt_gu, E * F, K, QLINEAR_MAX_N) != Q_OK || check_tensor(fmt_d, E * K, F, QLINEAR_MAX_N) != Q_OK)
        return Q_ESHAPE;
    // (a workspace below 2^40 bytes: 8.5 per value of H, 4 per value of the
    // down product, X; launches stay below 2^32 threads in each dimension)
    if (T * k * F > (int64_t(1) << 36) || T * k * K > (int64_t(1) << 36))
        return Q_ESHAPE;
    return Q_OK;
}

// the parts of the log-probability calls that do not depend on the logits
int logprob_args(const int32_t *targets, int top_n, const float *logprob, const int32_t *rank, const float *entropy,
                 const int32_t *top_ids, const float *top_logprobs)
{
    if (top_n < 0 || top_n > QLINEAR_MAX_TOP_N)
        return Q_ESHAPE;
    if ((logprob || rank) && !targets)
        return Q_EINVAL;
    if (top_n > 0 && (!top_ids || !top_logprobs))
        return Q_EINVAL;
    if (!logprob && !rank && !entropy && top_n == 0)
        return Q_EINVAL;  // nothing to compute
    if (!aligned4(targets) || !aligned4(logprob) || !aligned4(rank) || !aligned4(entropy) || !aligned4(top_ids) ||
        !aligned4(top_logprobs))
        return Q_EALIGN;
    return Q_OK;
}

// qmatmul_logprobs keeps at most 2^26 logits (256 MiB, the size of the last
// cache) at a time, in whole tiles of the prefill kernel where more than one
// tile of rows fits
int64_t head_rows(int64_t M, int64_t N)
{
    int64_t rows = ((int64_t)1 << 26) / N;
    rows = rows >= 256 ? rows / 256 * 256 : rows < 1 ? 1 : rows;
    return rows < M ? rows : M;
}
size_t head_logits_bytes(int64_t rows, int64_t N) { return (size_t)ql::up16(4 * rows * N); }
// partial results of the full chunks and of the last, shorter one
int64_t head_parts_need(int64_t M, int64_t rows, int64_t N, int top_n)
{
    const int64_t a = ql::logprobs_need(rows, N, top_n), last = M % rows;
    const int64_t b = last ? ql::logprobs_need(last, N, top_n) : 0;
    return a > b ? a : b;
}

// shapes of a gradient call on one or two [rows][K] weights
int grad_shape(int fmt, int64_t M, int64_t rows, int64_t K)
{
    const int st = check_tensor(fmt, rows, K, QLINEAR_MAX_N);
    if (st != Q_OK)
        return st;
    if (M < 0 || M > QLINEAR_MAX_M || M * K > kMaxElems || M * rows > kMaxElems)
        return Q_ESHAPE;
    return Q_OK;
}

int workspace_args(const void *workspace, size_t have, size_t need)
{
    if (!workspace)
        return Q_EINVAL;
    if (!aligned16(workspace))
        return Q_EALIGN;
    return have < need ? Q_EINVAL : Q_OK;
}

// the GEMV of a format: FP8 one- and two-token shapes on their own one-shot
// kernel, everything else on the GEMV kernels of the format
int gemv(int fmt, const uint8_t *B, const uint16_t *X, float *Y, int64_t M, int64_t N, int64_t K, hipStream_t s)
{
    if (fmt == QFMT_FP8) {
        hipError_t e = hipSuccess;
        if (ql::launch_gemv_fp8(B, X, Y, (int)M, N, K, s, e))
            return status_of(e);
    }
    return status_of(ql::launch_gemv(fmt, B, X, Y, (int)M, N, K, s));
}

// The fixed device buffer of qmatmul_static: one copy per GPU, held until the
// process ends.  Host code never uses the array's name as an address: the
// device address of each GPU's copy comes from hipGetSymbolAddress, taken
// once per device with that device current.
__device__ __align__(256) uint8_t scratch[QLINEAR_STATIC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::atomic<void *> scratch_addr[kMaxDevices];
std::mutex scratch_mu;

int scratch_of_current_device(void **out)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess)
        return Q_EHIP;
    if (dev < 0 || dev >= kMaxDevices)
        return Q_ENOTSUP;
    void *p = scratch_addr[dev].load(std::memory_order_acquire);
    if (!p) {
        std::lock_guard<std::mutex> lock(scratch_mu);
        p = scratch_addr[dev].load(std::memory_order_relaxed);
        if (!p) {
            if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p)
                return Q_EHIP;
            scratch_addr[dev].store(p, std::memory_order_release);
        }
    }
    *out = p;
    return Q_OK;
}

}  // namespace

extern "C" {

size_t q_blocks_bytes(int fmt, int64_t N, int64_t K)
{
    if (!implemented(fmt) || check_tensor(fmt, N, K, QLINEAR_MAX_N) != Q_OK)
        return 0;
    return (size_t)ql::planes_of(fmt, N, K).total;
}

int isq_quantize(int fmt, const void *W_bf16, int64_t N, int64_t K, void *out_blocks, void *stream)
{
    if (!known(fmt))
        return Q_EINVAL;
    if (!implemented(fmt))
        return Q_ENOTSUP;
    if (!W_bf16 || !out_blocks)
        return Q_EINVAL;
    if (!aligned16(W_bf16) || !aligned16(out_blocks))
        return Q_EALIGN;
    const int st = check_tensor(fmt, N, K, QLINEAR_MAX_N);
    if (st != Q_OK)
        return st;
    return status_of(ql::launch_isq(fmt, static_cast<const uint16_t *>(W_bf16), N, K,
                                    static_cast<uint8_t *>(out_blocks), as_stream(stream)));
}

int q_act_quantize(const void *X_bf16, int64_t M, int64_t K, void *out_blocks, void *stream)
{
    if (!X_bf16 || !out_blocks)
        return Q_EINVAL;
    if (!aligned16(X_bf16) || !aligned16(out_blocks))
        return Q_EALIGN;
    const int st = check_tensor(QFMT_Q8_0, M, K, QLINEAR_MAX_M);
    if (st != Q_OK)
        return st;
    return status_of(ql::launch_isq(ql::FMT_Q8_0, static_cast<const uint16_t *>(X_bf16), M, K,
                                    static_cast<uint8_t *>(out_blocks), as_stream(stream)));
}

size_t qmatmul_workspace_bytes(int fmt, int path, int64_t M, int64_t K)
{
    if (path == QPATH_MFMA_I8 && fmt == QFMT_Q8_0 && K % 256 == 0 && check_tensor(QFMT_Q8_0, M, K, QLINEAR_MAX_M) == Q_OK)
        return (size_t)ql::planes_of(ql::FMT_Q8_0, M, K).total;
    if (path == QPATH_MFMA_FP8 && fmt == QFMT_FP8 && check_tensor(QFMT_FP8, M, K, QLINEAR_MAX_M) == Q_OK)
        return (size_t)ql::planes_of(ql::FMT_FP8, M, K).total;
    return 0;
}

int qmatmul_ex(int fmt, const void *blocks, const void *X_bf16, float *Y_fp32, int64_t M, int64_t N,
               int64_t K, int path, void *workspace, size_t workspace_bytes, void *stream)
{
    int st = matmul_args(fmt, blocks, X_bf16, Y_fp32, M, N, K);
    if (st != Q_OK)
        return st;
    const auto *B = static_cast<const uint8_t *>(blocks);
    const auto *X = static_cast<const uint16_t *>(X_bf16);
    const hipStream_t s = as_stream(stream);
    switch (path) {
    case QPATH_AUTO:
        // measured crossovers on MI355X: the fused GEMV wins for one or two
        // tokens, and for three or four where its one-shot kernel takes the
        // shape (Q6K 14336 x 4096, 3 tokens: 13.2 vs 21.7 us on the MFMA
        // stream); for the generic formats, whose MFMA kernel streams the
        // weights less well, up to four (Q5K 14336 x 4096, 3 tokens: 33.6 vs
        // 54.3 us); beyond, the MFMA weight stream
        // (and for five or six Q4K tokens on weights of at most 2^25
        // elements where the one-shot kernel takes them: 4096 x 4096 at
        // five tokens 6.5 vs 7.2 us, 6144 x 4096 8.6 vs 9.3 us; from
        // 14336 x 4096 or eight tokens the MFMA stream is faster)
        if (M <= 2 || (M <= 4 && ((ql::generic_fmt(fmt) && fmt != QFMT_FP8) || ql::gemv_one_shot_fits(fmt, (int)M, K))) ||
            (fmt == QFMT_Q4K && M <= 6 && N * K <= ((int64_t)1 << 25) && ql::gemv_one_shot_fits(fmt, (int)M, K))) {
            st = gemv(fmt, B, X, Y_fp32, M, N, K, s);
            if (st != Q_ENOTSUP)
                return st;
        }
        return status_of(ql::launch_gemm_bf16(fmt, B, X, Y_fp32, M, N, K, s));
    case QPATH_GEMV:
        if (M > 8)
            return Q_ESHAPE;
        return gemv(fmt, B, X, Y_fp32, M, N, K, s);
    case QPATH_MFMA_BF16:
        return status_of(ql::launch_gemm_bf16(fmt, B, X, Y_fp32, M, N, K, s));
    case QPATH_MFMA_I8: {
        if (fmt != QFMT_Q8_0)
            return Q_ENOTSUP;
        if (K % 256 != 0)
            return Q_ESHAPE;  // the int8 kernels take the scales of two blocks per dword
        if (!workspace)
            return Q_EINVAL;
        if (!aligned16(workspace))
            return Q_EALIGN;
        if (workspace_bytes < qmatmul_workspace_bytes(fmt, path, M, K))
            return Q_EINVAL;
        auto *ws = static_cast<uint8_t *>(workspace);
        st = status_of(ql::launch_isq(ql::FMT_Q8_0, X, M, K, ws, s));
        if (st != Q_OK)
            return st;
        return status_of(ql::launch_gemm_i8(B, ws, Y_fp32, M, N, K, s));
    }
    case QPATH_MFMA_FP8: {
        if (fmt != QFMT_FP8)
            return Q_ENOTSUP;
        if (!workspace)
            return Q_EINVAL;
        if (!aligned16(workspace))
            return Q_EALIGN;
        if (workspace_bytes < qmatmul_workspace_bytes(fmt, path, M, K))
            return Q_EINVAL;
        auto *ws = static_cast<uint8_t *>(workspace);
        st = status_of(ql::launch_isq(ql::FMT_FP8, X, M, K, ws, s));
        if (st != Q_OK)
            return st;
        return status_of(ql::launch_gemm_fp8(B, ws, Y_fp32, M, N, K, s));
    }
    default:
        return Q_EINVAL;
    }
}

int qmatmul(int fmt, const void *blocks, const void *X_bf16, float *Y_fp32, int64_t M, int64_t N, int64_t K,
            void *stream)
{
    return qmatmul_ex(fmt, blocks, X_bf16, Y_fp32, M, N, K, QPATH_AUTO, nullptr, 0, stream);
}

int qmatmul_static(int fmt, const void *blocks, const void *X_bf16, float *Y_fp32, int64_t M, int64_t N, int64_t K,
                   int path, void *stream)
{
    const int st = matmul_args(fmt, blocks, X_bf16, Y_fp32, M, N, K);
    if (st != Q_OK)
        return st;
    const size_t need = qmatmul_workspace_bytes(fmt, path, M, K);
    if (need == 0)  // no workspace on this path (or invalid arguments, which qmatmul_ex reports)
        return qmatmul_ex(fmt, blocks, X_bf16, Y_fp32, M, N, K, path, nullptr, 0, stream);
    if (need > QLINEAR_STATIC_SCRATCH_BYTES)
        return Q_ESCRATCH;
    void *ws = nullptr;
    const int sst = scratch_of_current_device(&ws);
    if (sst != Q_OK)
        return sst;
    return qmatmul_ex(fmt, blocks, X_bf16, Y_fp32, M, N, K, path, ws, need, stream);
}

size_t qmatmul_glu_workspace_bytes(int fmt, int64_t M, int64_t F, int64_t K)
{
    // every valid shape (check_tensor: K % 256, Q8_0 K % 32) that the fused
    // kernel does not take needs G in the workspace
    if (!implemented(fmt) || M < 1 || M > QLINEAR_MAX_M || check_tensor(fmt, F, K, QLINEAR_MAX_N) != Q_OK ||
        M * F > kMaxElems)
        return 0;
    return ql::glu_fused_fits(fmt, (int)M, K) ? 0 : (size_t)(4 * M * F);
}

int qmatmul_glu(int fmt, const void *gate_blocks, const void *up_blocks, const void *X_bf16, float *H_fp32,
                int64_t M, int64_t F, int64_t K, int act, void *workspace, size_t workspace_bytes, void *stream)
{
    int st = matmul_args(fmt, gate_blocks, X_bf16, H_fp32, M, F, K);
    if (st != Q_OK)
        return st;
    if (!up_blocks)
        return Q_EINVAL;
    if (!aligned16(up_blocks))
        return Q_EALIGN;
    if (act < QACT_SILU || act > QACT_SIGMOID)
        return Q_EINVAL;
    const auto *Bg = static_cast<const uint8_t *>(gate_blocks);
    const auto *Bu = static_cast<const uint8_t *>(up_blocks);
    const auto *X = static_cast<const uint16_t *>(X_bf16);
    const hipStream_t s = as_stream(stream);
    if (ql::glu_fused_fits(fmt, (int)M, K))
        return status_of(ql::launch_glu_fused(fmt, Bg, Bu, X, H_fp32, (int)M, F, K, act, s));
    // two matmuls and the elementwise product: G in the workspace, U in H
    if (!workspace)
        return Q_EINVAL;
    if (!aligned16(workspace))
        return Q_EALIGN;
    if (workspace_bytes < qmatmul_glu_workspace_bytes(fmt, M, F, K))
        return Q_EINVAL;
    float *G = static_cast<float *>(workspace);
    st = qmatmul(fmt, gate_blocks, X_bf16, G, M, F, K, stream);
    if (st != Q_OK)
        return st;
    st = qmatmul(fmt, up_blocks, X_bf16, H_fp32, M, F, K, stream);
    if (st != Q_OK)
        return st;
    return status_of(ql::launch_glu_apply(G, H_fp32, M * F, act, s));
}

int q_moe_route(const float *logits, int64_t T, int64_t E, int top_k, int score, const float *bias, int renorm,
                float scale, int32_t *ids, float *weights, void *stream)
{
    if (!logits || !ids || !weights)
        return Q_EINVAL;
    if (score != QSCORE_SOFTMAX && score != QSCORE_SIGMOID)
        return Q_EINVAL;
    if (!aligned4(logits) || !aligned4(ids) || !aligned4(weights) || !aligned4(bias))
        return Q_EALIGN;
    if (T < 0 || T > QLINEAR_MAX_M || E < 1 || E > QLINEAR_MAX_EXPERTS || top_k < 1 || top_k > QLINEAR_MAX_TOP_K ||
        top_k > E)
        return Q_ESHAPE;
    if (bias && score != QSCORE_SIGMOID)
        return Q_ENOTSUP;
    if (T == 0)
        return Q_OK;
    return status_of(ql::launch_moe_route(logits, (int)T, (int)E, top_k, score, bias, renorm, scale, ids, weights,
                                          as_stream(stream)));
}

size_t qmatmul_moe_workspace_bytes(int fmt_gate_up, int fmt_down, int64_t T, int64_t E, int top_k, int64_t F, int64_t K)
{
    if (moe_shape(fmt_gate_up, fmt_down, T, E, top_k, F, K) != Q_OK || T == 0)
        return 0;
    return (size_t)ql::moe_workspace((int)T, (int)E, top_k, F, K);
}

int qmatmul_moe(int fmt_gate_up, const void *gate_blocks, const void *up_blocks, int fmt_down, const void *down_blocks,
                const void *X_bf16, const int32_t *ids, const float *weights, float *Y_fp32, int64_t T, int64_t E,
                int top_k, int64_t F, int64_t K, int act, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!known(fmt_gate_up) || !known(fmt_down))
        return Q_EINVAL;
    if (!implemented(fmt_gate_up) || !implemented(fmt_down))
        return Q_ENOTSUP;
    if (!gate_blocks || !up_blocks || !down_blocks || !X_bf16 || !ids || !weights || !Y_fp32)
        return Q_EINVAL;
    if (act < QACT_SILU || act > QACT_SIGMOID)
        return Q_EINVAL;
    if (!aligned16(gate_blocks) || !aligned16(up_blocks) || !aligned16(down_blocks) || !aligned16(X_bf16) ||
        !aligned16(Y_fp32) || !aligned4(ids) || !aligned4(weights))
        return Q_EALIGN;
    const int st = moe_shape(fmt_gate_up, fmt_down, T, E, top_k, F, K);
    if (st != Q_OK)
        return st;
    if (T == 0)
        return Q_OK;
    if (!workspace)
        return Q_EINVAL;
    if (!aligned16(workspace))
        return Q_EALIGN;
    if (workspace_bytes < qmatmul_moe_workspace_bytes(fmt_gate_up, fmt_down, T, E, top_k, F, K))
        return Q_EINVAL;
    ql::MoeArgs a;
    a.fmt_gu = fmt_gate_up, a.fmt_d = fmt_down, a.act = act;
    a.T = (int)T, a.E = (int)E, a.k = top_k, a.F = F, a.K = K;
    a.gate = static_cast<const uint8_t *>(gate_blocks);
    a.up = static_cast<const uint8_t *>(up_blocks);
    a.down = static_cast<const uint8_t *>(down_blocks);
    a.X = static_cast<const uint16_t *>(X_bf16);
    a.ids = ids, a.weights = weights, a.Y = Y_fp32;
    a.ws = static_cast<uint8_t *>(workspace);
    return status_of(ql::launch_moe(a, as_stream(stream)));
}

size_t q_logprobs_workspace_bytes(int64_t M, int64_t V, int top_n)
{
    if (M < 1 || M > QLINEAR_MAX_M || V < 1 || V > QLINEAR_MAX_N || top_n < 0 || top_n > QLINEAR_MAX_TOP_N)
        return 0;
    return (size_t)ql::logprobs_workspace(M, V, top_n);
}

int q_logprobs(const float *logits, int64_t M, int64_t V, int64_t ld, const int32_t *targets, int top_n, float *logprob,
               int32_t *rank, float *entropy, int32_t *top_ids, float *top_logprobs, void *workspace,
               size_t workspace_bytes, void *stream)
{
    int st = logprob_args(targets, top_n, logprob, rank, entropy, top_ids, top_logprobs);
    if (st != Q_OK)
        return st;
    if (!logits)
        return Q_EINVAL;
    if (!aligned4(logits))
        return Q_EALIGN;
    if (M < 0 || M > QLINEAR_MAX_M || V < 1 || V > QLINEAR_MAX_N || ld < V || ld > kMaxElems || M * ld > kMaxElems)
        return Q_ESHAPE;
    if (M == 0)
        return Q_OK;
    const size_t need = (size_t)ql::logprobs_need(M, V, top_n);
    if (need) {
        if (!workspace)
            return Q_EINVAL;
        if (!aligned16(workspace))
            return Q_EALIGN;
        if (workspace_bytes < need)
            return Q_EINVAL;
    }
    ql::LogprobArgs a;
    a.logits = logits, a.M = M, a.V = V, a.ld = ld, a.targets = targets, a.top = top_n;
    a.logprob = logprob, a.rank = rank, a.entropy = entropy, a.top_ids = top_ids, a.top_logprobs = top_logprobs;
    a.ws = static_cast<uint8_t *>(workspace);
    return status_of(ql::launch_logprobs(a, as_stream(stream)));
}

size_t qmatmul_logprobs_workspace_bytes(int fmt, int64_t M, int64_t N, int64_t K, int top_n)
{
    if (!implemented(fmt) || M < 1 || M > QLINEAR_MAX_M || check_tensor(fmt, N, K, QLINEAR_MAX_N) != Q_OK ||
        M * K > kMaxElems || top_n < 0 || top_n > QLINEAR_MAX_TOP_N)
        return 0;
    const int64_t rows = head_rows(M, N);
    return head_logits_bytes(rows, N) + ql::up16(ql::logprobs_workspace(rows, N, top_n));
}

int qmatmul_logprobs(int fmt, const void *blocks, const void *X_bf16, int64_t M, int64_t N, int64_t K,
                     const int32_t *targets, int top_n, float *logprob, int32_t *rank, float *entropy, int32_t *top_ids,
                     float *top_logprobs, void *workspace, size_t workspace_bytes, void *stream)
{
    int st = logprob_args(targets, top_n, logprob, rank, entropy, top_ids, top_logprobs);
    if (st != Q_OK)
        return st;
    if (M == 0)
        return !known(fmt) ? Q_EINVAL : !implemented(fmt) ? Q_ENOTSUP : !blocks || !X_bf16 ? Q_EINVAL : Q_OK;
    if (!workspace)
        return Q_EINVAL;
    st = matmul_args(fmt, blocks, X_bf16, static_cast<const float *>(workspace), M < 1 ? 1 : M, N, K);
    if (st != Q_OK)
        return st;
    if (M < 1)
        return Q_ESHAPE;
    const int64_t rows = head_rows(M, N);
    const size_t logits_bytes = head_logits_bytes(rows, N);
    if (workspace_bytes < logits_bytes + ql::up16(head_parts_need(M, rows, N, top_n)))
        return Q_EINVAL;
    float *logits = static_cast<float *>(workspace);
    uint8_t *parts = static_cast<uint8_t *>(workspace) + logits_bytes;
    const auto *X = static_cast<const uint16_t *>(X_bf16);
    for (int64_t m = 0; m < M; m += rows) {
        const int64_t n = M - m < rows ? M - m : rows;
        st = qmatmul(fmt, blocks, X + m * K, logits, n, N, K, stream);
        if (st != Q_OK)
            return st;
        st = q_logprobs(logits, n, N, N, targets ? targets + m : nullptr, top_n, logprob ? logprob + m : nullptr,
                        rank ? rank + m : nullptr, entropy ? entropy + m : nullptr,
                        top_n ? top_ids + m * top_n : nullptr, top_n ? top_logprobs + m * top_n : nullptr, parts,
                        workspace_bytes - logits_bytes, stream);
        if (st != Q_OK)
            return st;
    }
    return Q_OK;
}

size_t qmatmul_grad_workspace_bytes(int fmt, int64_t M, int64_t N, int64_t K)
{
    if (!implemented(fmt) || M < 1 || grad_shape(fmt, M, N, K) != Q_OK)
        return 0;
    return (size_t)ql::grad_workspace(fmt, M, N, K);
}

int qmatmul_grad(int fmt, const void *blocks, const void *dY, int dy_type, void *dX_bf16, int64_t M, int64_t N,
                 int64_t K, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!known(fmt))
        return Q_EINVAL;
    if (!implemented(fmt))
        return Q_ENOTSUP;
    if (!blocks || !dY || !dX_bf16 || (dy_type != QTYPE_F32 && dy_type != QTYPE_BF16))
        return Q_EINVAL;
    if (!aligned16(blocks) || !aligned16(dY) || !aligned16(dX_bf16))
        return Q_EALIGN;
    int st = grad_shape(fmt, M, N, K);
    if (st != Q_OK || M == 0)
        return st;
    st = workspace_args(workspace, workspace_bytes, qmatmul_grad_workspace_bytes(fmt, M, N, K));
    if (st != Q_OK)
        return st;
    ql::GradArgs a;
    a.fmt = fmt, a.W = static_cast<const uint8_t *>(blocks), a.dY = dY, a.dy_bf16 = dy_type == QTYPE_BF16;
    a.dX = static_cast<uint16_t *>(dX_bf16), a.M = M, a.N = N, a.K = K, a.ws = static_cast<uint8_t *>(workspace);
    return status_of(ql::launch_grad(a, as_stream(stream)));
}

size_t qmatmul_glu_grad_workspace_bytes(int fmt, int64_t M, int64_t F, int64_t K)
{
    if (!implemented(fmt) || M < 1 || grad_shape(fmt, M, F, K) != Q_OK)
        return 0;
    return (size_t)ql::glu_grad_workspace(fmt, M, F, K);
}

int qmatmul_glu_grad(int fmt, const void *gate_blocks, const void *up_blocks, const void *X_bf16, const void *dH,
                     int dh_type, void *dX_bf16, void *dG_bf16, void *dU_bf16, int64_t M, int64_t F, int64_t K, int act,
                     void *workspace, size_t workspace_bytes, void *stream)
{
    if (!known(fmt))
        return Q_EINVAL;
    if (!implemented(fmt))
        return Q_ENOTSUP;
    if (!gate_blocks || !up_blocks || !X_bf16 || !dH || !dX_bf16 || (dh_type != QTYPE_F32 && dh_type != QTYPE_BF16) ||
        act < QACT_SILU || act > QACT_SIGMOID)
        return Q_EINVAL;
    if (!aligned16(gate_blocks) || !aligned16(up_blocks) || !aligned16(X_bf16) || !aligned16(dH) || !aligned16(dX_bf16) ||
        !aligned16(dG_bf16) || !aligned16(dU_bf16))
        return Q_EALIGN;
    int st = grad_shape(fmt, M, F, K);
    if (st != Q_OK || M == 0)
        return st;
    st = workspace_args(workspace, workspace_bytes, qmatmul_glu_grad_workspace_bytes(fmt, M, F, K));
    if (st != Q_OK)
        return st;
    ql::GluGradArgs a;
    a.fmt = fmt, a.act = act;
    a.gate = static_cast<const uint8_t *>(gate_blocks), a.up = static_cast<const uint8_t *>(up_blocks);
    a.X = static_cast<const uint16_t *>(X_bf16), a.dH = dH, a.dh_bf16 = dh_type == QTYPE_BF16;
    a.dX = static_cast<uint16_t *>(dX_bf16), a.dG = static_cast<uint16_t *>(dG_bf16), a.dU = static_cast<uint16_t *>(dU_bf16);
    a.M = M, a.F = F, a.K = K, a.ws = static_cast<uint8_t *>(workspace);
    return status_of(ql::launch_glu_grad(a, as_stream(stream)));
}

size_t qmatmul_xent_workspace_bytes(int fmt, int64_t M, int64_t N, int64_t K, int grad)
{
    if (!implemented(fmt) || M < 1 || grad_shape(fmt, M, N, K) != Q_OK)
        return 0;
    return (size_t)ql::xent_workspace(fmt, M, N, K, grad != 0);
}

int qmatmul_xent(int fmt, const void *blocks, const void *X_bf16, int64_t M, int64_t N, int64_t K,
                 const int32_t *targets, const float *weights, float *loss, float *lse, void *dX_bf16, void *workspace,
                 size_t workspace_bytes, void *stream)
{
    if (!known(fmt))
        return Q_EINVAL;
    if (!implemented(fmt))
        return Q_ENOTSUP;
    if (!blocks || !X_bf16 || !targets || !loss)
        return Q_EINVAL;
    if (!aligned16(blocks) || !aligned16(X_bf16) || !aligned16(dX_bf16) || !aligned4(targets) || !aligned4(weights) ||
        !aligned4(loss) || !aligned4(lse))
        return Q_EALIGN;
    int st = grad_shape(fmt, M, N, K);
    if (st != Q_OK || M == 0)
        return st;
    st = workspace_args(workspace, workspace_bytes, qmatmul_xent_workspace_bytes(fmt, M, N, K, dX_bf16 != nullptr));
    if (st != Q_OK)
        return st;
    ql::XentArgs a;
    a.fmt = fmt, a.W = static_cast<const uint8_t *>(blocks), a.X = static_cast<const uint16_t *>(X_bf16);
    a.targets = targets, a.weights = weights, a.loss = loss, a.lse = lse, a.dX = static_cast<uint16_t *>(dX_bf16);
    a.M = M, a.N = N, a.K = K, a.ws = static_cast<uint8_t *>(workspace);
    return status_of(ql::launch_xent(a, as_stream(stream)));
}

int q_dequantize(int fmt, const void *blocks, int64_t N, int64_t K, float *W_fp32, void *stream)
{
    if (!known(fmt))
        return Q_EINVAL;
    if (!implemented(fmt))
        return Q_ENOTSUP;
    if (!blocks || !W_fp32)
        return Q_EINVAL;
    if (!aligned16(blocks) || !aligned16(W_fp32))
        return Q_EALIGN;
    const int st = check_tensor(fmt, N, K, QLINEAR_MAX_N);
    if (st != Q_OK)
        return st;
    return status_of(ql::launch_dequant(fmt, static_cast<const uint8_t *>(blocks), N, K, W_fp32,
                                        as_stream(stream)));
}

int q_embed(int fmt, const void *blocks, int64_t N, int64_t K, const int32_t *ids, int64_t n_ids, float *out_fp32,
            void *stream)
{
    if (!known(fmt))
        return Q_EINVAL;
    if (!implemented(fmt))
        return Q_ENOTSUP;
    if (!blocks || !ids || !out_fp32)
        return Q_EINVAL;
    if (!aligned16(blocks) || !aligned16(out_fp32) || (reinterpret_cast<uintptr_t>(ids) & 3u) != 0)
        return Q_EALIGN;
    const int st = check_tensor(fmt, N, K, QLINEAR_MAX_N);
    if (st != Q_OK)
        return st;
    if (n_ids < 0 || n_ids > QLINEAR_MAX_EMBED_IDS || n_ids * K > kMaxElems)
        return Q_ESHAPE;
    if (n_ids == 0)
        return Q_OK;
    return status_of(ql::launch_embed(fmt, static_cast<const uint8_t *>(blocks), N, K, ids, n_ids, out_fp32,
                                      as_stream(stream)));
}

int q_probe_read(const void *buf, int64_t bytes, float *out, void *stream)
{
    if (!buf || !out)
        return Q_EINVAL;
    if (!aligned16(buf))
        return Q_EALIGN;
    if (bytes < 16 || bytes % 16 != 0 || bytes > kMaxElems)
        return Q_ESHAPE;
    return status_of(ql::launch_read_probe(buf, bytes, out, as_stream(stream)));
}

int q_probe_mfma(float *out, int64_t iters, void *stream)
{
    if (!out)
        return Q_EINVAL;
    if (iters < 0 || iters > (int64_t(1) << 24))
        return Q_ESHAPE;
    if (iters == 0)
        return Q_OK;
    return status_of(ql::launch_mfma_probe(out, iters, as_stream(stream)));
}

int64_t q_probe_mfma_flops(int64_t iters) { return iters < 0 ? 0 : ql::mfma_probe_flops(iters); }

int q_probe_mix(float *out, int64_t iters, int mode, int waves_per_simd, void *stream)
{
    if (!out)
        return Q_EINVAL;
    if (iters < 0 || iters > (int64_t(1) << 24) || mode < 0 || mode > 2 || waves_per_simd < 1 || waves_per_simd > 8)
        return Q_ESHAPE;
    if (iters == 0)
        return Q_OK;
    return status_of(ql::launch_mix_probe(out, iters, mode, waves_per_simd, as_stream(stream)));
}

int64_t q_probe_mix_valu(int64_t iters, int waves_per_simd)
{
    return iters < 0 || waves_per_simd < 1 || waves_per_simd > 8 ? 0 : ql::mix_probe_valu_insts(iters, waves_per_simd);
}

int isq_resolve_level(int level, int *out_fmt)
{
    if (!out_fmt)
        return Q_EINVAL;
    int f;
    switch (level) {
    case 2: f = QFMT_Q2K; break;
    case 3: f = QFMT_Q3K; break;
    case 4: f = QFMT_Q4K; break;
    case 5: f = QFMT_Q5K; break;
    case 6: f = QFMT_Q6K; break;
    case 8: f = QFMT_Q8_0; break;
    default: return Q_EINVAL;
    }
    *out_fmt = f;
    return Q_OK;
}

int isq_sensitive_fmt(int model_default, int *out_fmt)
{
    if (!out_fmt)
        return Q_EINVAL;
    switch (model_default) {
    case QFMT_Q2K:
    case QFMT_Q3K:
    case QFMT_Q4K:
    case QFMT_Q4_0:
    case QFMT_Q4_1:
        *out_fmt = QFMT_Q6K;
        return Q_OK;
    case QFMT_Q5K:
    case QFMT_Q6K:
    case QFMT_Q8K:
    case QFMT_Q5_0:
    case QFMT_Q5_1:
    case QFMT_Q8_0:
    case QFMT_Q8_1:
        *out_fmt = QFMT_Q8_0;
        return Q_OK;
    default:
        return Q_EINVAL;
    }
}

int isq_tensor_fmt(int level, int is_embedding_or_head, int explicit_fmt, int *out_fmt)
{
    if (!out_fmt)
        return Q_EINVAL;
    if (explicit_fmt >= 0) {
        if (!known(explicit_fmt))
            return Q_EINVAL;
        *out_fmt = explicit_fmt;
        return Q_OK;
    }
    int f;
    int st = isq_resolve_level(level, &f);
    if (st != Q_OK)
        return st;
    if (is_embedding_or_head) {
        st = isq_sensitive_fmt(f, &f);
        if (st != Q_OK)
            return st;
    }
    *out_fmt = f;
    return Q_OK;
}

int q_fmt_supported(int fmt) { return implemented(fmt) ? 1 : 0; }

const char *q_fmt_name(int fmt)
{
    static const char *names[] = {"q8_0", "q4k", "q6k", "q2k", "q3k", "q5k", "q8k",
                                  "q4_0", "q4_1", "q5_0", "q5_1", "q8_1", "fp8"};
    return known(fmt) ? names[fmt] : nullptr;
}

const char *q_strerror(int status)
{
    switch (status) {
    case Q_OK: return "ok";
    case Q_EINVAL: return "invalid argument (null pointer, unknown format or path, bad workspace)";
    case Q_ESHAPE: return "shape out of range (M, N, K limits; K a multiple of 256, or of 32 for Q8_0)";
    case Q_EALIGN: return "pointer not aligned (16 bytes; 4 for ids, logits and per-row results)";
    case Q_ENOTSUP: return "format or path not implemented for these arguments";
    case Q_EHIP: return "HIP runtime error at launch";
    case Q_ESCRATCH: return "activation blocks larger than the library's fixed scratch buffer (QLINEAR_STATIC_SCRATCH_BYTES)";
    default: return "unknown status";
    }
}

}  // extern "C"
