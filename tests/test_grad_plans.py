"""The gradients and the cross entropy where a call goes through in parts:
products whose first columns stand whole in front of split ones, rows in chunks
with a last one of few rows, rows too long to be held in registers between two
passes, the most rows and the longest sides that the calls accept."""
import numpy as np
import pytest
import torch

import ggml_block_quant_amd as ql
import synth
from grad_util import FMTS, back, rounded, within
from gpu_util import to_dev_bf16
from test_parity_grad import act_and_slope, check_glu, check_grad, gradients
from test_parity_xent import case, check, want

pytestmark = pytest.mark.gpu


def guarded(size, M, *dims):
    """A workspace of exactly the stated size with a guard behind it."""
    n = size(*dims[:1], M, *dims[1:])
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
    return ws, ws[:n], ws[n:]


# ---------------------------------------------------------------------------
# whole columns of tiles in front of split ones
# ---------------------------------------------------------------------------

# M, F, K: the first column of gate and up that is split, splits, rows of a tile
@pytest.mark.parametrize("fmt,M,F,K", (("q4k", 70, 40000, 1024),   # 32768, 4, 128
                                       ("q8_0", 515, 14337, 1024),  # 10880, 2, 192
                                       ("fp8", 300, 20000, 512)))   # 16384, 2, 192
@pytest.mark.parametrize("dtype", (torch.float32, torch.bfloat16))
def test_gated_pair_partly_split(fmt, M, F, K, dtype):
    check_glu(fmt, M, F, K, "silu", dtype, empty=(M - 1,))


def test_gated_pair_partly_split_stays_in_its_workspace():
    fmt, M, F, K = "q6k", 70, 40000, 1024
    bg, bu = (ql.isq(fmt, to_dev_bf16(synth.weights_bf16(86000 + i, F, K))) for i in range(2))
    X, dH = to_dev_bf16(synth.activations_bf16(86002, M, K)), gradients(1, M, F)
    ws, inside, guard = guarded(ql.glu_grad_workspace_bytes, M, fmt, F, K)
    a = ql.qmatmul_glu_grad(fmt, bg, bu, X, dH, parts=True, workspace=inside)
    b = ql.qmatmul_glu_grad(fmt, bg, bu, X, dH, parts=True)
    assert all(torch.equal(u, v) for u, v in zip(a, b)) and (guard == 255).all()


# M, N, K: the first column of the logits that is split, splits, rows of a tile
@pytest.mark.parametrize("fmt,M,N,K,start", (("q8_0", 600, 32001, 1024, 21760),  # 2, 256
                                             ("q4k", 130, 70001, 2048, 65536),   # 8, 192
                                             ("fp8", 600, 32001, 1024, 21760)))
def test_logits_partly_split(fmt, M, N, K, start):
    X, W, b, t = case(fmt, M, N, K)
    # given tokens on both sides of the first split column and at the ends
    t[:8] = torch.tensor([0, N - 1, start - 1, start, start + 1, start - 64, start + 63, N // 2], device="cuda")
    ws, inside, guard = guarded(ql.xent_workspace_bytes, M, fmt, N, K)
    got = ql.qmatmul_xent(fmt, b, X, N, t, workspace=inside)
    check(fmt, X, W, b, t, got=got, label=f"{fmt} {M}x{N}x{K}")
    assert (guard == 255).all()
    alone = ql.qmatmul_xent(fmt, b, X, N, t, grad=False)
    assert torch.equal(alone.loss, got.loss) and torch.equal(alone.lse, got.lse)


# ---------------------------------------------------------------------------
# chunks of rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M,dtype", ((300, torch.float32), (300, torch.bfloat16), (257, torch.float32), (257, torch.bfloat16),
                                     (259, torch.bfloat16)))
def test_gated_pair_in_chunks_of_rows(M, dtype):
    """2^26 values of G at once: 256 rows of 262144.  The rows behind them are
    those of a call of their own, bit for bit (of one row too)."""
    fmt, F, K, R = "q4_0", 262144, 256, 256
    g = torch.Generator("cuda").manual_seed(M)
    bg, bu = (ql.isq(fmt, synth.device_normal_bf16(86100 + i, (F, K), synth.W_SIGMA)) for i in range(2))
    X = torch.randn((M, K), device="cuda", generator=g).bfloat16()
    dH = torch.randn((M, F), device="cuda", generator=g).to(dtype)
    assert ql.glu_grad_workspace_bytes(fmt, M, F, K) == ql.glu_grad_workspace_bytes(fmt, R, F, K)
    ws, inside, guard = guarded(ql.glu_grad_workspace_bytes, M, fmt, F, K)
    got = ql.qmatmul_glu_grad(fmt, bg, bu, X, dH, parts=True, workspace=inside)
    assert (guard == 255).all()
    for a, e in ((0, R), (R, M)):
        own = ql.qmatmul_glu_grad(fmt, bg, bu, X[a:e].contiguous(), dH[a:e].contiguous(), parts=True)
        for u, v in zip(got, own):
            assert torch.equal(u[a:e], v)
    Wg, Wu = (ql.dequantize(fmt, b, F, K).double() for b in (bg, bu))
    for m in sorted({0, R - 1, R, M - 1}):
        x, d = X[m:m + 1].double(), dH[m:m + 1].double()
        gate, up = x @ Wg.t(), x @ Wu.t()
        a, da = act_and_slope("silu", gate)
        # G and U within 2^-11 + K 2^-23 of their magnitudes (2^-10.5); slopes of silu up to 1.1 and 0.5
        eg, eu = (2.0 ** -10.5 * (x.abs() @ w.abs().t()) for w in (Wg, Wu))
        tu = d.abs() * 1.1 * eg + 2.0 ** -19 * (d * a).abs()
        tg = d.abs() * (da.abs() * eu + (up.abs() + eu) * 0.5 * eg + 2.0 ** -18 * up.abs())
        within(got.dG[m:m + 1], d * up * da, rounded(d * up * da, tg), f"dG row {m}")
        within(got.dU[m:m + 1], d * a, rounded(d * a, tu), f"dU row {m}")
        y, tol = back(torch.cat([d * up * da, d * a], 1), torch.cat([Wg, Wu], 0), torch.cat([tg, tu], 1))
        within(got.dX[m:m + 1], y, rounded(y, tol), f"dX row {m}")


@pytest.mark.parametrize("M", (257, 258, 260, 300))
def test_cross_entropy_in_chunks_with_a_short_last_one(M):
    """256 rows of 262144 logits at once; weights and tokens that are not scored
    in every chunk, one row to 44 in the last."""
    N, K, R = 262144, 256, 256
    b = ql.isq("q4_0", synth.device_normal_bf16(86200, (N, K), synth.W_SIGMA))
    X = to_dev_bf16(synth.activations_bf16(86201, M, K))
    t = torch.arange(M, dtype=torch.int32, device="cuda") * 800
    wt = torch.linspace(0.5, 2.0, M, device="cuda")
    if M > R + 1:
        t[R], t[7] = -1, N
    ws, inside, guard = guarded(ql.xent_workspace_bytes, M, "q4_0", N, K)
    got = ql.qmatmul_xent("q4_0", b, X, N, t, weights=wt, workspace=inside)
    assert (guard == 255).all()
    for a, e in ((0, R), (R, M)):
        own = ql.qmatmul_xent("q4_0", b, X[a:e].contiguous(), N, t[a:e].clone(), weights=wt[a:e].clone())
        for u, v in zip(got, own):
            assert torch.equal(u[a:e], v)
    W = ql.dequantize("q4_0", b, N, K).double()
    for a, e in ((0, 9), (R - 2, M if M - R < 9 else R + 9)):
        check("q4_0", X[a:e], W, b, t[a:e], wt[a:e], got=ql.Xent(*(v[a:e] for v in got)), label=f"rows {a}")


def test_grad_in_chunks_with_a_last_row():
    """4096 rows of 32768 values at once, and one more."""
    M, N, K = 4097, 32768, 256
    b = ql.isq("q4_0", synth.device_normal_bf16(86300, (N, K), synth.W_SIGMA))
    dY = torch.randn((M, N), device="cuda", generator=torch.Generator("cuda").manual_seed(9)).bfloat16()
    ws, inside, guard = guarded(ql.grad_workspace_bytes, M, "q4_0", N, K)
    got = ql.qmatmul_grad("q4_0", b, dY, K, workspace=inside)
    assert (guard == 255).all()
    assert torch.equal(got[:4096], ql.qmatmul_grad("q4_0", b, dY[:4096], K))
    W = ql.dequantize("q4_0", b, N, K).double()
    for m in (0, 4095, 4096):
        y, tol = back(dY[m:m + 1].double(), W)
        within(got[m:m + 1], y, rounded(y, tol), f"row {m}")


# ---------------------------------------------------------------------------
# rows of more than 16384 values, which are read twice
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", (torch.float32, torch.bfloat16))
@pytest.mark.parametrize("N", (16384, 16385, 16392, 20001))
def test_grad_long_rows(N, dtype):
    for M in (2, 35):
        check_grad("q4k", M, N, 256, dtype, empty=(1,))


@pytest.mark.parametrize("dtype", (torch.float32, torch.bfloat16))
@pytest.mark.parametrize("fmt,F", (("q6k", 16384), ("q6k", 16385), ("q8_0", 16392), ("fp8", 20001)))
def test_gated_pair_long_rows(fmt, F, dtype):
    for M, parts in ((2, True), (35, True), (70, False)):
        check_glu(fmt, M, F, 256, "silu", dtype, parts=parts, empty=(M - 1,))


@pytest.mark.parametrize("M,F", ((1, 300), (3, 300), (3, 16385), (40, 301), (100, 16392)))
def test_gated_pair_with_one_of_the_parts(M, F):
    """dG or dU alone: the same bits, nothing else written."""
    K = 256
    bg, bu = (ql.isq("q4k", to_dev_bf16(synth.weights_bf16(86500 + i, F, K))) for i in range(2))
    X, dH = to_dev_bf16(synth.activations_bf16(86502, M, K)), gradients(2, M, F)
    both = ql.qmatmul_glu_grad("q4k", bg, bu, X, dH, parts=True)
    for g, u in ((True, False), (False, True)):
        bf = [torch.zeros((M, n), dtype=torch.bfloat16, device="cuda") for n in (K, F, F)]
        r = ql.qmatmul_glu_grad("q4k", bg, bu, X, dH, out=ql.GluGrad(bf[0], bf[1] if g else None, bf[2] if u else None))
        assert torch.equal(r.dX, both.dX)
        assert torch.equal(bf[1], both.dG if g else torch.zeros_like(bf[1]))
        assert torch.equal(bf[2], both.dU if u else torch.zeros_like(bf[2]))


def test_long_inputs():
    """X's own rows: K beyond what is held, panels of either width."""
    K = 17408
    check_glu("q4k", 20, 130, K, "silu")
    check_glu("q8_0", 70, 130, K - 32, "sigmoid")
    for M in (20, 70):
        X, W, b, t = case("q6k", M, 300, K)
        check("q6k", X, W, b, t, label=f"{M} rows of {K}")


# ---------------------------------------------------------------------------
# addresses that are whole multiples of 16 bytes and of no more
# ---------------------------------------------------------------------------

def barely(t):
    """A copy of t at an address of 16 bytes more than a multiple of 256."""
    n = t.numel() * t.element_size()
    hold = torch.zeros(n + 512, dtype=torch.uint8, device="cuda")
    at = (16 - hold.data_ptr()) % 256
    out = hold[at:at + n].view(t.dtype).view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 256 == 16
    return out


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", (1, 3, 20, 60, 100, 300))
def test_barely_aligned_buffers(fmt, M):
    """Every buffer 16 bytes off a multiple of 256: the same bits."""
    N, K = 333, 512
    b = ql.isq(fmt, to_dev_bf16(synth.weights_bf16(86400, N, K)))
    X, d = to_dev_bf16(synth.activations_bf16(86401, M, K)), gradients(3, M, N)
    t, wt = torch.arange(M, dtype=torch.int32, device="cuda"), torch.linspace(0.5, 2.0, M, device="cuda")

    def space(n):
        return barely(torch.zeros(n, dtype=torch.uint8, device="cuda"))

    bf, f32 = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda"), torch.zeros(M, device="cuda")
    fb = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    b2, X2, t2, w2 = barely(b), barely(X), barely(t), barely(wt)
    for dY in (d, d.bfloat16()):
        d2 = barely(dY)
        got = ql.qmatmul_grad(fmt, b2, d2, K, out=barely(bf), workspace=space(ql.grad_workspace_bytes(fmt, M, N, K)))
        assert torch.equal(got, ql.qmatmul_grad(fmt, b, dY, K))
        got = ql.qmatmul_glu_grad(fmt, b2, b2, X2, d2, out=ql.GluGrad(barely(bf), barely(fb), barely(fb)),
                                  workspace=space(ql.glu_grad_workspace_bytes(fmt, M, N, K)))
        for u, v in zip(got, ql.qmatmul_glu_grad(fmt, b, b, X, dY, parts=True)):
            assert torch.equal(u, v)
    got = ql.qmatmul_xent(fmt, b2, X2, N, t2, weights=w2, out=ql.Xent(barely(f32), barely(f32), barely(bf)),
                          workspace=space(ql.xent_workspace_bytes(fmt, M, N, K)))
    for u, v in zip(got, ql.qmatmul_xent(fmt, b, X, N, t, weights=wt)):
        assert torch.equal(u, v)


# ---------------------------------------------------------------------------
# the most rows, the longest sides
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M", (32768, 32769, 65536))
def test_most_rows(M):
    check_grad("q8_0", M, 40, 32)
    check_glu("q8_0", M, 33, 32, "silu")
    X, W, b, t = case("q8_0", M, 50, 32)
    t[M - 1], t[5] = -1, 50
    check("q8_0", X, W, b, t, label=f"{M} rows")


def whole_q8_0(seed, N, K):
    """Q8_0 blocks of whole numbers from -3 to 3 times 1 or 1/2 a block, and
    their values."""
    g = torch.Generator("cuda").manual_seed(seed)
    q = torch.randint(-3, 4, (N, K), device="cuda", generator=g, dtype=torch.int8)
    d = 2.0 ** -torch.randint(0, 2, (N * K // 32,), device="cuda", generator=g).float()
    blocks = torch.cat([q.view(torch.uint8).reshape(-1), d.half().view(torch.uint8)])
    assert blocks.numel() == ql.blocks_bytes("q8_0", N, K)
    return blocks, (q.reshape(-1, 32) * d[:, None]).reshape(N, K)


def sparse(seed, M, n, count):
    """[M][n] with `count` places a row of +-1, the first and the last among them."""
    g = torch.Generator("cuda").manual_seed(seed)
    v = torch.zeros((M, n), device="cuda")
    at = torch.randint(0, n, (M, count), device="cuda", generator=g)
    at[:, 0], at[:, -1] = 0, n - 1
    v.scatter_(1, at, torch.randint(0, 2, (M, count), device="cuda", generator=g).float() * 2 - 1)
    return v


@pytest.mark.parametrize("M", (1, 2, 33))
def test_most_weight_rows(M):
    """2^24 rows of weights: whole numbers whose sums fit 24 bits, so the results
    are the exact sums' roundings to bf16."""
    N, K = 1 << 24, 32
    b, W = whole_q8_0(87000, N, K)
    dY = sparse(87001, M, N, 500)
    got = ql.qmatmul_grad("q8_0", b, dY, K)
    at = torch.nonzero(dY.any(0))[:, 0]
    assert torch.equal(got, (dY[:, at].double() @ W[at].double()).float().bfloat16())
    # ReLU's pair: |u dH| and |g dH| at most 18, sums below 2 * 500 * 18 * 3 in quarters
    b2, W2 = whole_q8_0(87002, N, K)
    X = sparse(87003, M, K, 6)
    r = ql.qmatmul_glu_grad("q8_0", b, b2, X.bfloat16(), dY, act="relu", parts=True)
    g, u, d = X.double() @ W[at].double().t(), X.double() @ W2[at].double().t(), dY[:, at].double()
    dg, du = d * u * (g > 0), d * g.clamp(min=0)
    assert torch.equal(r.dG[:, at].double(), dg) and torch.equal(r.dU[:, at].double(), du)
    assert int(torch.count_nonzero(r.dG)) == int(torch.count_nonzero(dg))
    assert torch.equal(r.dX, (dg @ W[at].double() + du @ W2[at].double()).float().bfloat16())


@pytest.mark.parametrize("M", (1, 2, 33))
def test_largest_vocabulary(M):
    """2^24 entries of logits up to 96, but one a row of 4064 (and those of the
    other rows, at least 1016 below it): e^(z - top) is 0 or 1, so loss, lse and
    gradient are exact."""
    N, K = 1 << 24, 32
    b, W = whole_q8_0(87100, N, K)
    top = (torch.arange(M, device="cuda") * 7919 * 31 + N - 5) % N
    t = (top + torch.where(torch.arange(M, device="cuda") % 2 == 0, 1 + N // 3, 0)) % N
    # the sure entries: codes of 127 under a scale of 1, signs of their own
    # (X of +-1 gives them 127 * 32 where the signs are X's)
    x = torch.randint(0, 2, (M, K), device="cuda", generator=torch.Generator("cuda").manual_seed(4)).float() * 2 - 1
    q = b[:N * K].view(torch.int8).reshape(N, K)
    q[top] = (x * 127).to(torch.int8)
    b[N * K:].view(torch.float16).reshape(N, K // 32)[top] = 1.0
    W[top] = x * 127
    if M > 1:  # (two sure entries of a row: a sign apart in at least four places)
        assert (x.double() @ x.double().t() - K * torch.eye(M, device="cuda")).amax() <= K - 8
    r = ql.qmatmul_xent("q8_0", b, x.bfloat16(), N, t.to(torch.int32))
    z = torch.full((M,), 127.0 * K, device="cuda")
    zt = (x * W[t]).sum(1)
    assert torch.equal(r.lse, z) and torch.equal(r.loss, z - zt)
    assert torch.equal(r.dX, (W[top] - W[t]).bfloat16())


@pytest.mark.parametrize("M", (1, 3, 5, 40, 70))
def test_longest_weight_rows(M):
    """2^20 columns: whole numbers again, every sum exact."""
    N, K = 5, 1 << 20
    b, W = whole_q8_0(87200, N, K)
    dY = sparse(87201, M, N, 4)
    assert torch.equal(ql.qmatmul_grad("q8_0", b, dY, K), (dY.double() @ W.double()).float().bfloat16())
    b2, W2 = whole_q8_0(87202, N, K)
    X = sparse(87203, M, K, 40)
    r = ql.qmatmul_glu_grad("q8_0", b, b2, X.bfloat16(), dY, act="relu", parts=True)
    g, u = X.double() @ W.double().t(), X.double() @ W2.double().t()
    dg, du = dY.double() * u * (g > 0), dY.double() * g.clamp(min=0)
    assert torch.equal(r.dG.double(), dg) and torch.equal(r.dU.double(), du)
    assert torch.equal(r.dX, (dg @ W.double() + du @ W2.double()).float().bfloat16())
    t = torch.arange(M, dtype=torch.int32, device="cuda") % N
    x = ql.qmatmul_xent("q8_0", b, X.bfloat16(), N, t)
    loss, lse, d, _ = want(X.double(), W.double(), t)
    # the logits are exact; five terms of expf, logf, a difference: some 2^-20
    within(x.lse, lse, 2.0 ** -19 * (1 + lse.abs()), "lse")
    within(x.loss, loss, 2.0 ** -19 * (1 + loss.abs()) * torch.ones_like(loss), "loss")
    y, tol = back(d, W.double(), d.abs() * 2.0 ** -18)
    within(x.dX, y, rounded(y, tol), "dX")
