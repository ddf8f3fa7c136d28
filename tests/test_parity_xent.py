"""GPU parity of the cross entropy over a quantized head and its gradient
(qmatmul_xent), against the formula in 64 bits on the oracle's weights."""
import numpy as np
import pytest
import torch

import ggml_block_quant_amd as ql
import synth
from grad_util import FMTS, U, back, forward, rounded, weights, within
from gpu_util import to_dev_bf16

pytestmark = pytest.mark.gpu


def want(X, W, t, wt=None):
    """loss, lse, p - onehot in 64 bits, and which rows are scored."""
    M, N = X.shape[0], W.shape[0]
    z = X @ W.t()
    lse = torch.logsumexp(z, 1)
    ok = (t >= 0) & (t < N)
    i, tc = torch.arange(M, device=X.device), t.clamp(0, N - 1).long()
    zo = z.clone()
    zo[i, tc] = -float("inf")
    rest = torch.logsumexp(zo, 1)  # ln of the others' sum
    loss = torch.where(ok, torch.nn.functional.softplus(rest - z[i, tc]), torch.zeros_like(lse))
    d = torch.exp(z - lse[:, None])
    d[i, tc] = -torch.exp(rest - lse)
    d = d * ok[:, None]
    if wt is not None:
        d = d * wt.double()[:, None]
    return loss, lse, d, ok


def check(fmt, X, W, blocks, t, wt=None, got=None, label=""):
    N = W.shape[0]
    Xd = X.double()
    loss, lse, d, ok = want(Xd, W, t, wt)
    got = got or ql.qmatmul_xent(fmt, blocks, X, N, t, weights=wt)
    _, ez = forward(Xd, W, pair=True)
    e = ez.amax(1)
    # FP8: the row's scale is one more rounding of each logit, as is 2^e's undoing
    z = (Xd @ W.t()).abs().amax(1)
    e = e + 4 * U * z
    # lse: the largest exponent's error, expf and its sums (terms of a thread,
    # lanes, waves and runs), logf
    sums = (N / 256 + 64) * U
    # (x - max) rounds once more, by 2^-24 of up to 2 z
    el = e + 2 * U * z + sums + 2.0 ** -21
    within(got.lse, lse, el + 2 * U * lse.abs(), f"lse {label}")
    # loss = ln(1 + rest / own): relative where it is small
    tol = torch.minimum(2 * el + 4 * U * (lse.abs() + z), (torch.expm1(2 * el) + 2.0 ** -20) * loss + 2.0 ** -149)
    within(got.loss, loss, torch.where(ok, tol, torch.zeros_like(tol)) + 8 * U * loss, f"loss {label}")
    if got.dX is not None:
        f = torch.expm1(2 * el + 8 * U)[:, None]
        y, tol = back(d, W, d.abs() * f)
        within(got.dX, y, rounded(y, tol) + 2 * U * y.abs(), f"dX {label}")
        assert not got.dX[~ok].any()
    return got


def case(fmt, M, N, K, seed=81000, lean=12.0):
    w, W = weights(fmt, seed + N, N, K)
    g = torch.Generator("cuda").manual_seed(seed + M)
    t = torch.randint(0, N, (M,), device="cuda", generator=g)
    # from guesses to tokens that the model is sure of
    X = torch.randn((M, K), device="cuda", generator=g)
    row = W[t].float()
    X = X + lean * torch.rand((M, 1), device="cuda", generator=g) * row / row.square().sum(1, keepdim=True).clamp(min=1e-6)
    return X.bfloat16(), W, ql.isq(fmt, to_dev_bf16(w)), t.to(torch.int32)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", ((1, 1000, 512), (7, 255, 256), (33, 257, 256), (70, 300, 512), (130, 700, 256), (300, 129, 256)))
def test_formats_and_sizes(fmt, M, N, K):
    X, W, b, t = case(fmt, M, N, K)
    wt = torch.rand(M, device="cuda", generator=torch.Generator("cuda").manual_seed(M)) if M % 2 else None
    check(fmt, X, W, b, t, wt, label=f"{fmt} {M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", ((1, 1, 256), (5, 1, 256), (1, 2, 256), (40, 3, 512), (2, 63, 256), (3, 64, 256), (3, 65, 256),
                                   (1, 30000, 256), (3, 4097, 1024), (520, 2100, 256), (17, 40001, 256)))
def test_small_and_long_vocabularies(M, N, K):
    X, W, b, t = case("q4k", M, N, K)
    check("q4k", X, W, b, t, label=f"{M}x{N}x{K}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", ((2, 333, 4096), (3, 333, 4096), (4, 331, 4096), (3, 200, 5120), (4, 201, 5120), (3, 97, 8192),
                                   (4, 97, 8192), (5, 97, 4096), (20, 1000, 4096), (50, 501, 5120)))
def test_few_rows_of_wide_heads(fmt, M, N, K):
    """Either side of where the logits' product changes its form."""
    X, W, b, t = case(fmt, M, N, K)
    check(fmt, X, W, b, t, label=f"{fmt} {M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", ((3, 100, 32), (50, 301, 1056), (129, 77, 224)))
def test_rows_of_whole_blocks(M, N, K):
    X, W, b, t = case("q8_0", M, N, K)
    check("q8_0", X, W, b, t, label=f"{M}x{N}x{K}")


def test_one_entry_vocabulary_is_exact():
    X, W, b, _ = case("q6k", 4, 1, 256)
    r = ql.qmatmul_xent("q6k", b, X, 1, torch.tensor([0, 0, -1, 5], dtype=torch.int32, device="cuda"))
    assert not r.loss.any() and not r.dX.any()


def test_rows_not_scored():
    """Targets outside the vocabulary, all of them or some; extreme numbers."""
    M, N, K = 70, 500, 256
    X, W, b, t = case("q5_0", M, N, K)
    t[3], t[4], t[69], t[0] = -1, N, -2 ** 31, 2 ** 31 - 1
    r = check("q5_0", X, W, b, t, label="some")
    assert (r.loss[[0, 3, 4, 69]] == 0).all() and not r.dX[[0, 3, 4, 69]].any()
    t[:] = -100
    r = ql.qmatmul_xent("q5_0", b, X, N, t)
    assert not r.loss.any() and not r.dX.any() and torch.isfinite(r.lse).all()


def test_sure_tokens_keep_their_digits():
    """Margins up to 80: losses down to e^-80 and gradients as small, relative
    to themselves."""
    M, N, K = 64, 300, 512
    w, W = weights("q8_0", 82000, N, K)
    b = ql.isq("q8_0", to_dev_bf16(w))
    t = torch.arange(M, device="cuda") * 4
    row = W[t].float()
    X = (torch.linspace(1, 80, M, device="cuda")[:, None] * row / row.square().sum(1, keepdim=True)).bfloat16()
    t = t.to(torch.int32)
    r = check("q8_0", X, W, b, t, label="sure")
    assert float(r.loss[-1]) < 1e-20 and float(r.loss[-1]) > 0
    assert r.dX[-1].any()


def test_zero_inputs_give_uniform_probabilities():
    N, K = 1000, 256
    X, W, b, t = case("q4_1", 5, N, K)
    X = torch.zeros_like(X)
    r = check("q4_1", X, W, b, t, label="zeros")
    assert (r.loss - np.log(N)).abs().max() <= 2.0 ** -19


def test_weights_of_rows():
    """weights enter dX alone: 0 leaves zeros, signs and sizes count."""
    M, N, K = 40, 600, 256
    X, W, b, t = case("q6k", M, N, K)
    wt = torch.linspace(-2, 3, M, device="cuda")
    wt[7], wt[8], wt[9] = 0.0, 1e-30, 1e30
    r = check("q6k", X, W, b, t, wt, label="weights")
    one = ql.qmatmul_xent("q6k", b, X, N, t)
    assert torch.equal(r.loss, one.loss) and torch.equal(r.lse, one.lse) and not r.dX[7].any()


def test_loss_alone_and_given_results():
    M, N, K = 50, 800, 512
    X, W, b, t = case("q3k", M, N, K)
    full = ql.qmatmul_xent("q3k", b, X, N, t)
    alone = ql.qmatmul_xent("q3k", b, X, N, t, grad=False)
    assert alone.dX is None and torch.equal(alone.loss, full.loss) and torch.equal(alone.lse, full.lse)
    out = ql.Xent(torch.empty(M, device="cuda"), None, torch.empty((M, K), dtype=torch.bfloat16, device="cuda"))
    got = ql.qmatmul_xent("q3k", b, X, N, t, out=out)
    assert got is out and torch.equal(got.loss, full.loss) and torch.equal(got.dX, full.dX)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,rows", ((40, (2, 30)), (130, (2, 129)), (2, (1,)), (2, (0,)), (1, (0,))))
def test_rows_that_are_not_finite_stay_alone(fmt, M, rows):
    N, K = 300, 256
    X, W, b, t = case(fmt, M, N, K)
    clean = ql.qmatmul_xent(fmt, b, X, N, t)
    bad = X.clone()
    for i, m in enumerate(rows):
        bad[m, 5 * i] = float("inf") if i else float("nan")
    got = ql.qmatmul_xent(fmt, b, bad, N, t)
    keep = [m for m in range(M) if m not in rows]
    for a, c in zip(got, clean):
        assert torch.equal(a[keep], c[keep])
    rows = list(rows)
    assert not torch.isfinite(got.loss[rows]).any() and not torch.isfinite(got.lse[rows]).any()
    assert not torch.isfinite(got.dX[rows]).any()


def test_same_bits_and_surroundings():
    N, K = 1001, 256
    w, W = weights("q4k", 83000, N, K)
    b = ql.isq("q4k", to_dev_bf16(w))
    big = ql.xent_workspace_bytes("q4k", 500, N, K)
    ws = torch.full((big + 256,), 255, dtype=torch.uint8, device="cuda")
    for M in (1, 2, 3, 31, 33, 64, 65, 128, 129, 192, 193, 256, 257, 300, 384, 385, 500):
        X = to_dev_bf16(synth.activations_bf16(83100 + M, M, K))
        t = torch.arange(M, dtype=torch.int32, device="cuda")
        hold = [torch.full((M + 2,), 7.0, device="cuda"), torch.full((M + 2,), 7.0, device="cuda"),
                torch.full((M + 2, K), 7.0, dtype=torch.bfloat16, device="cuda")]
        a = ql.qmatmul_xent("q4k", b, X, N, t, out=ql.Xent(*(h[1:M + 1] for h in hold)),
                            workspace=ws[:big])
        n = ql.xent_workspace_bytes("q4k", M, N, K)
        own = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
        c = ql.qmatmul_xent("q4k", b, X, N, t, workspace=own[:n])
        for u, v in zip(a, c):
            assert torch.equal(u, v)
        assert (own[n:] == 255).all() and (ws[big:] == 255).all()
        for h in hold:
            assert (h[0] == 7).all() and (h[M + 1] == 7).all()


def test_in_chunks_of_rows():
    """More rows than their logits go through at once: 256 of 262144, the last
    chunk ragged."""
    M, N, K = 300, 262144, 256
    w = to_dev_bf16(synth.weights_bf16(84000, N, K))
    b = ql.isq("q4_0", w)
    X = to_dev_bf16(synth.activations_bf16(84001, M, K))
    t = torch.arange(M, dtype=torch.int32, device="cuda") * 800
    assert ql.xent_workspace_bytes("q4_0", M, N, K) == ql.xent_workspace_bytes("q4_0", 256, N, K)
    got = ql.qmatmul_xent("q4_0", b, X, N, t)
    W = ql.dequantize("q4_0", b, N, K).double()
    for a, e in ((0, 8), (250, 262), (296, 300)):
        check("q4_0", X[a:e], W, b, t[a:e], got=ql.Xent(got.loss[a:e], got.lse[a:e], got.dX[a:e]), label=f"rows {a}")


def test_against_the_head_s_log_probabilities():
    """loss is the log probability's opposite, as the scoring call gives it (its
    logits within 2^-16 of their magnitudes, these within 2^-22)."""
    M, N, K = 90, 3000, 512
    X, W, b, t = case("q6k", M, N, K)
    r = ql.qmatmul_xent("q6k", b, X, N, t)
    lp = ql.qmatmul_logprobs("q6k", b, X, N, t).logprob
    den = (X.double().abs() @ W.abs().t()).amax(1)
    assert ((r.loss + lp).abs().double() <= 2 * (2.0 ** -16 + (2 * K + 8) * U + 2.0 ** -21) * den + 2.0 ** -18).all()


def test_gradient_against_differences():
    """Central differences of the loss in 64 bits along random directions."""
    M, N, K, h = 6, 400, 256, 1e-5
    X, W, b, t = case("q5_1", M, N, K)
    dX = ql.qmatmul_xent("q5_1", b, X, N, t).dX.double()
    E = torch.randn((M, K), device="cuda", dtype=torch.float64, generator=torch.Generator("cuda").manual_seed(3))
    x = X.double()
    diff = (want(x + h * E, W, t)[0] - want(x - h * E, W, t)[0]) / (2 * h)
    _, _, d, _ = want(x, W, t)
    y, tol = back(d, W, d.abs() * 1e-4)
    # third derivatives: h^2 (max |E . w|)^3
    own = h ** 2 * (E @ W.t()).abs().amax(1) ** 3 + 1e-9
    assert ((dX * E).sum(1) - diff).abs().le((rounded(y, tol) * E.abs()).sum(1) + own).all()
