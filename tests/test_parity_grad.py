"""GPU parity of the gradients through frozen quantized weights: the input
gradient of a linear layer (qmatmul_grad) and the gated projection's backward
pass (qmatmul_glu_grad), against their formulas in 64 bits on the oracle's
weights, and against differences of the forward products."""
import numpy as np
import pytest
import torch

import ggml_block_quant_amd as ql
import oracle
import synth
from grad_util import E16, FMTS, U, back, forward, rounded, weights, within
from gpu_util import to_dev_bf16
from test_moe_precision import pack, whole

pytestmark = pytest.mark.gpu

ACTS = ("silu", "relu", "sigmoid")
TUNED = ("q8_0", "q4k", "q6k")


def gradients(seed, M, N, dtype=torch.float32, empty=()):
    """Rows of sizes from 1e-6 to 1, long tails, some rows empty."""
    g = torch.Generator("cuda").manual_seed(seed)
    d = torch.randn((M, N), device="cuda", generator=g)
    d = d * (0.1 + d.abs()) * 10.0 ** -(torch.arange(M, device="cuda") % 7)[:, None]
    for m in empty:
        d[m % M] = 0
    return d.to(dtype)


def check_grad(fmt, M, N, K, dtype=torch.float32, empty=()):
    w, W = weights(fmt, 71000 + N, N, K, outliers=True)
    dY = gradients(N + M, M, N, dtype, empty)
    got = ql.qmatmul_grad(fmt, ql.isq(fmt, to_dev_bf16(w)), dY, K)
    y, tol = back(dY.double(), W)
    assert got.shape == (M, K) and got.dtype == torch.bfloat16
    within(got, y, rounded(y, tol), f"grad {fmt} {M}x{N}x{K}")
    return got


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", ((1, 1, 256), (1, 300, 512), (3, 63, 256), (32, 64, 768), (33, 65, 256), (64, 200, 256),
                                   (65, 129, 512), (128, 127, 256), (129, 640, 256), (257, 100, 512)))
def test_grad_sizes(fmt, M, N, K):
    check_grad(fmt, M, N, K, torch.bfloat16 if M % 2 else torch.float32)


@pytest.mark.parametrize("M,N,K", ((1, 40, 32), (5, 70, 96), (70, 33, 288), (130, 200, 1056), (300, 64, 224)))
def test_grad_rows_of_whole_blocks(M, N, K):
    """Q8_0 rows that are no multiple of 256."""
    check_grad("q8_0", M, N, K)


@pytest.mark.parametrize("fmt", TUNED)
@pytest.mark.parametrize("dtype", (torch.float32, torch.bfloat16))
def test_grad_wide_and_long(fmt, dtype):
    """Column tiles over several XCDs, splits of the reduction, rows of zeros."""
    check_grad(fmt, 2, 3000, 4096, dtype, empty=(1,))
    check_grad(fmt, 40, 2500, 2048, dtype, empty=(0, 17, 39))
    check_grad(fmt, 515, 1100, 1280, dtype, empty=(100, 514))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", ((1, 70, 512), (31, 200, 256), (60, 513, 768), (100, 90, 512), (260, 300, 1024)))
def test_grad_whole_numbers_are_exact(fmt, M, N, K):
    """Small whole numbers times powers of two, whose sums fit 24 bits: the
    results are the exact sums' roundings to bf16, bit for bit."""
    f, W, mag = whole(fmt, 72000 + N, N, K)
    rng = np.random.default_rng(M + K)
    dY = rng.integers(-4, 5, (M, N)) * (rng.random((M, N)) < 0.5)
    assert (np.abs(dY) @ mag).max() < 2.0 ** 24 * 2.0 ** -2
    got = ql.qmatmul_grad(fmt, pack(fmt, f, N, K), torch.from_numpy(dY.astype(np.float32)).cuda(), K)
    want = torch.from_numpy((dY @ W).astype(np.float32)).bfloat16()
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_grad_one_hot(fmt):
    """One value a row picks a row of the weights: each weight's rounding to
    fp16 and to bf16, whatever the size of the value (down to fp32's least)."""
    N, K = 130, 512
    w, W = weights(fmt, 72500, N, K, outliers=True)
    blocks = ql.isq(fmt, to_dev_bf16(w))
    for M, scale in ((40, 1.0), (130, 2.0 ** -60), (20, 2.0 ** 100)):
        rows = torch.arange(M, device="cuda") * 3 % N
        dY = torch.zeros((M, N), device="cuda")
        dY[torch.arange(M, device="cuda"), rows] = scale
        got = ql.qmatmul_grad(fmt, blocks, dY, K)
        # (FP8: the row's scale meets the gradient in fp32 and fp16 instead)
        within(got, W[rows] * scale, (W[rows] * scale).abs() * (E16 + 2 * U + 2.0 ** -8 * 1.001), f"one hot {fmt} {scale}")
    tiny = torch.zeros((1, N), device="cuda")
    tiny[0, 5] = 2.0 ** -149
    assert torch.isfinite(ql.qmatmul_grad(fmt, blocks, tiny, K)).all()


def test_grad_range_within_a_row():
    """Values 2^-24 of their row's largest keep their digits."""
    N, K, M = 256, 256, 4
    w, W = weights("q8_0", 72600, N, K)
    blocks = ql.isq("q8_0", to_dev_bf16(w))
    dY = torch.zeros((M, N), device="cuda")
    dY[:, 0] = 1.0
    dY[:, 1:] = 2.0 ** -24 * torch.randn((M, N - 1), device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    W0 = W.clone()
    W0[0] = 0  # the largest meets weights of 0 in a second weight
    b0 = ql.isq("q8_0", torch.where(torch.arange(N, device="cuda")[:, None] == 0, 0.0, to_dev_bf16(w).float()).bfloat16())
    y = dY.double() @ W0
    den = dY.double().abs() @ W0.abs()
    got = ql.qmatmul_grad("q8_0", b0, dY, K)
    # fp16 keeps 11 bits down to 2^-14 / 2^14 = 2^-28 of the largest
    within(got, y, rounded(y, (2 * E16 + (N + 9) * U) * den + 2.0 ** -39 * W0.abs().sum(0)), "range")
    del blocks, W


def test_grad_largest_and_smallest_values():
    """Gradients up to fp32's largest and down to its smallest normal."""
    N, K = 40, 256
    w, W = weights("q8_0", 72750, N, K)
    blocks = ql.isq("q8_0", to_dev_bf16(w))
    for M in (1, 3, 100):
        dY = gradients(4, M, N).sign() * torch.rand((M, N), device="cuda", generator=torch.Generator("cuda").manual_seed(M))
        for size in (torch.finfo(torch.float32).max, 2.0 ** -110):
            d = dY * size
            d[:, 0] = size
            y, tol = back(d.double(), W)
            got = ql.qmatmul_grad("q8_0", blocks, d, K)
            # (a result over bf16's range is infinite; one row's products lose
            # their last digits below 2^-126)
            fit = y.abs() < 3.3e38
            small = N * 2.0 ** -149
            within(torch.where(fit, got.double(), y), y, rounded(y, tol) + small, f"{M} rows of {size}")


def test_grad_rows_that_are_not_finite_stay_alone():
    N, K = 100, 256
    w, W = weights("q4k", 72700, N, K)
    blocks = ql.isq("q4k", to_dev_bf16(w))
    for M in (5, 40, 300):
        dY = gradients(3, M, N)
        clean = ql.qmatmul_grad("q4k", blocks, dY, K)
        bad = dY.clone()
        bad[1, 3], bad[2, 99], bad[4, 0] = float("inf"), float("nan"), -float("inf")
        got = ql.qmatmul_grad("q4k", blocks, bad, K)
        for m in (1, 2, 4):
            assert not torch.isfinite(got[m]).any()
        keep = [m for m in range(M) if m not in (1, 2, 4)]
        assert torch.equal(got[keep], clean[keep])


def test_grad_same_bits_and_surroundings():
    """Twice the same bits; nothing outside the results and the workspace is
    written, and a workspace of more rows gives the same."""
    N, K = 777, 512
    w, _ = weights("q6k", 72800, N, K)
    blocks = ql.isq("q6k", to_dev_bf16(w))
    big = ql.grad_workspace_bytes("q6k", 600, N, K)
    ws = torch.full((big + 256,), 255, dtype=torch.uint8, device="cuda")
    for M in (1, 2, 20, 33, 64, 100, 128, 129, 192, 193, 255, 256, 257, 300, 384, 385, 512, 576, 577, 600):
        dY = gradients(M, M, N)
        hold = torch.full((M + 2, K), 7.0, dtype=torch.bfloat16, device="cuda")
        a = ql.qmatmul_grad("q6k", blocks, dY, K, out=hold[1:M + 1], workspace=ws[:big])
        n = ql.grad_workspace_bytes("q6k", M, N, K)
        own = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
        b = ql.qmatmul_grad("q6k", blocks, dY, K, workspace=own[:n])
        assert torch.equal(a, b) and (own[n:] == 255).all() and (ws[big:] == 255).all()
        assert (hold[0] == 7).all() and (hold[M + 1] == 7).all()


def test_grad_in_chunks_of_rows():
    """More rows than go through at once (2^27 values: 4096 rows of 32768)."""
    M, N, K = 4400, 32768, 256
    w = to_dev_bf16(synth.weights_bf16(72900, N, K))
    blocks = ql.isq("q4_0", w)
    dY = torch.randn((M, N), device="cuda", generator=torch.Generator("cuda").manual_seed(9)).bfloat16()
    assert ql.grad_workspace_bytes("q4_0", M, N, K) == ql.grad_workspace_bytes("q4_0", 4096, N, K)
    got = ql.qmatmul_grad("q4_0", blocks, dY, K)
    for a, b in ((0, 4096), (4096, 4400)):
        assert torch.equal(got[a:b], ql.qmatmul_grad("q4_0", blocks, dY[a:b].contiguous(), K))
    W = ql.dequantize("q4_0", blocks, N, K).double()
    for m in (0, 4095, 4096, 4399):
        y, tol = back(dY[m:m + 1].double(), W)
        within(got[m:m + 1], y, rounded(y, tol), f"row {m}")


def test_grad_is_the_forward_products_difference():
    """<dY, qmatmul(X + h E) - qmatmul(X - h E)> / 2h is <dX, E>: exact in h, for
    a linear layer; X and E whole numbers that bf16 holds with their sums."""
    fmt, M, N, K = "q5_1", 6, 200, 512
    w, W = weights(fmt, 73000, N, K)
    blocks = ql.isq(fmt, to_dev_bf16(w))
    g = torch.Generator("cuda").manual_seed(4)
    X = torch.randint(-50, 51, (M, K), device="cuda", generator=g).float()
    E = torch.randint(-50, 51, (M, K), device="cuda", generator=g).float()
    dY = gradients(2, M, N)
    up, down = ql.qmatmul(fmt, blocks, (X + E).bfloat16(), N), ql.qmatmul(fmt, blocks, (X - E).bfloat16(), N)
    want = (dY.double() * (up.double() - down.double())).sum(1) / 2
    dX = ql.qmatmul_grad(fmt, blocks, dY, K).double()
    y, tol = back(dY.double(), W)
    # the forward bar: 1e-3 of its magnitudes
    f = 1e-3 * (dY.double().abs() * ((X.abs() + E.abs()).double() @ W.abs().t())).sum(1)
    assert ((dX * E).sum(1) - want).abs().le((rounded(y, tol) * E.abs()).sum(1) + f).all()


# ---------------------------------------------------------------------------
# the gated projection
# ---------------------------------------------------------------------------

# bounds of |act|' , |act'|' for the propagation of errors of G
SLOPE = {"silu": (1.1, 0.5), "relu": (1.0, 0.0), "sigmoid": (0.25, 0.0963)}


def act_and_slope(act, g):
    if act == "relu":
        return g.clamp(min=0), (g > 0).double()
    p, q = torch.sigmoid(g), torch.sigmoid(-g)
    return (g * p, p * (1 + g * q)) if act == "silu" else (p, p * q)


def check_glu(fmt, M, F, K, act, dtype=torch.float32, parts=True, empty=()):
    wg, Wg = weights(fmt, 74000 + F, F, K, outliers=True)
    wu, Wu = weights(fmt, 74001 + F, F, K)
    bg, bu = ql.isq(fmt, to_dev_bf16(wg)), ql.isq(fmt, to_dev_bf16(wu))
    X = to_dev_bf16(synth.activations_bf16(74100 + M, M, K))
    dH = gradients(M + F, M, F, dtype, empty)
    got = ql.qmatmul_glu_grad(fmt, bg, bu, X, dH, act=act, parts=parts)
    (g, eg), (u, eu) = forward(X.double(), Wg), forward(X.double(), Wu)
    d = dH.double()
    a, da = act_and_slope(act, g)
    dg, du = d * u * da, d * a
    s1, s2 = SLOPE[act]
    fp = 2.0 ** -19  # a dozen fp32 roundings, expf within two of them
    tu = d.abs() * s1 * eg + fp * du.abs()
    tg = d.abs() * (da.abs() * eu + (u.abs() + eu) * s2 * eg) + fp * dg.abs()
    # a term of act' that cancels (silu near its least) rounds against its parts
    tg = tg + fp * d.abs() * u.abs() * 2
    if act == "relu":  # at g = 0 but for its error, either side's derivative
        tg = torch.where(g.abs() <= eg, tg + d.abs() * (u.abs() + eu), tg)
    if parts:
        within(got.dG, dg, rounded(dg, tg), f"dG {fmt} {act} {M}x{F}x{K}")
        within(got.dU, du, rounded(du, tu), f"dU {fmt} {act} {M}x{F}x{K}")
    else:
        assert got.dG is None and got.dU is None
    y, tol = back(torch.cat([dg, du], 1), torch.cat([Wg, Wu], 0), torch.cat([tg, tu], 1))
    within(got.dX, y, rounded(y, tol), f"dX {fmt} {act} {M}x{F}x{K}")
    for m in empty:
        assert not got.dX[m % M].any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act", ACTS)
def test_glu_grad_formats(fmt, act):
    for M, F, K in ((1, 100, 512), (40, 130, 256), (130, 257, 512)):
        check_glu(fmt, M, F, K, act, torch.bfloat16 if M == 40 else torch.float32)


@pytest.mark.parametrize("fmt", TUNED)
@pytest.mark.parametrize("M,F,K", ((1, 1, 256), (2, 2000, 1024), (32, 64, 256), (33, 129, 768), (64, 127, 256), (65, 1000, 512),
                                   (128, 128, 256), (129, 65, 256), (300, 700, 1280)))
def test_glu_grad_sizes(fmt, M, F, K):
    check_glu(fmt, M, F, K, "silu", torch.float32 if M % 2 else torch.bfloat16, parts=F % 2 == 0, empty=(M - 1,) if M > 1 else ())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,F,K", ((3, 333, 4096), (4, 331, 4096), (3, 100, 5120), (3, 65, 8192), (20, 700, 4096), (85, 802, 1792)))
def test_glu_grad_few_rows(fmt, M, F, K):
    """Either side of where the first products change their form; splits of odd rows."""
    check_glu(fmt, M, F, K, "silu", parts=F % 2 == 1, empty=(M - 1,))


@pytest.mark.parametrize("M,F,K", ((3, 50, 32), (70, 100, 1056), (140, 33, 224)))
def test_glu_grad_rows_of_whole_blocks(M, F, K):
    check_glu("q8_0", M, F, K, "silu")


def test_glu_grad_far_gates():
    """Gates of +-100 and more, where e^-g overflows or vanishes: finite, and
    the limits' values."""
    F, K, M = 64, 256, 8
    W = torch.zeros((F, K), device="cuda")
    W[:, 0], W[:, 1] = 1.0, 0.5
    b = ql.isq("q8_0", W.bfloat16())
    X = torch.zeros((M, K), device="cuda")
    X[:, 0] = torch.tensor([0.0, 90.0, -90.0, 200.0, -200.0, 3e4, -3e4, 1.0], device="cuda")
    dH = torch.ones((M, F), device="cuda")
    Wd = ql.dequantize("q8_0", b, F, K).double()
    g = X.bfloat16().double() @ Wd.t()
    for act in ACTS:
        r = ql.qmatmul_glu_grad("q8_0", b, b, X.bfloat16(), dH, act=act, parts=True)
        a, da = act_and_slope(act, g)
        for got, want in ((r.dG, g * da), (r.dU, a)):
            assert torch.isfinite(got).all()
            # the results' 2^-8; g carries up to 2^-11 of itself, which e^-|g|
            # multiplies by |g|
            within(got, want, want.abs() * (2.0 ** -8 * 1.01 + 2.0 ** -10 * g.abs()) + 1e-30, f"far {act}")


def test_glu_grad_against_differences():
    """Central differences of the formula's forward pass in 64 bits along random
    directions of X."""
    fmt, M, F, K, h = "q6k", 5, 150, 256, 1e-5
    wg, Wg = weights(fmt, 75000, F, K)
    wu, Wu = weights(fmt, 75001, F, K)
    bg, bu = ql.isq(fmt, to_dev_bf16(wg)), ql.isq(fmt, to_dev_bf16(wu))
    X = to_dev_bf16(synth.activations_bf16(75002, M, K))
    dH = gradients(6, M, F)
    for act in ("silu", "sigmoid"):
        def loss(x):
            return (dH.double() * act_and_slope(act, x @ Wg.t())[0] * (x @ Wu.t())).sum(1)
        dX = ql.qmatmul_glu_grad(fmt, bg, bu, X, dH, act=act).dX.double()
        E = torch.randn((M, K), device="cuda", dtype=torch.float64, generator=torch.Generator("cuda").manual_seed(8))
        want = (loss(X.double() + h * E) - loss(X.double() - h * E)) / (2 * h)
        x = X.double()
        (g, eg), (u, eu) = forward(x, Wg), forward(x, Wu)
        a, da = act_and_slope(act, g)
        d = dH.double()
        tg, tu = d.abs() * (da.abs() * eu + (u.abs() + eu) * 0.5 * eg + 2.0 ** -18 * u.abs()), d.abs() * (1.1 * eg + 2.0 ** -19 * a.abs())
        y, tol = back(torch.cat([d * u * da, d * a], 1), torch.cat([Wg, Wu], 0), torch.cat([tg, tu], 1))
        # the differences' own error: h^2 times third derivatives, below 1e-6 of the magnitudes
        mag = (d.abs() * (a.abs() + da.abs() * u.abs())).sum(1) * E.abs().amax(1) * (Wg.abs() + Wu.abs()).sum(1).amax()
        assert ((dX * E).sum(1) - want).abs().le((rounded(y, tol) * E.abs()).sum(1) + 1e-6 * mag).all()


def test_glu_grad_same_bits_and_surroundings():
    F, K = 300, 512
    bg, bu = (ql.isq("q4k", to_dev_bf16(synth.weights_bf16(76000 + i, F, K))) for i in range(2))
    big = ql.glu_grad_workspace_bytes("q4k", 400, F, K)
    ws = torch.full((big + 256,), 255, dtype=torch.uint8, device="cuda")
    for M in (1, 2, 3, 33, 64, 65, 128, 192, 193, 200, 256, 385, 400):
        X = to_dev_bf16(synth.activations_bf16(76010 + M, M, K))
        dH = gradients(M, M, F)
        hold = [torch.full((M + 16, n), 7.0, dtype=torch.bfloat16, device="cuda") for n in (K, F, F)]
        a = ql.qmatmul_glu_grad("q4k", bg, bu, X, dH, out=ql.GluGrad(*(h[8:M + 8] for h in hold)), workspace=ws[:big])
        n = ql.glu_grad_workspace_bytes("q4k", M, F, K)
        own = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
        b = ql.qmatmul_glu_grad("q4k", bg, bu, X, dH, parts=True, workspace=own[:n])
        for u, v in zip(a, b):
            assert torch.equal(u, v)
        assert (own[n:] == 255).all() and (ws[big:] == 255).all()
        for h in hold:
            assert (h[:8] == 7).all() and (h[M + 8:] == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,x,h", ((40, 3, 9), (130, 128, 0), (2, 1, None), (2, None, 0), (1, 0, None), (1, None, 0)))
def test_glu_grad_rows_that_are_not_finite_stay_alone(fmt, act, M, x, h):
    """A NaN in row x of X, an infinity in row h of dH."""
    F, K = 100, 256
    bg, bu = (ql.isq(fmt, to_dev_bf16(synth.weights_bf16(76100 + i, F, K))) for i in range(2))
    X = to_dev_bf16(synth.activations_bf16(76110, M, K))
    dH = gradients(1, M, F)
    clean = ql.qmatmul_glu_grad(fmt, bg, bu, X, dH, act=act, parts=True)
    Xb, db = X.clone(), dH.clone()
    if x is not None:
        Xb[x, 7] = float("nan")
    if h is not None:
        db[h, 2] = float("inf")
    got = ql.qmatmul_glu_grad(fmt, bg, bu, Xb, db, act=act, parts=True)
    keep = [m for m in range(M) if m not in (x, h)]
    for a, b in zip(got, clean):
        assert torch.equal(a[keep], b[keep])
    if x is not None:
        assert not torch.isfinite(got.dX[x]).any()
    if h is not None and act != "relu":  # (a gate that ReLU holds shut takes no gradient)
        assert not torch.isfinite(got.dX[h]).any()


# ---------------------------------------------------------------------------
# streams, graphs, a training step
# ---------------------------------------------------------------------------


def test_two_streams_at_once():
    """Two calls in flight with workspaces of their own."""
    N, K, M = 2000, 1024, 300
    w, _ = weights("q4k", 77000, N, K)
    blocks = ql.isq("q4k", to_dev_bf16(w))
    dY = [gradients(i, M, N) for i in range(2)]
    want = [ql.qmatmul_grad("q4k", blocks, d, K) for d in dY]
    ws = [torch.empty(ql.grad_workspace_bytes("q4k", M, N, K), dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [torch.zeros((M, K), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                ql.qmatmul_grad("q4k", blocks, dY[i], K, out=out[i], workspace=ws[i])
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)


def test_training_step_together():
    """A step through a frozen decoder block and its head, as adapters' training
    runs it: the gated projection, the down projection, the head's cross
    entropy, and back -- eager and as a captured graph, replayed -- against the
    same step's gradients in 64 bits."""
    V, K, F, M = 1500, 512, 768, 37
    head, Wh = weights("q6k", 78000, V, K)
    (wg, Wg), (wu, Wu), (wd, Wd) = (weights(f, 78001 + i, r, c) for i, (f, r, c) in
                                    enumerate((("q4k", F, K), ("q4k", F, K), ("q5k", K, F))))
    bh, bg, bu, bd = (ql.isq(f, to_dev_bf16(w)) for f, w in (("q6k", head), ("q4k", wg), ("q4k", wu), ("q5k", wd)))
    X = to_dev_bf16(synth.activations_bf16(78010, M, K))
    t = torch.arange(M, dtype=torch.int32, device="cuda") * 13
    t[5] = -1
    wt = torch.full((M,), 1.0 / (M - 1), device="cuda")

    def step():
        h = ql.qmatmul_glu("q4k", bg, bu, X, F)
        y = (X.float() + ql.qmatmul("q5k", bd, h.bfloat16(), K)).bfloat16()
        r = ql.qmatmul_xent("q6k", bh, y, V, t, weights=wt)
        dh = ql.qmatmul_grad("q5k", bd, r.dX, F)
        dx = ql.qmatmul_glu_grad("q4k", bg, bu, X, dh).dX
        return r.loss, r.dX, dh, dx, (r.dX.float() + dx.float())

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
        with torch.cuda.graph(g, stream=s):
            res = step()
    torch.cuda.current_stream().wait_stream(s)
    for i in range(3):
        X.copy_(to_dev_bf16(synth.activations_bf16(78020 + i, M, K)))
        t.copy_((torch.arange(M, dtype=torch.int32, device="cuda") * 13 + i) % V)
        t[5 + i] = V if i else -1
        g.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        for a, b in zip(res[1:], eager[1:]):
            # qmatmul's split sums are atomic: y may round apart between two
            # runs, by a bf16 step in few places
            n = (a.double() - b.double()).norm() / b.double().norm()
            assert n <= 2.0 ** -8, n
        # the step in 64 bits on the oracle's weights
        x = X.double().requires_grad_()
        gate = x @ Wg.t()
        y = x + (gate * torch.sigmoid(gate) * (x @ Wu.t())) @ Wd.t()
        z = y @ Wh.t()
        ok = (t >= 0) & (t < V)
        lse = torch.logsumexp(z, 1)
        loss = torch.where(ok, lse - z.gather(1, t.clamp(0, V - 1).long()[:, None])[:, 0], 0.0)
        (loss * wt.double()).sum().backward()
        # y and h carry bf16's rounding: up to 2 * 2^-8 of y in each logit, of
        # which the loss sees two
        assert ((eager[0].double() - loss).abs() <= 2 * 2.0 ** -8 * (y.abs() @ Wh.abs().t()).amax(1)).all()
        rel = (eager[4].double() - x.grad).norm() / x.grad.norm()
        assert rel <= 4 * 2.0 ** -8, rel  # four bf16 tensors on the way
        assert eager[0][5 + i] == 0 and not eager[1][5 + i].any()


def test_captured_grad_replays_equal():
    """Every gradient call in one graph, replayed with eager work between:
    equal to the eager results, bit for bit."""
    N, K, M = 500, 512, 70
    w, _ = weights("q8_0", 79000, N, K)
    b = ql.isq("q8_0", to_dev_bf16(w))
    X = to_dev_bf16(synth.activations_bf16(79001, M, K))
    dY = gradients(7, M, N)
    t = torch.arange(M, dtype=torch.int32, device="cuda")

    def step():
        return (ql.qmatmul_grad("q8_0", b, dY, K), *ql.qmatmul_glu_grad("q8_0", b, b, X, dY, parts=True),
                *ql.qmatmul_xent("q8_0", b, X, N, t))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
        with torch.cuda.graph(g, stream=s):
            res = step()
    torch.cuda.current_stream().wait_stream(s)
    for i in range(4):
        X.copy_(to_dev_bf16(synth.activations_bf16(79010 + i, M, K)))
        dY.copy_(gradients(20 + i, M, N))
        g.replay()
        eager = step()
        torch.cuda.synchronize()
        for u, v in zip(res, eager):
            assert torch.equal(u, v)
