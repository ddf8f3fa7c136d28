"""GPU parity of the mixture-of-experts layer (qmatmul_moe) and its router
(q_moe_route) against their definitions in 64 bits.

Bar of the layer.  With A the largest |w| of each 32-element block of a row
(what a block's scale and minimum are of the order of), G = sum A_g |x|,
U = sum A_u |x|, an output's error is at most
    c * sum_j |w_j| sum_f A_d (L G |u| + |a(g)| U + |h| + c' G U)
where L is the activation's slope (at most 1.1) and c the relative error of
one product: for up to four tokens, fp32 sums of 32 terms per lane and at
most 32 joins after them, c = 64 * 2^-24; for more, bf16 pairs of weights and
H, each within 2^-17, so c = 2^-16 for the rounding of both operands of the
second product (one of a weight's and one of H), plus the sums:
c = 2^-16 + 2^-15 * 2^-1 + 64 * 2^-24 <= 2^-15."""
import numpy as np
import pytest
import torch

import ggml_block_quant_amd as ql
import oracle
import synth
from gpu_util import to_dev_bf16

pytestmark = pytest.mark.gpu

ALL = ("q8_0", "q4k", "q6k", "q2k", "q3k", "q5k", "q4_0", "q4_1", "q5_0", "q5_1", "fp8")


def bf16_to_f64(u16):
    return (u16.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def act64(name, g):
    if name == "relu":
        return np.maximum(g, 0)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-g))
    return g * s if name == "silu" else s


class Layer:
    """Random experts, quantized on the GPU and in the oracle."""

    def __init__(self, fmt, fmt_down, E, F, K, seed, scale=1.0):
        self.fmt, self.fmt_down, self.E, self.F, self.K = fmt, fmt_down, E, F, K
        self.dev, self.W, self.A = [], [], []
        for i, (f, n, k) in enumerate(((fmt, E * F, K), (fmt, E * F, K), (fmt_down, E * K, F))):
            w = synth.weights_bf16(seed + i, n, k, outliers=i == 0)
            self.dev.append(ql.isq(f, to_dev_bf16(w)))
            W = oracle.dequant_fp8(oracle.quantize_fp8(w)) if f == "fp8" else oracle.dequant(f, oracle.quantize(f, w), n, k)
            self.W.append(W.reshape(E, n // E, k))
            A = np.repeat(np.abs(W).reshape(n, k // 32, 32).max(2), 32, 1)
            self.A.append(A.reshape(E, n // E, k))

    def run(self, x, ids, w, act, **kw):
        return ql.qmatmul_moe(self.fmt, *self.dev, to_dev_bf16(x), torch.from_numpy(ids).cuda(),
                              torch.from_numpy(w).cuda(), self.E, self.F, act=act, fmt_down=self.fmt_down, **kw)

    def want(self, x, ids, w, act):
        X = bf16_to_f64(x)
        T, k = ids.shape
        y, bar = np.zeros((T, self.K)), np.zeros((T, self.K))
        for t in range(T):
            for j in range(k):
                e = int(ids[t, j])
                if not 0 <= e < self.E:
                    continue
                g, u = self.W[0][e] @ X[t], self.W[1][e] @ X[t]
                G, U = self.A[0][e] @ np.abs(X[t]), self.A[1][e] @ np.abs(X[t])
                a = act64(act, g)
                h = a * u
                y[t] += float(w[t, j]) * (self.W[2][e] @ h)
                bar[t] += abs(float(w[t, j])) * (self.A[2][e] @ (1.1 * G * np.abs(u) + np.abs(a) * U + np.abs(h) + 2.0 ** -15 * G * U))
        return y, bar

    def check(self, x, ids, w, act, label):
        got = self.run(x, ids, w, act).cpu().numpy().astype(np.float64)
        y, bar = self.want(x, ids, w, act)
        c = 64 * 2.0 ** -24 if len(ids) <= 4 else 2.0 ** -15
        err = np.abs(got - y)
        assert np.isfinite(got).all(), label
        assert (err <= c * bar).all(), f"{label}: {np.max(err / np.maximum(bar, 1e-30)):.3e} of the magnitudes > {c:.3e}"


def choice(seed, T, E, k, holes=True):
    """ids with repeated experts, ids outside [0, E), and a row without any."""
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    if holes:
        ids[rng.random((T, k)) < 0.15] = -1
        ids[rng.random((T, k)) < 0.05] = E
        if T > 2:
            ids[T // 2] = -1
            ids[T - 1] = [0] * k  # the same expert k times
    return ids, w


@pytest.mark.parametrize("fmt", ALL)
@pytest.mark.parametrize("T", (1, 3, 4, 5, 37))
def test_moe_every_format(fmt, T):
    E, F, K, k = 3, 256, 512, 2
    L = Layer(fmt, fmt, E, F, K, 41000 + T)
    ids, w = choice(T, T, E, k)
    if T == 1:
        ids[0] = [2, 0]
    L.check(synth.activations_bf16(41100 + T, T, K), ids, w, "silu", f"moe {fmt} T={T}")


@pytest.mark.parametrize("fmt,fmt_down,E,F,K,k,Ts", [
    ("q4k", "q6k", 5, 768, 1280, 3, (1, 2, 4, 7, 33)),
    ("q6k", "q4k", 4, 1280, 768, 4, (1, 3, 11, 64)),
    ("q8_0", "q8_0", 6, 352, 1056, 2, (1, 2, 4, 6, 50)),   # row lengths no multiple of 64 or 256
    ("q8_0", "q4k", 2, 256, 32, 1, (1, 2, 5)),             # the smallest rows
    ("q4k", "q8_0", 2, 32, 256, 2, (1, 4, 9)),
    ("q4k", "q4k", 1, 256, 256, 1, (1, 4, 5, 130, 300)),   # one expert: every pair in its tiles
])
@pytest.mark.parametrize("act", ("silu", "relu", "sigmoid"))
def test_moe_shapes(fmt, fmt_down, E, F, K, k, Ts, act):
    L = Layer(fmt, fmt_down, E, F, K, 42000 + F)
    for T in Ts:
        ids, w = choice(100 + T, T, E, k, holes=T != 1)
        L.check(synth.activations_bf16(42100 + T, T, K), ids, w, act, f"moe {fmt}/{fmt_down} {act} T={T}")


@pytest.mark.parametrize("fmt,fmt_down,F,K", [
    ("q4k", "q6k", 4096, 256),
    ("q6k", "q4k", 4352, 512),
    ("q8_0", "q8_0", 4128, 288),   # row lengths no multiple of a slab
    ("q8_0", "q4k", 4096, 32),
    ("q4k", "q8_0", 5152, 768),
])
def test_moe_tiles_of_sixteen(fmt, fmt_down, F, K):
    """Long rows of F and up to twelve pairs an expert (tiles of 16 pairs), and
    just above (tiles of 64)."""
    L = Layer(fmt, fmt_down, 3, F, K, 46000)
    for T in (5, 8, 18, 21):
        ids, w = choice(300 + T, T, 3, 2)
        L.check(synth.activations_bf16(46100 + T, T, K), ids, w, "silu", f"moe {fmt}/{fmt_down} F={F} T={T}")


@pytest.mark.parametrize("fmt", ("q8_0", "q4k", "q6k", "q5k", "q4_0"))
@pytest.mark.parametrize("F", (512, 4096))
def test_moe_scales_of_zero_and_wide_ranges(fmt, F):
    """Blocks, groups and rows of zeros, constants and offsets far above their
    spread (scales of 0, minimums of many scales), first in a row, inside and
    last; tokens of zeros, of one value, and over thirty binades."""
    E, K, k = 4, 768, 2
    L = Layer.__new__(Layer)
    L.fmt, L.fmt_down, L.E, L.F, L.K, L.dev, L.W, L.A = fmt, fmt, E, F, K, [], [], []
    for i, (n, kk) in enumerate(((E * F, K), (E * F, K), (E * K, F))):
        w = synth.weights_bf16(47000 + i, n, kk, outliers=False).reshape(n, kk)
        one = np.float32(1 / 64).view(np.uint32) >> 16
        w[0::16, :256] = 0                   # a group of zeros first,
        w[1::16, 256:512] = 0                # inside
        w[2::16, -256:] = 0                  # and last
        w[3::16] = 0                         # nothing but zeros
        w[4::16] = one                       # a constant row
        w[5::16, 32:64] = one                # a constant block
        w[6::16] = one + (w[6::16] & 1)      # the spread far below the offset
        w[7::16, :256] = one | 0x8000
        w[8::16, 64:] = 0                    # two blocks alone
        L.dev.append(ql.isq(fmt, to_dev_bf16(w)))
        W = oracle.dequant(fmt, oracle.quantize(fmt, w), n, kk)
        L.W.append(W.reshape(E, n // E, kk))
        A = np.repeat(np.abs(W).reshape(n, kk // 32, 32).max(2), 32, 1)
        L.A.append(A.reshape(E, n // E, kk))
    for T in (2, 6, 9, 20, 60):
        x = synth.activations_bf16(47100 + T, T, K).reshape(T, K)
        x[0] = 0
        if T > 2:
            x[1] = 0x3F80
            e = np.random.default_rng(T).integers(-15, 16, K)
            x[2] = (x[2] & 0x807F) | ((127 + e) << 7).astype(np.uint16)
        ids, w = choice(400 + T, T, E, k, holes=False)
        L.check(x, ids, w, "relu", f"moe {fmt} F={F} T={T}")


@pytest.mark.parametrize("fmt", ("q8_0", "q4k", "q6k", "q5k"))
@pytest.mark.parametrize("F,T", ((512, 3), (4096, 9), (512, 40)))
def test_moe_infinities_and_nan_stay_in_their_token(fmt, F, T):
    """A token whose X holds an infinity or a NaN has no finite output; the
    other tokens', which share its experts, are bit for bit what they were.
    (Every row of the weights meets the value: a product with 0 is NaN.)"""
    E, K, k = 3, 512, 2
    L = Layer(fmt, fmt, E, F, K, 49000)
    ids, w = choice(600 + T, T, E, k, holes=False)
    x = synth.activations_bf16(49100 + T, T, K).reshape(T, K)
    want = L.run(x, ids, w, "silu").cpu().numpy()
    bad = {0: 0x7FC0, T - 1: 0xFF80} if T > 1 else {0: 0x7FC0}
    for t, v in bad.items():
        x[t, 37 + t] = v
    got = L.run(x, ids, w, "silu").cpu().numpy()
    for t in range(T):
        if t in bad:
            assert not np.isfinite(got[t]).any(), t
        else:
            assert np.array_equal(got[t], want[t]), t


@pytest.mark.parametrize("T", (2, 9, 40))
def test_moe_two_streams_at_once(T):
    """Two calls in flight, each with its own workspace and stream, give what
    they give alone."""
    E, F, K, k = 8, 4096, 512, 2
    L = Layer("q4k", "q6k", E, F, K, 48000)
    args = []
    for i in range(2):
        ids, w = choice(500 + i, T, E, k, holes=False)
        args.append((to_dev_bf16(synth.activations_bf16(48100 + i, T, K)), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()))
    n = ql.moe_workspace_bytes("q4k", "q6k", T, E, k, F, K)
    bufs = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [[torch.zeros((T, K), device="cuda") for _ in range(8)] for _ in range(2)]

    def call(i, out):
        ql.qmatmul_moe("q4k", *L.dev, *args[i], E, F, fmt_down="q6k", out=out, workspace=bufs[i])

    alone = [torch.zeros((T, K), device="cuda") for _ in range(2)]
    for i in range(2):
        call(i, alone[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for r in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                call(i, outs[i][r])
    torch.cuda.synchronize()
    for i in range(2):
        for r in range(8):
            assert torch.equal(outs[i][r], alone[i])


def test_moe_long_rows():
    """Rows long enough for every wave of a workgroup and a second pass (K =
    18432: 576 chunks), and a down product over eight choices (2048 chunks)."""
    L = Layer("q4k", "q4k", 2, 256, 18432, 43000)
    ids, w = choice(5, 2, 2, 2, holes=False)
    L.check(synth.activations_bf16(43100, 2, 18432), ids, w, "silu", "moe long K")
    L = Layer("q8_0", "q4k", 8, 8192, 256, 43200)
    ids = np.arange(8, dtype=np.int32)[None].repeat(2, 0)
    w = np.random.default_rng(1).random((2, 8)).astype(np.float32)
    L.check(synth.activations_bf16(43300, 2, 256), ids, w, "silu", "moe long down")


def test_moe_many_experts():
    """More experts than pairs and than a tile's pairs; experts never chosen."""
    E, F, K, k = 100, 256, 256, 8
    L = Layer("q4k", "q4k", E, F, K, 44000)
    for T in (1, 4, 9, 200):
        rng = np.random.default_rng(T)
        ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
        L.check(synth.activations_bf16(44100 + T, T, K), ids, rng.random((T, k)).astype(np.float32), "silu", f"T={T}")


def test_moe_uneven_load():
    """All tokens on one expert of many, and pad rows behind the sequences."""
    E, F, K, k, T = 16, 256, 512, 2, 150
    L = Layer("q6k", "q6k", E, F, K, 45000)
    ids = np.full((T, k), 3, np.int32)
    ids[:, 1] = 7
    ids[100:] = -1
    w = np.random.default_rng(2).random((T, k)).astype(np.float32)
    x = synth.activations_bf16(45100, T, K)
    L.check(x, ids, w, "silu", "uneven")
    y = L.run(x, ids, w, "silu").cpu().numpy()
    assert (y[100:] == 0).all()


@pytest.mark.parametrize("T", (1, 4, 40))
def test_moe_no_expert_at_all(T):
    L = Layer("q4k", "q4k", 2, 256, 256, 46000)
    ids, w = np.full((T, 2), -1, np.int32), np.full((T, 2), np.nan, np.float32)
    ws = torch.full((ql.moe_workspace_bytes("q4k", "q4k", T, 2, 2, 256, 256),), 255, dtype=torch.uint8, device="cuda")
    y = L.run(synth.activations_bf16(46100, T, 256), ids, w, "silu", workspace=ws,
              out=torch.full((T, 256), float("nan"), device="cuda")).cpu().numpy()
    assert (y == 0).all()


@pytest.mark.parametrize("T", (2, 30))
def test_moe_workspace_and_surroundings(T):
    """A workspace full of NaN patterns changes nothing, twice the same call
    gives the same bits, and nothing beyond the given sizes is written."""
    E, F, K, k = 4, 256, 512, 2
    L = Layer("q4k", "q6k", E, F, K, 47000)
    ids, w = choice(9, T, E, k)
    x = synth.activations_bf16(47100, T, K)
    n = ql.moe_workspace_bytes("q4k", "q6k", T, E, k, F, K)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
    big = torch.full((T + 2, K), 7.0, device="cuda")
    a = L.run(x, ids, w, "silu", out=big[1:T + 1], workspace=ws[:n]).clone()
    b = L.run(x, ids, w, "silu")
    assert torch.equal(a, b)
    assert (big[0] == 7).all() and (big[T + 1] == 7).all() and (ws[n:] == 255).all()


def test_moe_empty():
    L = Layer("q4k", "q4k", 2, 256, 256, 48000)
    y = L.run(np.zeros((0, 256), np.uint16), np.zeros((0, 2), np.int32), np.zeros((0, 2), np.float32), "silu")
    assert y.shape == (0, 256)


@pytest.mark.parametrize("T", (1, 24))
def test_moe_graph_replays_and_streams(T):
    """Captured on a stream of its own and replayed with other inputs in the
    same buffers; every replay equals the eager call."""
    E, F, K, k = 4, 512, 512, 2
    L = Layer("q4k", "q4k", E, F, K, 49000)
    X = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    I = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    Wt = torch.zeros((T, k), device="cuda")
    lg = torch.zeros((T, E), device="cuda")
    Y = torch.zeros((T, K), device="cuda")
    ws = torch.empty(ql.moe_workspace_bytes("q4k", "q4k", T, E, k, F, K), dtype=torch.uint8, device="cuda")

    def call(out, ids, w, work):
        ql.moe_route(lg, k, ids=ids, weights=w)
        ql.qmatmul_moe("q4k", *L.dev, X, ids, w, E, F, out=out, workspace=work)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        call(Y, I, Wt, ws)
        with torch.cuda.graph(g, stream=s):
            call(Y, I, Wt, ws)
    torch.cuda.current_stream().wait_stream(s)
    for i in range(4):
        X.copy_(to_dev_bf16(synth.activations_bf16(49100 + i, T, K)))
        lg.copy_(torch.from_numpy(np.random.default_rng(i).standard_normal((T, E)).astype(np.float32)))
        g.replay()
        torch.cuda.synchronize()
        y, ids, w = torch.empty_like(Y), torch.empty_like(I), torch.empty_like(Wt)
        call(y, ids, w, torch.empty_like(ws))
        torch.cuda.synchronize()
        assert torch.equal(ids, I) and torch.equal(w, Wt) and torch.equal(y, Y), i


# ----------------------------------------------------------------------------
# router
# ----------------------------------------------------------------------------

def route_want(x, k, score, bias=None, renorm=True, scale=1.0):
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    x = np.minimum(x, np.finfo(np.float32).max)
    T, E = x.shape
    live = x > -np.inf
    if score == "softmax":
        m = np.where(live.any(1), x.max(1), 0)[:, None]
        e = np.where(live, np.exp(np.where(live, x - m, 0)), 0)
        p = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    else:
        with np.errstate(over="ignore"):
            p = np.where(live, 1 / (1 + np.exp(-np.where(live, x, 0))), 0)
    key = x if bias is None else np.where(live, p + bias.astype(np.float64), -np.inf)
    order = np.argsort(-key, axis=1, kind="stable")[:, :k]
    ids = np.where(np.take_along_axis(key, order, 1) > -np.inf, order, -1).astype(np.int32)
    w = np.where(ids >= 0, np.take_along_axis(p, order, 1), 0)
    if renorm:
        z = w.sum(1, keepdims=True)
        w = np.where(z > 0, w / np.where(z > 0, z, 1), 0)
    return ids, w * scale


def check_route(x, k, **kw):
    bias = kw.get("bias")
    got_ids, got_w = ql.moe_route(torch.from_numpy(x).cuda(), k, **{**kw, "bias": None if bias is None else torch.from_numpy(bias).cuda()})
    ids, w = route_want(x, k, **kw)
    assert np.array_equal(got_ids.cpu().numpy(), ids)
    got = got_w.cpu().numpy().astype(np.float64)
    # fp32 e^(x - m) of differences up to 32: the difference rounds by half a
    # step (32 * 2^-24 in the exponent), expf by 2 steps, the sum of up to
    # 1024 such terms and the quotient by less than 16 more; both sides of the quotient
    tol = 2 * (32 + 2 + 16) * 2.0 ** -24
    assert (np.abs(got - w) <= tol * np.abs(w) + 1e-37).all(), np.abs(got - w).max()


@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
@pytest.mark.parametrize("E,k", ((1, 1), (2, 2), (8, 2), (63, 8), (64, 1), (65, 32), (128, 8), (200, 7), (256, 8), (512, 5), (1000, 32), (1024, 9)))
def test_route(score, E, k):
    for T in (1, 3, 66):
        x = np.random.default_rng(E + T).standard_normal((T, E)).astype(np.float32) * 2
        for renorm in (True, False):
            check_route(x, k, score=score, renorm=renorm, scale=2.5)
        if score == "sigmoid":
            check_route(x, k, score=score, bias=np.random.default_rng(3).standard_normal(E).astype(np.float32) * 0.2)


@pytest.mark.parametrize("E", (8, 130, 700))
def test_route_ties_masks_and_extremes(E):
    rng = np.random.default_rng(E)
    k = 8
    x = rng.integers(0, 3, (40, E)).astype(np.float32)   # ties everywhere
    x[1] = 0.0
    x[2, ::2] = -0.0
    x[2, 1::2] = 0.0                                      # -0 equals +0
    x[3] = -np.inf                                        # nothing left
    x[4, 3:] = -np.inf                                    # fewer than k left
    x[5] = np.finfo(np.float32).min                       # the lowest value is a value
    x[6, ::3] = np.finfo(np.float32).min
    x[7, 1] = np.nan
    x[8, :] = np.nan
    x[9, 2] = np.inf
    x[10] = -np.inf
    x[10, E - 1] = -50.0
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check_route(x[:9], k, score=score, renorm=renorm)
            check_route(x[10:], k, score=score, renorm=renorm)
    check_route(x[:9], k, score="sigmoid", bias=np.zeros(E, np.float32))
    got, w = ql.moe_route(torch.from_numpy(x[9:10]).cuda(), k)
    assert got[0, 0].item() == 2 and w[0, 0].item() == 1.0


def test_route_close_keys_with_bias():
    """Keys that differ by less than a step of fp32 are told apart."""
    E = 64
    x = np.zeros((2, E), np.float32)
    x[0, 10], x[0, 50] = 4.0, np.nextafter(np.float32(4.0), np.float32(5))
    b = np.zeros(E, np.float32)
    ids, _ = ql.moe_route(torch.from_numpy(x).cuda(), 2, score="sigmoid", bias=torch.from_numpy(b).cuda())
    assert ids[0].tolist() == [50, 10] and ids[1].tolist() == [0, 1]


def test_route_into_given_buffers_and_empty():
    x = torch.randn(5, 32, device="cuda")
    ids, w = torch.empty(5, 4, dtype=torch.int32, device="cuda"), torch.empty(5, 4, device="cuda")
    a, b = ql.moe_route(x, 4, ids=ids, weights=w)
    assert a.data_ptr() == ids.data_ptr() and b.data_ptr() == w.data_ptr()
    assert torch.allclose(w.sum(1), torch.ones(5, device="cuda"), atol=5 * 2.0 ** -23)
    ids, w = ql.moe_route(x[:0], 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)


def test_route_bias_that_switches_off():
    """A bias of -inf or NaN: the expert is never chosen, by any token; one of
    +inf: always, the lowest such expert first."""
    T, E, k = 9, 130, 8
    x = np.random.default_rng(5).standard_normal((T, E)).astype(np.float32)
    b = np.zeros(E, np.float32)
    b[[0, 64, 129]] = np.nan
    b[[1, 63, 128]] = -np.inf
    b[[70, 5]] = np.inf
    ids, w = ql.moe_route(torch.from_numpy(x).cuda(), k, score="sigmoid", bias=torch.from_numpy(b).cuda())
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    off = (0, 64, 129, 1, 63, 128)
    for t in range(T):
        rest = sorted((e for e in range(E) if e not in off and e not in (5, 70)), key=lambda e: (-np.float64(x[t, e]), e))
        assert list(ids[t]) == [5, 70] + rest[:k - 2]
    assert np.isfinite(w).all()
    b[:] = np.nan
    ids, w = ql.moe_route(torch.from_numpy(x).cuda(), k, score="sigmoid", bias=torch.from_numpy(b).cuda())
    assert (ids == -1).all() and (w == 0).all()
