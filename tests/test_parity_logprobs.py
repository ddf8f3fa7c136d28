"""GPU parity of the log-probability calls against their definition in 64 bits
on the same fp32 logits.

Bar.  lse = m + ln z with z a sum of V terms e^(x - m): each term's exponent
rounds by |x - m| 2^-24 twice (the difference and its scaling to base 2) and
v_exp_f32 by a step; terms with |x - m| = d weigh e^-d, and d e^-d <= 1/e, so
z is off by at most (2 d + 4) 2^-24 relative where most of its mass sits at d
<= 32; a thread adds its V / 512 terms one by one (error at most V / 512 *
2^-24 relative) and the joins add 16 more.  With ln z and two subtractions
an absolute error of
    (2 * 32 + 4 + V / 512 + 20) 2^-24 + 3 * 2^-24 * max(|x - m|, ln z)
bounds lse - m, a log probability and, through the weighted sum of (x - m),
min(32, ln V + 1) times the first part bounds the entropy."""
import numpy as np
import pytest
import torch

import ggml_block_quant_amd as ql
import oracle
import synth
from gpu_util import to_dev_bf16

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def want(x, t, top):
    x = x.astype(np.float64)
    M, V = x.shape
    m = x.max(1, keepdims=True)
    m0 = np.where(m > -np.inf, m, 0)
    live = x > -np.inf
    e = np.where(live, np.exp(np.where(live, x - m0, 0)), 0)
    z = e.sum(1, keepdims=True)
    some = z[:, 0] > 0
    lz = np.log(np.where(z > 0, z, 1))
    lp = np.where(live, x - m0 - lz, -np.inf)
    ent = np.where(some, (lz - np.where(live, e * (x - m0), 0).sum(1, keepdims=True) / np.where(z > 0, z, 1))[:, 0], 0)
    out = {"entropy": ent, "lz": lz[:, 0]}
    if t is not None:
        ok = (t >= 0) & (t < V)
        at = np.clip(t, 0, V - 1)
        xt = x[np.arange(M), at]
        out["logprob"] = np.where(ok, lp[np.arange(M), at], 0)
        out["rank"] = np.where(ok, (x > xt[:, None]).sum(1) + 1, 0)
    if top:
        order = np.argsort(-x, axis=1, kind="stable")[:, :top]
        ids = np.full((M, top), -1)
        tl = np.full((M, top), -np.inf)
        n = order.shape[1]
        v = np.take_along_axis(lp, order, 1)
        ids[:, :n] = np.where(v > -np.inf, order, -1)
        tl[:, :n] = v
        out["top_ids"], out["top_logprobs"] = ids, tl
    return out


def close(got, ref, part, label):
    got = got.cpu().numpy().astype(np.float64)
    inf = ~np.isfinite(ref)
    assert np.array_equal(got[inf], ref[inf]), f"{label}: masked places"
    tol = part + 3 * U * np.abs(ref[~inf])
    assert (np.abs(got[~inf] - ref[~inf]) <= tol).all(), f"{label}: {np.abs(got[~inf] - ref[~inf]).max():.3e} > {np.max(tol):.3e}"


def check(x, t, top, got=None, label="", extra=0.0):
    """x, t: host arrays; got: a LogProbs (computed here if None); extra: error
    of the logits themselves."""
    M, V = x.shape
    if got is None:
        got = ql.logprobs(torch.from_numpy(x).cuda(), None if t is None else torch.from_numpy(t).cuda(), top)
    ref = want(x, t, top)
    part = (2 * 32 + 4 + V / 512 + 20 + 3 * np.log(V + 1)) * U + extra
    if t is not None:
        if not extra:
            assert np.array_equal(got.rank.cpu().numpy(), ref["rank"]), f"{label}: rank"
        close(got.logprob, ref["logprob"], part, f"{label} logprob")
    close(got.entropy, ref["entropy"], part * min(32, np.log(V) + 1) + extra, f"{label} entropy")
    if top:
        if not extra:
            assert np.array_equal(got.top_ids.cpu().numpy(), ref["top_ids"]), f"{label}: alternatives"
        close(got.top_logprobs, ref["top_logprobs"], part, f"{label} top")


def logits(seed, M, V):
    return (np.random.default_rng(seed).standard_normal((M, V)) * 3).astype(np.float32)


@pytest.mark.parametrize("V", (1, 2, 3, 5, 63, 64, 65, 511, 1000, 8189, 8192, 8193, 20001, 70000))
@pytest.mark.parametrize("top", (0, 1, 5, 20, 64))
def test_sizes(V, top):
    for M in (1, 2, 7):
        x = logits(V + M, M, V)
        t = np.random.default_rng(V).integers(0, V, M).astype(np.int32)
        check(x, t, top, label=f"M={M} V={V} top={top}")


@pytest.mark.parametrize("M,V,top", ((1, 131072, 5), (1100, 9001, 8), (3, 300001, 20), (2000, 700, 3)))
def test_many_rows_and_long_rows(M, V, top):
    """One part per row and several; odd rows start at every alignment."""
    x = logits(M, M, V)
    t = np.random.default_rng(V).integers(-2, V + 2, M).astype(np.int32)
    check(x, t, top, label=f"M={M} V={V}")


def test_without_targets_and_partial_results():
    x = logits(1, 4, 999)
    check(x, None, 3)
    X = torch.from_numpy(x).cuda()
    out = ql.LogProbs(None, torch.empty(4, dtype=torch.int32, device="cuda"), None, None, None)
    r = ql.logprobs(X, torch.tensor([1, 2, 3, 998], dtype=torch.int32, device="cuda"), out=out)
    assert np.array_equal(r.rank.cpu().numpy(), want(x, np.array([1, 2, 3, 998]), 0)["rank"])
    assert ql.logprobs(X[:0], top=2).top_ids.shape == (0, 2)


@pytest.mark.parametrize("M,V", ((3, 5000), (2, 40000), (1200, 3000)))
def test_strided_rows(M, V):
    """Rows apart, starting at an odd element; what lies between and behind
    them (NaN) is not part of any row."""
    ld = V + 13
    buf = torch.full((M * ld + 1,), float("nan"), device="cuda")
    x = logits(7, M, V)
    view = buf[1:].as_strided((M, V), (ld, 1))
    view.copy_(torch.from_numpy(x))
    t = np.random.default_rng(1).integers(0, V, M).astype(np.int32)
    check(x, t, 6, ql.logprobs(view, torch.from_numpy(t).cuda(), 6), "strided")
    # the last row ends where its allocation ends
    tail = torch.empty(M * V + 3, device="cuda")[3:].view(M, V)
    tail.copy_(torch.from_numpy(x))
    check(x, t, 6, ql.logprobs(tail, torch.from_numpy(t).cuda(), 6), "tail")


@pytest.mark.parametrize("V", (300, 9000, 50000))
def test_masks(V):
    rng = np.random.default_rng(V)
    x = logits(2, 9, V)
    low = np.finfo(np.float32).min
    x[0] = -np.inf                                  # nothing left
    x[1, 1:] = -np.inf                              # one token left
    x[2, rng.random(V) < 0.99] = -np.inf
    x[3] = low                                      # the lowest value everywhere: uniform
    x[4, rng.random(V) < 0.9] = low                 # and as a mask
    x[5, :V // 2] = -np.inf
    x[6] = -np.inf
    x[6, V - 1] = low
    x[7, 5] = 1e30                                  # one token takes everything
    x[8] *= 30                                      # differences past e^-100
    t = np.full(9, V - 1, np.int32)
    t[7], t[1] = 5, 0
    check(x[:8], t[:8], 10, label="masks")
    check(x[:8], np.zeros(8, np.int32), 64, label="masks 64")
    got = ql.logprobs(torch.from_numpy(x[8:]).cuda(), torch.from_numpy(t[8:]).cuda(), 10)
    ref = want(x[8:], t[8:], 10)
    assert np.array_equal(got.top_ids.cpu().numpy(), ref["top_ids"]) and np.array_equal(got.rank.cpu().numpy(), ref["rank"])


@pytest.mark.parametrize("V", (100, 8192, 30000, 140000))
@pytest.mark.parametrize("top", (1, 20, 64))
def test_ties_and_orders(V, top):
    """Rows that defeat a threshold taken from the row's start: all equal, a
    few distinct values, rising, falling, the best at the end, bf16 steps."""
    rng = np.random.default_rng(V)
    rows = [np.zeros(V), np.full(V, -3.5), rng.integers(0, 2, V), rng.integers(0, 9, V),
            np.arange(V) * 1e-3, -np.arange(V) * 1e-3, np.r_[np.zeros(V - 30), np.arange(1, 31)],
            np.where(np.arange(V) % 2 == 0, 0.0, -0.0), (np.arange(V) // 700) * 0.5]
    x = np.stack(rows).astype(np.float32)
    b = logits(5, 2, V)
    x = np.concatenate([x, (b.view(np.uint32) & 0xFFFF0000).view(np.float32)])
    t = rng.integers(0, V, len(x)).astype(np.int32)
    check(x, t, top, label=f"ties V={V} top={top}")


def test_many_tied_rows():
    """One part per row (M over a thousand): the same rows through the
    single-kernel form."""
    V = 20000
    x = np.zeros((1030, V), np.float32)
    x[1::4] = np.arange(V) * 1e-3
    x[2::4, ::3] = 1.0
    x[3::4] = logits(1, 1, V)
    t = np.arange(1030).astype(np.int32)
    check(x, t, 20, label="tied rows")


def test_same_bits_twice_and_surroundings():
    x = torch.from_numpy(logits(11, 5, 50000)).cuda()
    t = torch.arange(5, dtype=torch.int32, device="cuda")
    n = ql.logprobs_workspace_bytes(5, 50000, 9)
    ws = torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda")
    big = torch.full((7, 9), 3.0, device="cuda")
    a = ql.logprobs(x, t, 9)
    out = ql.LogProbs(*[torch.zeros_like(v) for v in a[:4]], big[1:6])
    b = ql.logprobs(x, t, 9, out=out, workspace=ws[:n])
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    assert (big[0] == 3).all() and (big[6] == 3).all() and (ws[n:] == 255).all()


@pytest.mark.parametrize("fmt,M,N,K", (("q6k", 1, 5000, 512), ("q4k", 9, 3001, 256), ("q8_0", 70, 1000, 544), ("q5_0", 3, 777, 256)))
def test_head(fmt, M, N, K):
    """The logits themselves are qmatmul's, whose error is bounded by 2^-16 of
    sum |w||x| (a bf16 pair per weight, fp32 sums) on every path."""
    w = synth.weights_bf16(51000 + N, N, K)
    blocks = ql.isq(fmt, to_dev_bf16(w))
    x = synth.activations_bf16(51100, M, K)
    W = oracle.dequant(fmt, oracle.quantize(fmt, w), N, K)
    y, den = oracle.matmul_a16(W, x)
    t = np.random.default_rng(N).integers(0, N, M).astype(np.int32)
    got = ql.qmatmul_logprobs(fmt, blocks, to_dev_bf16(x), N, torch.from_numpy(t).cuda(), 4)
    check(np.asarray(y).astype(np.float64), t, 4, got, f"head {fmt}", extra=2 * 2.0 ** -16 * float(np.max(den)))
    # and exactly those of the logits that qmatmul gives
    two = ql.logprobs(ql.qmatmul(fmt, blocks, to_dev_bf16(x), N), torch.from_numpy(t).cuda(), 4)
    for a, b in zip(got, two):
        assert torch.equal(a, b)


def test_head_in_chunks():
    """More rows than the workspace's logits hold: 2^26 / 262144 = 256 rows at
    a time, the last chunk ragged."""
    fmt, M, N, K = "q4_0", 300, 262144, 256
    w = synth.weights_bf16(52000, N, K)
    blocks = ql.isq(fmt, to_dev_bf16(w))
    x = to_dev_bf16(synth.activations_bf16(52100, M, K))
    t = torch.arange(M, dtype=torch.int32, device="cuda")
    assert ql.head_workspace_bytes(fmt, M, N, K, 3) < 4 * M * N
    got = ql.qmatmul_logprobs(fmt, blocks, x, N, t, 3)
    for a, b in ((0, 256), (256, 300)):
        part = ql.logprobs(ql.qmatmul(fmt, blocks, x[a:b].contiguous(), N), t[a:b].contiguous(), 3)
        for u, v in zip(got, part):
            assert torch.equal(u[a:b], v)


def test_decoder_step_together():
    """The operators in a row, as a decode step uses them: embedding, a
    quantized router, the experts, the tied head's log probabilities -- eager
    and as a captured graph, replayed."""
    V, K, F, E, k, T = 3000, 512, 256, 8, 2, 6
    table = ql.isq("q6k", to_dev_bf16(synth.weights_bf16(53000, V, K)))
    router = ql.isq("q8_0", to_dev_bf16(synth.weights_bf16(53001, E, K)))
    gate, up = (ql.isq("q4k", to_dev_bf16(synth.weights_bf16(53002 + i, E * F, K))) for i in range(2))
    down = ql.isq("q6k", to_dev_bf16(synth.weights_bf16(53004, E * K, F)))
    tok = torch.zeros(T, dtype=torch.int32, device="cuda")
    nxt = torch.zeros(T, dtype=torch.int32, device="cuda")

    def step():
        x = (ql.embed("q6k", table, V, K, tok) * 40).bfloat16()
        ids, w = ql.moe_route(ql.qmatmul("q8_0", router, x, E), k)
        y = ql.qmatmul_moe("q4k", gate, up, down, x, ids, w, E, F, fmt_down="q6k")
        h = (x.float() + y).bfloat16()
        return ql.qmatmul_logprobs("q6k", table, h, V, nxt, 5), ids, h

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
        with torch.cuda.graph(g, stream=s):
            res, ids, h = step()
    torch.cuda.current_stream().wait_stream(s)
    for i in range(3):
        tok.copy_(torch.arange(T, dtype=torch.int32) * 97 + i)
        nxt.copy_(torch.arange(T, dtype=torch.int32) * 31 + i)
        g.replay()
        torch.cuda.synchronize()
        r2, ids2, h2 = step()
        torch.cuda.synchronize()
        assert torch.equal(ids, ids2) and torch.equal(h, h2)
        for a, b in zip(res, r2):
            assert torch.equal(a, b)
        y = ql.qmatmul("q6k", table, h2, V).cpu().numpy()
        check(y, nxt.cpu().numpy(), 5, r2, "step")
