"""The cross entropy over a quantized head (qmatmul_xent): heads some of whose
rows are not finite, and every digit of the logits, seen through lse and loss
where one entry is sure."""
import numpy as np
import pytest
import torch

import ggml_block_quant_amd as ql
import oracle
import synth
from grad_util import E16, FMTS, rounded, within
from gpu_util import to_dev_bf16
from test_moe_precision import LEG, fields, pack, values


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", (1, 2, 5, 40, 130))
def test_head_rows_that_are_not_finite_reach_every_token(fmt, M):
    """Entries of the vocabulary whose scale is NaN, all of those that one
    workgroup passes over (1728 of 5000 logits, the last 1544) and no others:
    every scored token's loss, lse and gradient are not finite, whichever run
    they and the token's own entry are in."""
    N, K, run = 5000, 256, 1728
    f = oracle.quantize_fp8(synth.weights_bf16(85000, N, K)) if fmt == "fp8" else oracle.quantize(fmt, synth.weights_bf16(85000, N, K))
    X = to_dev_bf16(synth.activations_bf16(85001 + M, M, K))
    for bad in range(3):
        a, e = bad * run, min(N, (bad + 1) * run)
        g = {k: v.copy() for k, v in f.items()}
        if fmt == "fp8":
            g["s"][a:e] = np.nan
        else:
            d = g["d16"].reshape(N, -1)
            d[a:e] = 0x7e00
        blocks = pack(fmt, g, N, K)
        for other in (1, 2):
            t = torch.full((M,), run * ((bad + other) % 3) + 7, dtype=torch.int32, device="cuda")
            for grad in (True, False):
                r = ql.qmatmul_xent(fmt, blocks, X, N, t, grad=grad)
                assert not torch.isfinite(r.loss).any() and not torch.isfinite(r.lse).any(), (bad, other, grad)
                assert r.dX is None or not torch.isfinite(r.dX).any(), (bad, other)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", (1, 2, 3, 4, 5, 40, 130))
@pytest.mark.parametrize("N", (300, 5000))
def test_masked_tokens_that_are_not_finite(fmt, M, N):
    """Padding whose inputs are NaN or infinite: a token that is not scored has a
    loss of 0 and a gradient of zeros, one of weight 0 a gradient of zeros, and
    the others have the bits that they have beside finite padding."""
    K = 256
    blocks = ql.isq(fmt, to_dev_bf16(synth.weights_bf16(85100, N, K)))
    X = to_dev_bf16(synth.activations_bf16(85101 + M, M, K))
    t = torch.arange(M, dtype=torch.int32, device="cuda") * 7 % N
    wt = torch.linspace(0.5, 2.0, M, device="cuda")
    for pad in ([0], [M - 1], list(range(0, M, 3))):
        keep = [m for m in range(M) if m not in pad]
        for unscored in (True, False):
            tt, ww = t.clone(), wt.clone()
            if unscored:
                tt[pad] = -100
            else:
                ww[pad] = 0.0
            clean = ql.qmatmul_xent(fmt, blocks, X, N, tt, weights=ww)
            assert not clean.dX[pad].any()
            for value in (float("nan"), float("inf")):
                bad = X.clone()
                bad[pad, 9] = value
                r = ql.qmatmul_xent(fmt, blocks, bad, N, tt, weights=ww)
                assert not r.dX[pad].any() and not torch.isnan(r.dX[pad]).any(), (pad, unscored, value)
                if unscored:
                    assert not r.loss[pad].any()
                for a, b in zip(r, clean):
                    assert torch.equal(a[keep], b[keep])


# ---------------------------------------------------------------------------
# every digit of the logits
# ---------------------------------------------------------------------------

def digits(fmt, seed, N, K):
    """A [N][K] weight of up to 18 bits a value, all whole multiples of a format's
    unit, at most 2^7: (fields, values, magnitudes that sums may meet, unit)."""
    rng = np.random.default_rng(seed)
    G, B = N * K // 256, (N, K // 32)

    def ints(lo, hi, shape):
        return rng.integers(lo, hi + 1, shape)

    lo, hi = {"q8_0": (-127, 127), "q4k": (0, 15), "q6k": (-32, 31), "q5k": (0, 31), "q3k": (-4, 3), "q2k": (0, 3), "q4_0": (-8, 7),
              "q4_1": (0, 15), "q5_0": (-16, 15), "q5_1": (0, 31), "fp8": (-15, 15)}[fmt]
    q = ints(lo, hi, (N, K))
    if fmt == "fp8":
        f = fields(fmt, N, K, q, 2.0)
        w = values(fmt, f, N, K)
        return f, w, np.abs(w), 2.0
    if fmt in LEG or fmt == "q8_0":
        # d of 11 bits; a minimum near the middle of the codes
        unit = 2.0 ** -11 if fmt == "q8_0" else 2.0 ** -9
        d = ints(512, 767, B) * 2 + 1
        m = -(d * (hi // 2) // 32 * 32)  # (11 bits at most 2^15: fp16 holds it)
        f = fields(fmt, N, K, q, d * unit, m=m * unit if fmt in ("q4_1", "q5_1") else 0)
        w = values(fmt, f, N, K)
        mag = np.abs(np.repeat(d * unit, 32, 1) * q) + (np.repeat(np.abs(m) * unit, 32, 1) if fmt in ("q4_1", "q5_1") else 0)
        return f, w, mag, unit
    # d of 4 to 10 bits times sub-scales of 6 or 7 (Q2K: 4), minima in the middle
    bits, top, unit = {"q4k": (6, 63, 2.0 ** -10), "q5k": (5, 63, 2.0 ** -10), "q6k": (4, 127, 2.0 ** -10), "q3k": (8, 63, 2.0 ** -10),
                       "q2k": (10, 15, 2.0 ** -10)}[fmt]
    d = ints(2 ** (bits - 2), 2 ** (bits - 1) - 1, (G,)) * 2 + 1
    sc = ints(top // 2, top, (G, 8 if fmt == "q4k" else 16))
    mins = fmt in ("q4k", "q5k", "q2k")
    ml, mh = {"q4k": (7, 7), "q5k": (15, 15), "q2k": (1, 1)}.get(fmt, (0, 0))
    f = fields(fmt, N, K, q, d * unit, sc, d * ml * unit if mins else 0, np.minimum(sc, 63) if mins else 0)
    w = values(fmt, f, N, K)
    s = f["sc"][:, :8] if fmt == "q5k" else f["sc"].astype(np.int64)
    if fmt == "q6k":
        s = np.abs(s & ~15) + (s & 15)
    mag = np.repeat(s, 256 // s.shape[1], 1) * np.repeat(d, 256).reshape(G, 256) * unit * np.abs(q.reshape(G, 256))
    if mins:
        n = 16 if fmt == "q2k" else 8
        mag = mag + np.repeat(np.asarray(d * ml * unit)[:, None] * f["mq"][:, :n], 256 // n, 1)
    return f, w, mag.reshape(N, K), unit


DIGITS_N, DIGITS_K = 301, 4096


def digits_case(fmt, M):
    """Tokens whose logit of one entry (top) is more than 104 above any other, by
    X of +-1 with the entry's own signs at 32 places of either: e^(z - top) is 0
    in fp32 but for that entry, so lse is its logit, exactly, and the loss the
    difference of two logits, rounded once."""
    N, K = DIGITS_N, DIGITS_K
    f, w, mag, unit = digits(fmt, 88000, N, K)
    rng = np.random.default_rng(88001 + M)
    top = (np.arange(M) * 37 + 11) % N
    t = (top + 1 + np.arange(M) % (N - 1)) % N
    x = np.zeros((M, K))
    for m in range(M):
        for sign in (1, -1):
            x[m, rng.choice(np.flatnonzero(sign * w[top[m]] > 0), 32, replace=False)] = sign
    return f, w, mag, unit, x, top, t


@pytest.mark.parametrize("fmt", FMTS)
def test_digits_case_fits(fmt):
    """On the CPU: no sum rounds, the margins hold, and weights of one fp16 each
    (the low halves lost) would give most tokens another lse."""
    f, w, mag, unit, x, top, t = digits_case(fmt, 385)
    assert np.array_equal(w, np.round(w / unit) * unit) and np.abs(w).max() <= 128 and (np.abs(x) @ mag.T).max() * 1.002 < 2.0 ** 24 * unit
    z = x @ w.T
    i = np.arange(len(x))
    rest = z.copy()
    rest[i, top] = -np.inf
    assert (z[i, top] - rest.max(1) > 104).all() and (t != top).all()
    if fmt != "fp8":  # (codes of four bits under the row's scale)
        half = x @ w.astype(np.float16).astype(np.float64).T
        assert (half[i, top] != z[i, top]).mean() > 0.5


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", (1, 2, 3, 4, 20, 50, 100, 170, 256, 385))
def test_every_digit_of_the_logits(fmt, M):
    """Matrix-vector products, tiles of 32, 64, 128, 192 and 256 rows."""
    N, K = DIGITS_N, DIGITS_K
    f, w, _, _, x, top, t = digits_case(fmt, M)
    z = x @ w.T
    i = np.arange(M)
    X = to_dev_bf16(synth.bf16_bits_from_f32(x.astype(np.float32)))
    r = ql.qmatmul_xent(fmt, pack(fmt, f, N, K), X, N, torch.from_numpy(t.astype(np.int32)).cuda())
    assert np.array_equal(r.lse.cpu().numpy(), z[i, top].astype(np.float32))
    assert np.array_equal(r.loss.cpu().numpy(), (z[i, top] - z[i, t]).astype(np.float32))
    # dX = W[top] - W[t], each weight rounded to fp16 (FP8's codes and the scale of 2: exact)
    a, b = (torch.from_numpy(w[j]).cuda() for j in (top, t))
    within(r.dX, a - b, rounded(a - b, E16 * (a.abs() + b.abs())), f"dX {fmt} {M}")
