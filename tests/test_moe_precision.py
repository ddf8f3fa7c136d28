"""The mixture-of-experts layer against bars that see a lost bit.

A bar on the magnitudes summed by two products after each other is far above
what the values between them (H) lose to their own rounding.  Here the block
buffers are written field by field instead, so that no sum rounds and what is
left is one thing at a time:

one-hot rows   every row of every weight has one non-zero code, so a value of
               H is one product of two exact numbers and an output one weight
               times one value of H: H seen place by place.
whole numbers  dense rows of small whole numbers times powers of two, of which
               every partial sum fits 24 bits: outputs have to be equal.

Bars of the one-hot outputs (u = 2^-24, half a step of fp32; y the outputs'
terms, each held to its own bar).  h = act(g) * u is exact but for one fp32
rounding (u |h|); after it a term meets at most eight more (unit times weight,
scale, the digits' two, the sum of the two choices, the products hi and lo,
their sum): 9 u |y| in all.  H itself rounds by its form:
  digits   (up to four tokens, or two pairs an expert; Q4K, Q6K, Q8_0 down)
           half a unit of 2^-e, the largest of a chunk of 32 being at least
           4177855 units: below 1.01 * 2^-23 of that largest;
  fp32     (the same, the other down formats) nothing;
  fp16     (more pairs; both formats of the three) hi and lo of 11 bits, 2^-23
           of the value, and half the smallest fp16 where the row's largest is
           at least 2^14: 2^-39 of that largest;
  bf16     (more pairs, any other pair of formats) hi and lo of 8 bits, 2^-17."""
import numpy as np
import pytest
import torch

import ggml_block_quant_amd as ql
import oracle
import synth
from gpu_util import to_dev_bf16

U = 2.0 ** -24
TUNED = ("q8_0", "q4k", "q6k")
LEG = ("q4_0", "q4_1", "q5_0", "q5_1")


def form_of(fmt, fmt_down, T, E, k, F=0, K=0):
    """How H is held between the two products (include/qlinear.h)."""
    if T <= 4 or T * k <= 2 * E:
        return "digits" if fmt_down in TUNED else "fp32"
    fits = F * K < 2 ** 31 and T * ((K + 255) // 256 * 256) < 2 ** 31
    return "fp16" if fmt in TUNED and fmt_down in TUNED and fits else "bf16"


def h_error(form, h):
    """The largest error of each value of H [..., F] in its form."""
    a = np.abs(h)
    if form == "digits":
        c = a.reshape(*a.shape[:-1], -1, 32).max(-1, keepdims=True)
        return np.broadcast_to(1.01 * 2.0 ** -23 * c, c.shape[:-1] + (32,)).reshape(a.shape)
    if form == "fp16":
        return 2.0 ** -23 * a + 2.0 ** -39 * a.max(-1, keepdims=True)
    return 2.0 ** -17 * a if form == "bf16" else 0 * a


def f16_bits(a):
    return np.asarray(a, np.float16).view(np.uint16)


def fields(fmt, rows, cols, q, d, sc=1, dmin=0, mq=0, m=0):
    """The logical fields of `fmt`: codes q, one d per 256 (legacy and Q8_0: per
    32), sub-scales sc, Q4K's / Q5K's / Q2K's dmin and mq, Q4_1's / Q5_1's m."""
    G, B = rows * cols // 256, (rows, cols // 32)
    if fmt == "fp8":
        return {"q": oracle.e4m3_from_f32_array(np.asarray(q, np.float32)), "s": np.full(rows, d, np.float32)}
    if fmt in LEG or fmt == "q8_0":
        f = {"d16": np.broadcast_to(f16_bits(d), B).copy(), "q": q.astype(np.int8)}
        if fmt != "q8_0":
            f["m16"] = np.broadcast_to(f16_bits(m), B).copy()
        return f
    ns = 8 if fmt == "q4k" else 16
    f = {"d16": np.broadcast_to(f16_bits(d), (G,)).copy(), "sc": np.broadcast_to(sc, (G, ns)).astype(np.int8 if fmt == "q6k" else np.uint8),
         "q": q.astype(np.uint8 if fmt == "q4k" else np.int8)}
    if fmt != "q6k":
        f["dmin16"] = np.broadcast_to(f16_bits(dmin), (G,)).copy()
        f["mq"] = np.broadcast_to(mq, (G, ns)).astype(np.uint8)
    return f


def pack(fmt, f, rows, cols):
    b = oracle.pack_fp8(f) if fmt == "fp8" else oracle.pack(fmt, f, rows, cols)
    return torch.from_numpy(b).cuda()


def values(fmt, f, rows, cols):
    return oracle.dequant_fp8(f) if fmt == "fp8" else oracle.dequant(fmt, f, rows, cols)


# ----------------------------------------------------------------------------
# one-hot rows
# ----------------------------------------------------------------------------

def one_hot(fmt, seed, rows, cols, pos, any_scale=False):
    """A [rows][cols] weight whose row n is zero but for column pos[n], as
    (fields, value per row): at most 8 bits, the scales powers of 2; positive,
    or any_scale: of either sign and over the whole range of fp16."""
    rng = np.random.default_rng(seed)
    top = {"q8_0": 127, "q4k": 15, "q6k": 31, "q5k": 31, "q3k": 3, "q2k": 3, "q4_0": 7, "q4_1": 15, "q5_0": 15, "q5_1": 31, "fp8": 15}[fmt]
    q = np.zeros((rows, cols), np.int16)
    q[np.arange(rows), pos] = rng.integers((top + 1) // 2, top + 1, rows)
    per = 32 if fmt in LEG or fmt == "q8_0" else 256
    shape = (rows, cols // per) if per == 32 else rows * cols // per
    d = 0.5 if fmt == "fp8" else 2.0 ** rng.integers(-6, -2, shape)
    if any_scale:
        d = rng.choice([-1.0, 1.0], shape) * 2.0 ** rng.integers(-24, 16, shape)
    sc = 1
    if fmt == "q4k":
        sc = rng.integers(1, 16, (rows * cols // 256, 8))
    elif fmt == "q6k":
        sc = 2 ** rng.integers(0, 7, (rows * cols // 256, 16))  # (q has 5 bits)
    f = fields(fmt, rows, cols, q, d, sc)
    w = values(fmt, f, rows, cols)
    assert (np.count_nonzero(w, 1) == 1).all()
    return f, w[np.arange(rows), pos]


def one_hot_layer(fmt, fmt_down, E, F, K, seed, any_scale=False, first=0):
    """The layer's (fields, column per row, value per row) of gate, up and down;
    gate and up leave the columns before `first` zero."""
    rng = np.random.default_rng(seed)
    gp, up = rng.integers(first, K, (E, F)), rng.integers(first, K, (E, F))
    dp = np.stack([(rng.permutation(max(F, K)) % F)[:K] for _ in range(E)])  # every column where K >= F
    out = []
    for i, (f, rows, cols, pos) in enumerate(((fmt, E * F, K, gp), (fmt, E * F, K, up), (fmt_down, E * K, F, dp))):
        fl, v = one_hot(f, seed + i, rows, cols, pos.reshape(-1), any_scale)
        out.append((fl, pos, v.reshape(pos.shape)))
    return out


def one_hot_h(layer, x, ids):
    """H [T][k][F] in 64 bits (relu)."""
    (_, gp, gv), (_, up, uv), _ = layer
    T, k = ids.shape
    t = np.arange(T)[:, None, None]
    return np.maximum(x[t, gp[ids]] * gv[ids], 0) * (x[t, up[ids]] * uv[ids])


def one_hot_terms(layer, h, ids, w):
    """The outputs' terms [T][k][K] for values h between the products."""
    _, _, (_, dp, dv) = layer
    T, k = ids.shape
    return w[:, :, None] * dv[ids] * np.take_along_axis(h, dp[ids], 2)


def one_hot_inputs(seed, T, E, K, k):
    rng = np.random.default_rng(seed)
    x = synth.bf16_bits_from_f32(np.exp(rng.uniform(-2, 2, (T, K))).astype(np.float32))
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    return x, ids, rng.uniform(0.5, 1, (T, k)).astype(np.float32)


def one_hot_bar(layer, form, h, ids, w):
    y = one_hot_terms(layer, h, ids, w)
    return y.sum(1), (np.abs(one_hot_terms(layer, h_error(form, h), ids, w)) + 9 * U * np.abs(y)).sum(1)


ONE_HOT = [
    # fmt, fmt_down, E, F, K, k, T
    *[(f, f, 3, 512, 512, 2, T) for f in TUNED for T in (1, 3, 40)],
    *[(f, f, 3, 256, 512, 2, T) for f in ("q2k", "q3k", "q5k", "fp8") + LEG for T in (3, 24)],
    ("q4k", "q6k", 30, 256, 256, 2, 30),     # two pairs an expert
    ("q4k", "q8_0", 3, 352, 512, 2, 50),     # rows that end inside a slab
    ("q8_0", "q8_0", 3, 352, 1056, 3, 70),
    ("q4k", "q6k", 4, 4096, 1024, 2, 17),    # tiles of 16 pairs
    ("q6k", "q4k", 4, 4096, 1024, 2, 9),
    ("q8_0", "q8_0", 2, 4128, 288, 2, 12),
    ("q4k", "q5k", 3, 256, 512, 2, 24),      # a tuned format beside another one
    ("q5_1", "q8_0", 3, 256, 512, 2, 3),
]


def run_one_hot(fmt, fmt_down, E, F, K, k, T, any_scale=False):
    layer = one_hot_layer(fmt, fmt_down, E, F, K, 61000 + F + T, any_scale)
    x, ids, w = one_hot_inputs(61100 + T, T, E, K, k)
    h = one_hot_h(layer, synth.bf16_bits_to_f32(x).astype(np.float64), ids)
    form = form_of(fmt, fmt_down, T, E, k, F, K)
    y, bar = one_hot_bar(layer, form, h, ids, w.astype(np.float64))
    dev = [pack(f, fl[0], E * n, c) for f, fl, n, c in zip((fmt, fmt, fmt_down), layer, (F, F, K), (K, K, F))]
    got = ql.qmatmul_moe(fmt, *dev, to_dev_bf16(x), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), E, F,
                         act="relu", fmt_down=fmt_down).cpu().numpy().astype(np.float64)
    err = np.abs(got - y)
    assert (err <= bar).all(), f"{form}: {np.max((err / bar)[bar > 0]):.2f} of the bar, largest error {err.max():.2e}"


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,fmt_down,E,F,K,k,T", ONE_HOT)
def test_h_holds_its_bits(fmt, fmt_down, E, F, K, k, T):
    run_one_hot(fmt, fmt_down, E, F, K, k, T)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,fmt_down,E,F,K,k,T", [c for c in ONE_HOT if c[0] in TUNED and c[1] in TUNED])
def test_scales_of_any_size_and_sign(fmt, fmt_down, E, F, K, k, T):
    """Scales from the smallest fp16 to the largest powers of two, of either
    sign, side by side in a row.  (Powers of two: a change of units is exact.)"""
    run_one_hot(fmt, fmt_down, E, F, K, k, T, any_scale=True)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,fmt_down,E,F,K,k,T", [
    ("q4k", "q4k", 3, 512, 512, 2, 3), ("q8_0", "q8_0", 3, 512, 512, 2, 40), ("q4k", "q6k", 3, 512, 512, 2, 40),
    ("q6k", "q4k", 4, 4096, 512, 2, 17), ("q5k", "q5k", 3, 256, 512, 2, 24), ("q8_0", "q4_0", 3, 256, 512, 2, 24)])
@pytest.mark.parametrize("below", (20, 31, 33, 36, 45))
def test_largest_values_of_x_that_meet_zeros(fmt, fmt_down, E, F, K, k, T, below):
    """A token whose largest values, 2^below times the others, meet weights of 0:
    exact but for the fp16 form, and there down to 2^-31 of the largest; below
    it within 2^-39 of the largest.  That keeps the accuracy of the header: 1e-3
    where x counts as at least 2^-29 of the largest."""
    layer = one_hot_layer(fmt, fmt_down, E, F, K, 64000 + F, first=8)
    x, ids, w = one_hot_inputs(64100 + T, T, E, K, k)
    v = np.random.default_rng(64200).uniform(1, 2, (T, K))
    v[:, :8] = 2.0 ** below
    x = synth.bf16_bits_from_f32((v * 0.25).astype(np.float32))
    v = synth.bf16_bits_to_f32(x).astype(np.float64)
    form = form_of(fmt, fmt_down, T, E, k, F, K)
    h = one_hot_h(layer, v, ids)
    big = v[:, 0].max()
    ex = 2.0 ** -39 * big if form == "fp16" and below > 31 else 0.0
    t = np.arange(T)[:, None, None]
    (_, gp, gv), (_, up, uv), _ = layer
    eh = gv[ids] * uv[ids] * (ex * v[t, gp[ids]] + ex * v[t, up[ids]] + ex * ex)
    y, bar = one_hot_bar(layer, form, h, ids, w.astype(np.float64))
    bar = bar + one_hot_terms(layer, eh * (1 + 2.0 ** -20) + h_error(form, eh), ids, w.astype(np.float64)).sum(1)
    counted = np.maximum(v, 2.0 ** -29 * big) if form == "fp16" else v
    said = 1e-3 * one_hot_terms(layer, one_hot_h(layer, counted, ids), ids, w.astype(np.float64)).sum(1)
    dev = [pack(f, fl[0], E * n, c) for f, fl, n, c in zip((fmt, fmt, fmt_down), layer, (F, F, K), (K, K, F))]
    got = ql.qmatmul_moe(fmt, *dev, to_dev_bf16(x), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), E, F,
                         act="relu", fmt_down=fmt_down).cpu().numpy().astype(np.float64)
    err = np.abs(got - y)
    assert (err <= bar).all(), f"{form}: {np.max(err / bar):.2f} of the bar"
    assert (bar <= said).all()


def device_one_hot(rows, cols, pos, seed):
    """A [rows][cols] Q8_0 weight on the device, zero but for column pos[n] of
    row n, as (block buffer, value per row): codes 64 to 127, scales of 2^-6."""
    n = rows * cols
    buf = torch.zeros(n + n // 16, dtype=torch.uint8, device="cuda")
    code = torch.randint(64, 128, (rows,), device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
    at = torch.arange(rows, device="cuda") * cols + pos
    buf[at] = code.to(torch.uint8)
    assert torch.equal(buf[at].long(), code)
    buf[n:].view(torch.float16).fill_(2.0 ** -6)
    return buf, code.double() * 2.0 ** -6


@pytest.mark.gpu
@pytest.mark.parametrize("F,K,T", [
    (32768 - 32, 65536, 5), (32768, 65536, 5),      # F * K: the last below 2^31 and 2^31, tiles of 16 pairs
    (32768 - 32, 65536, 24), (32768, 65536, 24),    # the same, tiles of 64
    (65536, 32768 - 32, 24), (65536, 32768, 24),
    (32, 65536, 32767), (32, 65536, 32768),         # T * K
])
def test_sizes_on_both_sides_of_the_fp16_form(F, K, T):
    """The largest sizes whose offsets are 32 bits, and the first past them,
    where H is held in bf16 pairs: each within the bar of its form."""
    g = torch.Generator("cuda").manual_seed(65000 + T)
    pos = [torch.randint(0, c, (r,), device="cuda", generator=g) for r, c in ((F, K), (F, K), (K, F))]
    for p, c in zip(pos, (K, K, F)):
        p[-1], p[0] = c - 1, 0   # the last value of the last row
    (gate, gv), (up, uv), (down, dv) = (device_one_hot(r, c, p, 65100 + i) for i, (r, c, p) in enumerate(zip((F, F, K), (K, K, F), pos)))
    x = torch.empty((T, K), dtype=torch.bfloat16, device="cuda").uniform_(0.5, 2.0, generator=g)
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    w = torch.ones((T, 1), device="cuda")
    form = form_of("q8_0", "q8_0", T, 1, 1, F, K)
    assert form == ("fp16" if F * K < 2 ** 31 and T * K < 2 ** 31 else "bf16")
    got = ql.qmatmul_moe("q8_0", gate, up, down, x, ids, w, 1, F, act="relu")
    rel = 2.0 ** -23 if form == "fp16" else 2.0 ** -17
    for a in range(0, T, 2048):
        xa = x[a:a + 2048].double()
        h = (xa[:, pos[0]] * gv) * (xa[:, pos[1]] * uv)
        bar = rel * h + 2.0 ** -39 * h.amax(1, keepdim=True)
        for c in range(0, K, 8192):
            p, d = pos[2][c:c + 8192], dv[c:c + 8192]
            y = h[:, p] * d
            err = (got[a:a + 2048, c:c + 8192].double() - y).abs()
            assert (err <= bar[:, p] * d + 9 * U * y).all(), (form, a, c)


def round_bits(a, bits):
    m, e = np.frexp(a)
    return np.ldexp(np.rint(m * 2.0 ** bits), e - bits)


def digits(h, lost=0):
    """H in whole numbers of 2^-e per chunk of 32, without its `lost` lowest
    base-256 digits."""
    c = h.reshape(*h.shape[:-1], -1, 32)
    m = np.abs(c).max(-1, keepdims=True)
    e = 23 - np.frexp(m)[1]
    e = e - (np.ldexp(m, e) > 8355711)
    v = np.rint(np.ldexp(c, e)).astype(np.int64)
    out = np.zeros_like(v)
    for i in range(3):
        d = ((v + 128) & 255) - 128
        v = (v - d) >> 8
        out += (d << (8 * i)) * (i >= lost)
    return np.ldexp(out.astype(np.float64), -e).reshape(h.shape)


@pytest.mark.parametrize("form,good,bad", [
    ("digits", lambda h: digits(h), (lambda h: digits(h, 1), lambda h: digits(h, 2), lambda h: round_bits(h, 16), lambda h: round_bits(h, 11))),
    ("fp16", lambda h: round_bits(h, 11) + round_bits(h - round_bits(h, 11), 11),
     (lambda h: round_bits(h, 11), lambda h: round_bits(h, 16), lambda h: round_bits(h, 20),
      lambda h: round_bits(h, 11) + np.roll(round_bits(h - round_bits(h, 11), 11), 1, -1))),
    ("bf16", lambda h: round_bits(h, 8) + round_bits(h - round_bits(h, 8), 8), (lambda h: round_bits(h, 8), lambda h: round_bits(h, 14))),
])
def test_the_bar_sees_a_lost_part_of_h(form, good, bad):
    """On the CPU: H rounded as its form says passes the bar; without its low
    plane, with that plane one place off, without a digit, or held in 16 bits,
    it does not."""
    layer = one_hot_layer("q8_0", "q8_0", 3, 512, 512, 62000)
    x, ids, w = one_hot_inputs(62100, 9, 3, 512, 2)
    h = one_hot_h(layer, synth.bf16_bits_to_f32(x).astype(np.float64), ids)
    y, bar = one_hot_bar(layer, form, h, ids, w.astype(np.float64))

    def passes(v):
        return (np.abs(one_hot_terms(layer, v, ids, w.astype(np.float64)).sum(1) - y) <= bar).all()

    assert passes(good(h))
    for b in bad:
        assert not passes(b(h))


# ----------------------------------------------------------------------------
# whole numbers
# ----------------------------------------------------------------------------

def whole(fmt, seed, rows, cols, zeros=0.0):
    """A dense weight of small whole numbers times powers of two, as (fields,
    values, magnitudes its sums meet: |scale * code| + |minimum|).  zeros: the
    part of scales d that are 0 under sub-scales and codes that are not."""
    rng = np.random.default_rng(seed)
    lo, hi = {"q8_0": (-3, 3), "q4k": (0, 3), "q6k": (-3, 3), "q5k": (0, 3), "q3k": (-3, 3), "q2k": (0, 3), "q4_0": (-3, 3), "q4_1": (0, 3),
              "q5_0": (-3, 3), "q5_1": (0, 3), "fp8": (-3, 3)}[fmt]
    q = rng.integers(lo, hi + 1, (rows, cols))
    G = rows * cols // 256
    shape = (rows, cols // 32) if fmt in LEG or fmt == "q8_0" else (G,)
    d = 1.0 if fmt == "fp8" else 2.0 ** rng.integers(-1, 1, shape) * (rng.random(shape) >= zeros)
    m = -(2.0 ** rng.integers(-1, 1, shape)) if fmt in ("q4_1", "q5_1") else 0
    sc = rng.integers(-2, 3, (G, 16)) if fmt == "q6k" else rng.integers(0, 3, (G, 8 if fmt == "q4k" else 16)) if fmt not in LEG + ("q8_0", "fp8") else 1
    mins = fmt in ("q4k", "q5k", "q2k")
    dmin = 2.0 ** rng.integers(-1, 1, (G,)) if mins else 0
    f = fields(fmt, rows, cols, q, d, sc, dmin, rng.integers(0, 4, np.shape(sc)) if mins else 0, m)
    w = values(fmt, f, rows, cols)
    if fmt == "fp8":
        return f, w, np.abs(w)
    if fmt in LEG or fmt == "q8_0":
        mag = np.abs(np.repeat(d, 32, 1) * q) + (np.repeat(np.abs(m), 32, 1) if np.ndim(m) else 0)
    else:
        # (Q6K's sub-scale goes in two parts, its multiple of 16 and the rest)
        s = f["sc"][:, :8] if fmt == "q5k" else f["sc"].astype(np.int64)
        if fmt == "q6k":
            s = np.abs(s & ~15) + (s & 15)
        s = np.repeat(s, 256 // s.shape[1], 1)
        dd = np.repeat(d, 256).reshape(G, 256)
        mag = np.abs(dd * s * q.reshape(G, 256))
        if mins:
            n = 8 if fmt != "q2k" else 16
            mag = mag + np.repeat(np.asarray(dmin)[:, None] * f["mq"][:, :n], 256 // n, 1)
        mag = mag.reshape(rows, cols)
    return f, w, mag


WHOLE = [
    *[(f, f, 3, 512, 768, 2, T) for f in TUNED for T in (1, 4, 70)],
    *[(f, f, 3, 256, 512, 2, T) for f in ("q2k", "q3k", "q5k", "fp8") + LEG for T in (3, 24, 60)],
    ("q4k", "q6k", 30, 256, 256, 2, 30),
    ("q4k", "q6k", 3, 1280, 512, 2, 30),
    ("q8_0", "q8_0", 3, 352, 1056, 3, 70),
    ("q8_0", "q8_0", 3, 1376, 288, 2, 40),
    ("q4k", "q4k", 3, 4096, 512, 2, 12),
    ("q6k", "q6k", 3, 4096, 512, 2, 12),
    ("q8_0", "q8_0", 2, 4128, 288, 2, 12),
    ("q4k", "q5k", 3, 256, 512, 2, 24),
]


def whole_case(fmt, fmt_down, E, F, K, k, T, zeros=0.0):
    """Weights (fields), X, ids, weights and the outputs, exact in 64 bits."""
    rng = np.random.default_rng(63000 + F + T)
    W = [whole(f, 63100 + i, E * n, c, zeros) for i, (f, n, c) in enumerate(((fmt, F, K), (fmt, F, K), (fmt_down, K, F)))]
    x = np.zeros((T, K))
    for t in range(T):  # two values of +-1 a token
        x[t, rng.choice(K, 2, replace=False)] = rng.choice([-1.0, 1.0], 2)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    w = (2.0 ** rng.integers(-1, 1, (T, k))).astype(np.float32)
    g3 = [v.reshape(E, -1, v.shape[1]) for _, v, _ in W]
    m3 = [v.reshape(E, -1, v.shape[1]) for _, _, v in W]
    y = np.zeros((T, K))
    lsb = 2.0 ** -2 * 2.0 ** -1 * 2.0 ** -1  # of h, of a weight, of a choice's weight
    for t in range(T):
        mag = np.zeros(K)
        for j in range(k):
            e = ids[t, j]
            h = np.maximum(g3[0][e] @ x[t], 0) * (g3[1][e] @ x[t])
            y[t] += w[t, j] * (g3[2][e] @ h)
            mag += w[t, j] * (m3[2][e] @ np.abs(h))
        assert mag.max() < 2.0 ** 24 * lsb, "a partial sum may need more than 24 bits"
    return W, synth.bf16_bits_from_f32(x.astype(np.float32)), ids, w, y


def run_whole(fmt, fmt_down, E, F, K, k, T, zeros=0.0):
    W, x, ids, w, y = whole_case(fmt, fmt_down, E, F, K, k, T, zeros)
    dev = [pack(f, v[0], E * n, c) for f, v, n, c in zip((fmt, fmt, fmt_down), W, (F, F, K), (K, K, F))]
    got = ql.qmatmul_moe(fmt, *dev, to_dev_bf16(x), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), E, F,
                         act="relu", fmt_down=fmt_down).cpu().numpy()
    assert np.count_nonzero(y) > y.size // 4
    bad = got != y
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outputs off, by up to {np.abs(got - y).max():.3e}"


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,fmt_down,E,F,K,k,T", WHOLE)
def test_whole_numbers_are_exact(fmt, fmt_down, E, F, K, k, T):
    run_whole(fmt, fmt_down, E, F, K, k, T)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,fmt_down,E,F,K,k,T", [c for c in WHOLE if "fp8" not in c])
def test_scales_of_zero_above_codes_that_are_not(fmt, fmt_down, E, F, K, k, T):
    """A block whose scale is 0 is its minimum alone, whatever its sub-scales
    and codes hold (isq_quantize writes zeros there, other writers of a block
    buffer need not), in every form: half of the scales are 0."""
    run_whole(fmt, fmt_down, E, F, K, k, T, zeros=0.5)


def test_whole_number_cases_fit():
    """On the CPU: the largest cases' partial sums fit 24 bits (asserted inside)
    and their outputs are not mostly zero."""
    for c in (("q4k", "q4k", 3, 4096, 512, 2, 12), ("q6k", "q6k", 3, 4096, 512, 2, 12), ("q8_0", "q8_0", 2, 4128, 288, 2, 12),
              ("q5_1", "q5_1", 3, 256, 512, 2, 60), ("q2k", "q2k", 3, 256, 512, 2, 60)):
        y = whole_case(*c)[4]
        assert np.count_nonzero(y) > y.size // 4
