"""Measured cases of the operators behind a decoder's quantized linear layers:
the mixture-of-experts layer on block-quantized weights (the router's choice
and the experts' gated products) and the output head's log probabilities (of
given logits, and fused behind the quantized head).

`run` computes a pass either in its plain form (elementary torch operations in
32 bits) or, where `own` is true, through this repository's package.
"""
import math

import torch

own = False

# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one token of a decode loop through a many-expert router: latency
        dict(name="route one token", op="route", T=1, E=128, k=8, score="softmax", bias=False, masked=0),
        # a prefill chunk through a sigmoid router whose load-balancing bias
        # takes part in the choice only; some experts are switched off
        dict(name="route prefill", op="route", T=4096, E=256, k=8, score="sigmoid", bias=True, masked=5),
        # single-token decode with few wide experts (the decoder's own
        # feed-forward shape 14336 x 4096 as eight experts)
        dict(name="moe decode wide q4k", op="moe", T=1, E=8, k=2, K=4096, F=14336, fmt="q4k", fmt_down="q4k",
             act="silu", pad=0),
        # single-token decode with many narrow experts
        dict(name="moe decode narrow q8_0", op="moe", T=1, E=128, k=8, K=2048, F=768, fmt="q8_0", fmt_down="q8_0",
             act="silu", pad=0),
        # a continuous batch of odd size, padded to its captured size by rows
        # that choose no expert; the down weights in the promoted format
        dict(name="moe batch q4k q6k", op="moe", T=24, E=8, k=2, K=4096, F=14336, fmt="q4k", fmt_down="q6k",
             act="silu", pad=3),
        # a ragged prompt through narrow experts whose width is no multiple
        # of 256 (whole Q8_0 blocks only)
        dict(name="moe prompt q8_0", op="moe", T=515, E=64, k=6, K=2048, F=1408, fmt="q8_0", fmt_down="q8_0",
             act="silu", pad=0),
        # a long prompt through the wide experts: matrix-core work
        dict(name="moe prompt q4k", op="moe", T=2048, E=8, k=2, K=4096, F=14336, fmt="q4k", fmt_down="q4k",
             act="silu", pad=0),
        # one decode step's answer with its top alternatives
        dict(name="logprobs one row", op="logprobs", M=1, V=131072, top=5, kind="fp32"),
        # a batch under a grammar's mask (most tokens -inf, one row with
        # nothing left), logits that carry bf16 roundings and hence ties, an
        # odd vocabulary
        dict(name="logprobs masked odd", op="logprobs", M=49, V=32003, top=20, kind="masked"),
        # scoring a prompt: every row's given token, and alternatives
        dict(name="logprobs prompt", op="logprobs", M=2048, V=131072, top=8, kind="fp32"),
        # the decoder's promoted Q6K output head, one token
        dict(name="head one token q6k", op="head", M=1, N=131072, K=5120, fmt="q6k"),
        # scoring a ragged prompt through a Q4K head without holding its logits
        dict(name="head prompt q4k", op="head", M=600, N=32000, K=4096, fmt="q4k"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "moe", "logprobs", "head"])
    if op == "route":
        E = rng.choice([_log_int(rng, 8, 64), _log_int(rng, 64, 512)])
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, T=_log_int(rng, 1, 4096 * 256 // E if E > 256 else 4096), E=E,
                    k=rng.randint(2, min(8, E)), score=score, bias=score == "sigmoid" and rng.random() < 0.5,
                    masked=rng.choice([0, 0, rng.randint(1, E // 2)]))
    if op == "moe":
        fmt, fmt_down = rng.choice([("q4k", "q4k"), ("q4k", "q6k"), ("q6k", "q6k"), ("q8_0", "q8_0")])
        T, E = _log_int(rng, 1, 2048), _log_int(rng, 4, 128)
        k = rng.randint(1, min(8, E))
        K = 256 * rng.randint(4, 24)
        F = 32 * _log_int(rng, 16, 448) if fmt == "q8_0" else 256 * _log_int(rng, 2, 56)
        while 3 * E * F * K > 8 * 3 * 14336 * 4096:
            E = max(4, E // 2) if E > 4 else E
            F = F if E > 4 else (F // 512) * 256
        k = min(k, E)
        while T * k * F * K > 2048 * 2 * 14336 * 4096:
            T = T // 2
        return dict(op=op, T=T, E=E, k=k, K=K, F=F, fmt=fmt, fmt_down=fmt_down, act=rng.choice(["silu", "relu"]),
                    pad=rng.choice([0, T // 5]))
    if op == "logprobs":
        M, V = _log_int(rng, 1, 2048), _log_int(rng, 1000, 131072)
        return dict(op=op, M=M, V=V, top=rng.randint(0, 20), kind=rng.choice(["fp32", "bf16", "masked"]))
    fmt = rng.choice(["q4k", "q6k", "q8_0"])
    M, N, K = _log_int(rng, 1, 600), _log_int(rng, 8000, 131072), 256 * rng.randint(4, 20)
    while M * N * K > 600 * 131072 * 4096:
        M = M // 2
    return dict(op=op, M=M, N=N, K=K, fmt=fmt)


_BITS = {"q8_0": 8.5, "q4k": 4.5, "q6k": 6.5625}


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 4 * T * E}
    if op == "moe":
        T, E, k, K, F = (case[n] for n in ("T", "E", "k", "K", "F"))
        live = T - case["pad"]
        active = E * (1 - (1 - k / E) ** live)  # experts expected to be chosen
        weights = active * F * K * (2 * _BITS[case["fmt"]] + _BITS[case["fmt_down"]]) / 8
        return {"bytes": weights + 2 * T * K + 8 * T * k + 4 * T * K, "flops": 6 * live * k * F * K}
    if op == "logprobs":
        M, V, n = case["M"], case["V"], case["top"]
        return {"bytes": 4 * M * V + 16 * M + 8 * M * n, "flops": 6 * M * V}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": N * K * _BITS[case["fmt"]] / 8 + 2 * M * K + 12 * M, "flops": 2 * M * N * K + 6 * M * N}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _bell(n, lo, hi, g):
    """n whole numbers of a triangular distribution over 0 .. lo + hi, uint8."""
    a = torch.randint(0, lo + 1, (n,), dtype=torch.uint8, device="cuda", generator=g)
    return a + torch.randint(0, hi + 1, (n,), dtype=torch.uint8, device="cuda", generator=g)


def _blocks(fmt, rows, K, g):
    """The block buffer of a [rows][K] weight of standard deviation near 0.02:
    bell-shaped codes and scales that vary from block to block."""
    n = rows * K
    G = n // 256

    def uni(count, lo, hi):
        return torch.rand(count, device="cuda", generator=g) * (hi - lo) + lo

    if fmt == "q8_0":
        out = torch.empty(n + n // 16, dtype=torch.uint8, device="cuda")
        q = torch.randn(n, device="cuda", generator=g, dtype=torch.float16).mul_(40).round_().clamp_(-127, 127)
        out[:n] = q.to(torch.int8).view(torch.uint8)
        out[n:] = uni(n // 32, 3.75e-4, 6.25e-4).half().view(torch.uint8)
        return out
    if fmt == "q4k":
        out = torch.empty(144 * G, dtype=torch.uint8, device="cuda")
        out[:128 * G] = _bell(128 * G, 7, 8, g) | (_bell(128 * G, 7, 8, g) << 4)
        sc = torch.randint(32, 64, (G, 8), device="cuda", generator=g)
        m = (sc + torch.randint(-4, 5, (G, 8), device="cuda", generator=g)).clamp_(0, 63)
        d = uni(G, 0.9e-4, 1.5e-4)
        at4, at2 = 4 * torch.arange(8, device="cuda"), 2 * torch.arange(8, device="cuda")
        words = torch.stack([((sc & 15) << at4).sum(1), ((m & 15) << at4).sum(1),
                             ((sc >> 4) << at2).sum(1) | (((m >> 4) << at2).sum(1) << 16)], 1)
        words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
        head = out[128 * G:].view(torch.int32).view(G, 4)
        head[:, 0] = torch.stack([d, 7.5 * d], 1).half().view(torch.int32).view(G)
        head[:, 1:] = words
        return out
    out = torch.zeros((210 * G + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
    codes = out[:192 * G].view(G, 192)
    codes[:, :128] = torch.randint(0, 256, (G, 128), dtype=torch.uint8, device="cuda", generator=g)
    hi = _bell(64 * G, 1, 2, g) | (_bell(64 * G, 1, 2, g) << 2) | (_bell(64 * G, 1, 2, g) << 4) | (_bell(64 * G, 1, 2, g) << 6)
    codes[:, 128:] = hi.view(G, 64)
    sign = 1 - 2 * torch.randint(0, 2, (16 * G,), device="cuda", generator=g)
    out[192 * G:208 * G] = (sign * torch.randint(64, 128, (16 * G,), device="cuda", generator=g)).to(torch.int8).view(torch.uint8)
    out[208 * G:210 * G] = uni(G, 1.2e-5, 2e-5).half().view(torch.uint8)
    return out


def _activations(T, K, g):
    """Normed hidden states: unit variance, channels of their own gain, a few
    of them large."""
    gain = torch.exp(0.3 * torch.randn(K, device="cuda", generator=g))
    gain = torch.where(torch.rand(K, device="cuda", generator=g) < 0.003, 8 * gain, gain)
    return (torch.randn(T, K, device="cuda", generator=g) * gain).bfloat16()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "route":
        T, E = case["T"], case["E"]
        x = 1.5 * torch.randn(T, E, device="cuda", generator=g) + 0.5 * torch.randn(E, device="cuda", generator=g)
        if case["masked"]:
            off = torch.randperm(E, device="cuda", generator=g)[:case["masked"]]
            x[:, off] = -math.inf
        s["logits"] = x
        s["bias_"] = 0.1 * torch.randn(E, device="cuda", generator=g) if case["bias"] else None
        return s
    if op == "moe":
        T, E, k, K, F = (case[n] for n in ("T", "E", "k", "K", "F"))
        s["gate"] = _blocks(case["fmt"], E * F, K, g)
        s["up"] = _blocks(case["fmt"], E * F, K, g)
        s["down"] = _blocks(case["fmt_down"], E * K, F, g)
        s["x"] = _activations(T, K, g)
        score = torch.randn(T, E, device="cuda", generator=g) + 0.3 * torch.randn(E, device="cuda", generator=g)
        v, i = torch.softmax(score, 1).topk(k, 1)
        ids, w = i.to(torch.int32), v / v.sum(1, keepdim=True)
        if case["pad"]:
            ids[T - case["pad"]:] = -1
            w[T - case["pad"]:] = 0
        s["ids"], s["w"] = ids.contiguous(), w.contiguous()
        return s
    if op == "logprobs":
        M, V, kind = case["M"], case["V"], case["kind"]
        x = 2.5 * torch.randn(M, V, device="cuda", generator=g)
        peak = torch.randint(0, V, (M, 3), device="cuda", generator=g)
        x.scatter_add_(1, peak, 8 + 3 * torch.randn(M, 3, device="cuda", generator=g))
        if kind != "fp32":
            x = x.bfloat16().float()
        if kind == "masked":
            share = torch.rand(M, 1, device="cuda", generator=g) ** 4
            x.masked_fill_(torch.rand(M, V, device="cuda", generator=g) > share, -math.inf)
            x[M // 2] = -math.inf
        t = torch.where(torch.rand(M, device="cuda", generator=g) < 0.5, peak[:, 0],
                        torch.randint(0, V, (M,), device="cuda", generator=g)).to(torch.int32)
        if M > 8:
            t[M - M // 8:] = -1  # rows of a prompt's padding, whose token is not scored
        s["x"], s["t"] = x, t
        return s
    M, N, K = case["M"], case["N"], case["K"]
    s["head"] = _blocks(case["fmt"], N, K, g)
    s["x"] = (1.5 * _activations(M, K, g)).bfloat16()
    s["t"] = torch.randint(0, N, (M,), device="cuda", generator=g, dtype=torch.int32)
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------


def _nibbles(dwords):
    """int32 dwords [..., D] -> their eight nibbles in element order (element
    2p at nibble p, element 2p + 1 at nibble p + 4) [..., D, 8]."""
    e = torch.arange(8, device=dwords.device, dtype=torch.int32)
    return (dwords.unsqueeze(-1) >> (4 * (e // 2) + 16 * (e % 2))) & 15


def _dequant(fmt, buf, parts, rows, K, which):
    """fp32 weights [len(which)][rows][K] of the chosen of `parts` stacked
    [rows][K] tensors."""
    n = parts * rows * K
    G = n // 256
    if fmt == "q8_0":
        q = buf[:n].view(torch.int8).view(parts, -1, 32)[which].float()
        d = buf[n:n + n // 16].view(torch.float16).view(parts, -1, 1)[which].float()
        return (q * d).view(-1, rows, K)
    if fmt == "q4k":
        q = _nibbles(buf[:128 * G].view(torch.int32).view(parts, -1, 32)[which]).float()
        h = buf[128 * G:144 * G].view(torch.int32).view(parts, -1, 4)[which]
        dd = buf[128 * G:144 * G].view(torch.float16).view(parts, -1, 8)[which].float()
        j = torch.arange(8, device=buf.device, dtype=torch.int32)
        sc = ((h[..., 1:2] >> (4 * j)) & 15) | (((h[..., 3:4] >> (2 * j)) & 3) << 4)
        m = ((h[..., 2:3] >> (4 * j)) & 15) | (((h[..., 3:4] >> (16 + 2 * j)) & 3) << 4)
        S, Mn = dd[..., 0:1] * sc, dd[..., 1:2] * m
        q = q.view(*S.shape, 32)
        return (q * S.unsqueeze(-1) - Mn.unsqueeze(-1)).view(-1, rows, K)
    codes = buf[:192 * G].view(torch.int32).view(parts, -1, 48)[which]
    lo = _nibbles(codes[..., :32])
    e = torch.arange(16, device=buf.device, dtype=torch.int32)
    hi = (codes[..., 32:].unsqueeze(-1) >> (8 * (e // 8) + 16 * (e % 2) + 2 * (e % 8 // 2))) & 3
    q = ((hi.view(lo.shape) << 4) | lo).float() - 32
    sc = buf[192 * G:208 * G].view(torch.int8).view(parts, -1, 16)[which].float()
    d = buf[208 * G:210 * G].view(torch.float16).view(parts, -1, 1)[which].float()
    S = d * sc
    return (q.view(*S.shape, 16) * S.unsqueeze(-1)).view(-1, rows, K)


def _plain_route(s):
    x, k = s["logits"], s["k"]
    x64 = x.double()
    p = torch.softmax(x64, 1) if s["score"] == "softmax" else torch.sigmoid(x64)
    p = torch.where(x == -math.inf, torch.zeros_like(p), p)
    key = x64 if s["bias_"] is None else torch.where(x == -math.inf, x64, p + s["bias_"].double())
    key, ids = torch.sort(key, dim=1, descending=True, stable=True)
    key, ids = key[:, :k], ids[:, :k]
    w = p.gather(1, ids)
    total = w.sum(1, keepdim=True)
    w = torch.where(total > 0, w / total, torch.zeros_like(w))
    ids = torch.where(key == -math.inf, torch.full_like(ids, -1), ids)
    return {"ids": ids.to(torch.int32), "weights": w.float()}


def _act(name, g):
    return g * torch.sigmoid(g) if name == "silu" else torch.clamp(g, min=0)


def _plain_moe(s):
    T, E, k, K, F = (s[n] for n in ("T", "E", "k", "K", "F"))
    flat = s["ids"].reshape(-1).long()
    pairs = torch.nonzero((flat >= 0) & (flat < E)).squeeze(1)
    y = torch.zeros(T * k, K, device="cuda")
    if pairs.numel():
        which, slot = torch.unique(flat[pairs], return_inverse=True)
        counts = torch.bincount(slot)
        order = torch.argsort(slot, stable=True)
        pairs, slot = pairs[order], slot[order]
        pos = torch.arange(pairs.numel(), device="cuda") - (torch.cumsum(counts, 0) - counts)[slot]
        x = torch.zeros(which.numel(), int(counts.max()), K, device="cuda")
        x[slot, pos] = s["x"][pairs // k].float()
        gate = torch.bmm(x, _dequant(s["fmt"], s["gate"], E, F, K, which).transpose(1, 2))
        up = torch.bmm(x, _dequant(s["fmt"], s["up"], E, F, K, which).transpose(1, 2))
        out = torch.bmm(_act(s["act"], gate) * up, _dequant(s["fmt_down"], s["down"], E, K, F, which).transpose(1, 2))
        y[pairs] = out[slot, pos] * s["w"].reshape(-1)[pairs].unsqueeze(1)
    return y.view(T, k, K).sum(1)


def _plain_logprobs(x, t, top):
    M, V = x.shape
    live = x > -math.inf
    m = x.amax(1, keepdim=True)
    m0 = torch.where(m > -math.inf, m, torch.zeros_like(m))
    e = torch.exp(x - m0)
    z = e.sum(1, keepdim=True)
    lse = torch.log(z) + m0
    given = (t >= 0) & (t < V)
    xt = x.gather(1, t.long().clamp(0, V - 1).unsqueeze(1))
    lp = torch.where(xt > -math.inf, xt - lse, xt).squeeze(1)
    rank = (x > xt).sum(1).to(torch.int32) + 1
    ent = (torch.log(z) - torch.where(live, e * (x - m0), torch.zeros_like(e)).sum(1, keepdim=True) / z).squeeze(1)
    out = {"logprob": torch.where(given, lp, torch.zeros_like(lp)),
           "rank": torch.where(given, rank, torch.zeros_like(rank)),
           "entropy": torch.where(m.squeeze(1) > -math.inf, ent, torch.zeros_like(ent))}
    if top:
        # whole-number keys: the value's order first, then the lower index
        b = (x + 0.0).view(torch.int32).long()
        key = torch.where(b >= 0, b, -(b & 0x7FFFFFFF)) * 2 ** 32 - torch.arange(V, device=x.device)
        i = key.topk(top, 1).indices
        v = x.gather(1, i)
        alive = v > -math.inf
        out["top_ids"] = torch.where(alive, i, torch.full_like(i, -1)).to(torch.int32)
        out["top_logprobs"] = torch.where(alive, v - lse, v)
    return out


def _plain_head(s):
    w = _dequant(s["fmt"], s["head"], 1, s["N"], s["K"], torch.zeros(1, dtype=torch.long, device="cuda"))[0]
    out = _plain_logprobs(s["x"].float() @ w.t(), s["t"], 0)
    return {"logprob": out["logprob"], "entropy": out["entropy"]}


# ---------------------------------------------------------------------------
# a pass
# ---------------------------------------------------------------------------


def run(state):
    s, op = state, state["op"]
    if own:
        import ggml_block_quant_amd as ql

        if op == "route":
            ids, w = ql.moe_route(s["logits"], s["k"], score=s["score"], bias=s["bias_"], renorm=True)
            return {"ids": ids, "weights": w}
        if op == "moe":
            if "ws" not in s:  # a serving loop keeps its workspace
                n = ql.moe_workspace_bytes(s["fmt"], s["fmt_down"], s["T"], s["E"], s["k"], s["F"], s["K"])
                s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
            return ql.qmatmul_moe(s["fmt"], s["gate"], s["up"], s["down"], s["x"], s["ids"], s["w"], s["E"], s["F"],
                                  act=s["act"], fmt_down=s["fmt_down"], workspace=s["ws"])
        if op == "logprobs":
            r = ql.logprobs(s["x"], s["t"], top=s["top"])
            out = {"logprob": r.logprob, "rank": r.rank, "entropy": r.entropy}
            if s["top"]:
                out["top_ids"], out["top_logprobs"] = r.top_ids, r.top_logprobs
            return out
        r = ql.qmatmul_logprobs(s["fmt"], s["head"], s["x"], s["N"], s["t"])
        return {"logprob": r.logprob, "entropy": r.entropy}
    if op == "route":
        return _plain_route(s)
    if op == "moe":
        return _plain_moe(s)
    if op == "logprobs":
        return _plain_logprobs(s["x"], s["t"], s["top"])
    return _plain_head(s)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------


def _weights64(fmt, buf, parts, rows, K, e):
    """Part e of `parts` stacked [rows][K] tensors in 64 bits, byte by byte."""
    n, G = parts * rows * K, parts * rows * K // 256
    per, gp = rows * K, rows * K // 256
    if fmt == "q8_0":
        q = buf[e * per:(e + 1) * per].view(torch.int8).double().view(-1, 32)
        d = buf[n:n + n // 16].view(torch.float16)[e * per // 32:(e + 1) * per // 32].double()
        return (q * d[:, None]).view(rows, K)
    order = [0, 2, 4, 6, 1, 3, 5, 7]  # the elements of a dword's nibbles from the lowest
    if fmt == "q4k":
        b = buf[128 * gp * e:128 * gp * (e + 1)].view(-1, 4)
        q = torch.empty(b.shape[0], 8, dtype=torch.float64, device="cuda")
        for i in range(8):
            q[:, order[i]] = ((b[:, i // 2] >> (4 * (i % 2))) & 15).double()
        h = buf[128 * G:].view(G, 16)[gp * e:gp * (e + 1)]
        dd = h[:, :4].contiguous().view(torch.float16).double()
        q = q.view(gp, 8, 32)
        for j in range(8):
            sc = ((h[:, 4 + j // 2] >> (4 * (j % 2))) & 15) | (((h[:, 12 + j // 4] >> (2 * (j % 4))) & 3) << 4)
            m = ((h[:, 8 + j // 2] >> (4 * (j % 2))) & 15) | (((h[:, 14 + j // 4] >> (2 * (j % 4))) & 3) << 4)
            q[:, j] = q[:, j] * (dd[:, 0] * sc.double())[:, None] - (dd[:, 1] * m.double())[:, None]
        return q.view(rows, K)
    c = buf[:192 * G].view(G, 192)[gp * e:gp * (e + 1)]
    lo, hi = c[:, :128].reshape(gp, 32, 4), c[:, 128:].reshape(gp, 8, 2, 4)
    q = torch.empty(gp, 32, 8, dtype=torch.float64, device="cuda")
    for i in range(8):
        q[:, :, order[i]] = ((lo[:, :, i // 2] >> (4 * (i % 2))) & 15).double()
    q = q.view(gp, 8, 2, 2, 8)  # chunk, dword, octet of the dword, element
    for o in range(2):
        for k in range(4):
            q[:, :, :, o, 2 * k] += 16 * ((hi[..., o] >> (2 * k)) & 3).double()
            q[:, :, :, o, 2 * k + 1] += 16 * ((hi[..., 2 + o] >> (2 * k)) & 3).double()
    sc = buf[192 * G:208 * G].view(torch.int8).view(G, 16)[gp * e:gp * (e + 1)].double()
    d = buf[208 * G:210 * G].view(torch.float16)[gp * e:gp * (e + 1)].double()
    return ((q - 32).view(gp, 16, 16) * (sc * d[:, None])[:, :, None]).view(rows, K)


def _logprobs64(x, t, top):
    M, V = x.shape
    lp, ent = torch.zeros(M, dtype=torch.float64, device="cuda"), torch.zeros(M, dtype=torch.float64, device="cuda")
    tops = torch.full((M, top), -math.inf, dtype=torch.float64, device="cuda")
    for a in range(0, M, 256):
        y = x[a:a + 256].double()
        lse = torch.logsumexp(y, 1)
        some = lse > -math.inf
        logp = torch.where(some[:, None], y - lse[:, None], torch.full_like(y, -math.inf))
        p = torch.exp(logp)
        ent[a:a + 256] = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
        u = t[a:a + 256].long()
        ok = (u >= 0) & (u < V)
        lp[a:a + 256] = torch.where(ok, logp[torch.arange(u.numel(), device="cuda"), u.clamp(0, V - 1)], torch.zeros_like(lse))
        if top:
            tops[a:a + 256] = logp.topk(top, 1).values
    return lp, ent, tops


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        x, k = s["logits"].double(), s["k"]
        p = torch.exp(x - torch.logsumexp(x, 1, keepdim=True)) if s["score"] == "softmax" else 1 / (1 + torch.exp(-x))
        p = torch.nan_to_num(p)
        key = x if s["bias_"] is None else torch.where(x > -math.inf, p + s["bias_"].double(), x)
        i = torch.argsort(-key, dim=1, stable=True)[:, :k]
        w = torch.gather(p, 1, i)
        z = w.sum(1, keepdim=True)
        return {"ids": None, "weights": torch.where(z > 0, w / z, torch.zeros_like(w))}
    if op == "moe":
        T, E, k, K, F = (case[n] for n in ("T", "E", "k", "K", "F"))
        y = torch.zeros(T, K, dtype=torch.float64, device="cuda")
        x, ids, w = s["x"].double(), s["ids"], s["w"].double()
        for e in range(E):
            rows, slots = torch.nonzero(ids == e, as_tuple=True)
            if rows.numel() == 0:
                continue
            g = x[rows] @ _weights64(case["fmt"], s["gate"], E, F, K, e).t()
            h = g / (1 + torch.exp(-g)) if case["act"] == "silu" else g * (g > 0)
            h = h * (x[rows] @ _weights64(case["fmt"], s["up"], E, F, K, e).t())
            y.index_add_(0, rows, w[rows, slots][:, None] * (h @ _weights64(case["fmt_down"], s["down"], E, K, F, e).t()))
        return y
    if op == "logprobs":
        lp, ent, tops = _logprobs64(s["x"], s["t"], case["top"])
        out = {"logprob": lp, "rank": None, "entropy": ent}
        if case["top"]:
            out["top_ids"], out["top_logprobs"] = None, tops
        return out
    logits = s["x"].double() @ _weights64(case["fmt"], s["head"], 1, case["N"], case["K"], 0).t()
    lp, ent, _ = _logprobs64(logits, s["t"], 0)
    return {"logprob": lp, "entropy": ent}
