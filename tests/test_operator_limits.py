"""The mixture-of-experts and log-probability calls at the largest counts they
accept: tokens, experts, choices, rows, logits."""
import numpy as np
import pytest
import torch

import ggml_block_quant_amd as ql
import synth
from gpu_util import to_dev_bf16
from test_moe_precision import pack, whole
from test_parity_logprobs import U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k", ((65536, 3, 2), (65535, 1, 1), (60, 1024, 32), (70, 1024, 32), (4, 1024, 32), (5, 1, 32)))
def test_moe_most_tokens_experts_and_choices(T, E, k):
    """Whole numbers whose sums fit 24 bits: equal outputs."""
    F, K = 32, 32
    W = [whole("q8_0", 67000 + i, E * n, c) for i, (n, c) in enumerate(((F, K), (F, K), (K, F)))]
    g, u, d = (v.reshape(E, -1, v.shape[1]) for _, v, _ in W)
    rng = np.random.default_rng(67010 + T)
    x = np.zeros((T, K))
    for _ in range(2):
        x[np.arange(T), rng.integers(0, K, T)] = rng.choice([-1.0, 1.0], T)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    w = (2.0 ** rng.integers(-1, 1, (T, k))).astype(np.float32)
    y = np.zeros((T, K))
    for j in range(k):
        for e in range(E):
            t = np.flatnonzero(ids[:, j] == e)
            h = np.maximum(x[t] @ g[e].T, 0) * (x[t] @ u[e].T)
            y[t] += w[t, j, None] * (h @ d[e].T)
    got = ql.qmatmul_moe("q8_0", *(pack("q8_0", f, E * n, c) for (f, _, _), n, c in zip(W, (F, F, K), (K, K, F))),
                         to_dev_bf16(synth.bf16_bits_from_f32(x.astype(np.float32))), torch.from_numpy(ids).cuda(),
                         torch.from_numpy(w).cuda(), E, F, act="relu")
    assert np.array_equal(got.cpu().numpy(), y.astype(np.float32))


def test_route_most_tokens():
    T, E, k = 65536, 9, 4
    x = np.random.default_rng(67100).standard_normal((T, E)).astype(np.float32)
    ids, w = ql.moe_route(torch.from_numpy(x).cuda(), k)
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    assert np.array_equal(ids.cpu().numpy(), order)
    p = np.exp(np.take_along_axis(x, order, 1).astype(np.float64))
    assert np.abs(w.cpu().numpy() - p / p.sum(1, keepdims=True)).max() <= 100 * U


@pytest.mark.parametrize("M,V,top", ((65536, 50, 3), (32769, 777, 0), (40001, 4100, 20), (1, 1 << 24, 64), (2, (1 << 24) - 3, 5), (4095, 131072, 1)))
def test_logprobs_most_rows_and_logits(M, V, top):
    """Against 64 bits on the device (chunks of rows); ids by a stable sort of a
    few rows."""
    gen = torch.Generator("cuda").manual_seed(V)
    x = torch.randn((M, V), device="cuda", generator=gen) * 3
    t = torch.randint(0, V, (M,), device="cuda", generator=gen, dtype=torch.int32)
    got = ql.logprobs(x, t, top)
    # the terms of one thread (of 256, in one part or more), as in the parity tests
    part = (2 * 32 + 4 + V / 256 + 16 + 20 + 3 * np.log(V + 1)) * U
    step = max(1, (1 << 26) // V)
    for a in range(0, M, step):
        xa = x[a:a + step].double()
        lse = torch.logsumexp(xa, 1)
        xt = xa.gather(1, t[a:a + step, None].long())
        lp = xt[:, 0] - lse
        assert ((got.logprob[a:a + step].double() - lp).abs() <= part + 3 * U * lp.abs()).all()
        assert torch.equal(got.rank[a:a + step].long(), (xa > xt).sum(1) + 1)
        p = torch.exp(xa - lse[:, None])
        ent = -(p * (xa - lse[:, None])).sum(1)
        assert ((got.entropy[a:a + step].double() - ent).abs() <= part * min(32, np.log(V) + 1) + 3 * U * ent).all()
    for m in {0, M // 2, M - 1}:
        order = torch.sort(x[m].cpu(), descending=True, stable=True).indices[:top]
        if top:
            assert torch.equal(got.top_ids[m].cpu().long(), order)
