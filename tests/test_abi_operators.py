"""Argument checks of the mixture-of-experts and log-probability calls: every
refusal happens before anything is launched, so no GPU is needed.  Pointers
are made-up aligned addresses that no refused call may touch."""
import ctypes

import pytest
import torch

import ggml_block_quant_amd as ql

P = 0x10000  # aligned, never read
OK, EINVAL, ESHAPE, EALIGN, ENOTSUP = ql.Q_OK, ql.Q_EINVAL, ql.Q_ESHAPE, ql.Q_EALIGN, ql.Q_ENOTSUP
BIG = 1 << 40


def route(**kw):
    a = dict(logits=P, T=4, E=16, k=2, score=0, bias=None, renorm=1, scale=1.0, ids=P, w=P)
    a.update(kw)
    return ql.lib().q_moe_route(*a.values(), None)


def moe(**kw):
    a = dict(fmt=1, g=P, u=P, fd=1, d=P, X=P, ids=P, w=P, Y=P, T=4, E=8, k=2, F=512, K=256, act=0, ws=P, wsb=BIG)
    a.update(kw)
    return ql.lib().qmatmul_moe(*a.values(), None)


def lp(**kw):
    a = dict(x=P, M=4, V=100, ld=100, t=P, n=2, lp=P, rank=P, ent=P, ids=P, tl=P, ws=P, wsb=BIG)
    a.update(kw)
    return ql.lib().q_logprobs(*a.values(), None)


def head(**kw):
    a = dict(fmt=1, B=P, X=P, M=4, N=100, K=256, t=P, n=2, lp=P, rank=P, ent=P, ids=P, tl=P, ws=P, wsb=BIG)
    a.update(kw)
    return ql.lib().qmatmul_logprobs(*a.values(), None)


def test_route_refusals():
    for n in ("logits", "ids", "w"):
        assert route(**{n: None}) == EINVAL
        assert route(**{n: P + 2}) == EALIGN
    assert route(score=2) == EINVAL and route(score=-1) == EINVAL
    assert route(T=-1) == ESHAPE and route(T=65537) == ESHAPE
    assert route(E=0) == ESHAPE and route(E=1025) == ESHAPE
    assert route(k=0) == ESHAPE and route(k=17) == ESHAPE and route(E=100, k=33) == ESHAPE
    assert route(bias=P) == ENOTSUP                 # a bias takes sigmoid scores
    assert route(bias=P + 1, score=1) == EALIGN
    assert route(T=0) == OK                          # nothing to do


def test_moe_refusals():
    for n in ("g", "u", "d", "X", "ids", "w", "Y"):
        assert moe(**{n: None}) == EINVAL, n
        assert moe(**{n: P + 2}) == EALIGN, n
    for n in ("g", "u", "d", "X", "Y", "ws"):
        assert moe(**{n: P + 4}) == EALIGN, n
    assert moe(fmt=6) == ENOTSUP and moe(fd=11) == ENOTSUP   # Q8K, Q8_1
    assert moe(fmt=13) == EINVAL and moe(fd=-1) == EINVAL
    assert moe(act=3) == EINVAL and moe(act=-1) == EINVAL
    assert moe(K=288) == ESHAPE and moe(F=288) == ESHAPE and moe(K=0) == ESHAPE and moe(F=0) == ESHAPE
    assert moe(fmt=0, fd=0, K=33) == ESHAPE
    assert moe(T=-1) == ESHAPE and moe(T=65537) == ESHAPE
    assert moe(E=0) == ESHAPE and moe(E=1025) == ESHAPE and moe(k=0) == ESHAPE and moe(k=33) == ESHAPE
    assert moe(E=1024, F=1 << 15) == ESHAPE          # E * F rows over the limit
    assert moe(T=65536, k=32, F=1 << 20, E=1, fd=1) == ESHAPE
    assert moe(ws=None) == EINVAL
    need = ql.moe_workspace_bytes("q4k", "q4k", 4, 8, 2, 512, 256)
    assert need > 0 and moe(wsb=need - 1) == EINVAL
    assert moe(T=0, ws=None, wsb=0) == OK


def test_logprobs_refusals():
    assert lp(x=None) == EINVAL and lp(x=P + 2) == EALIGN
    for n in ("t", "lp", "rank", "ent", "ids", "tl"):
        assert lp(**{n: P + 2}) == EALIGN, n
    assert lp(t=None) == EINVAL                       # logprob wanted without targets
    assert lp(t=None, lp=None) == EINVAL              # rank wanted without targets
    assert lp(ids=None) == EINVAL and lp(tl=None) == EINVAL
    assert lp(lp=None, rank=None, ent=None, n=0) == EINVAL  # nothing to compute
    assert lp(n=-1) == ESHAPE and lp(n=65) == ESHAPE
    assert lp(M=-1) == ESHAPE and lp(M=65537) == ESHAPE and lp(V=0) == ESHAPE and lp(V=(1 << 24) + 1) == ESHAPE
    assert lp(ld=99) == ESHAPE and lp(ld=0) == ESHAPE
    assert lp(M=0) == OK
    need = ql.logprobs_workspace_bytes(1, 131072, 5)
    assert need > 0
    assert lp(M=1, V=131072, ld=131072, n=5, wsb=need - 1) == EINVAL
    assert lp(M=1, V=131072, ld=131072, n=5, ws=None) == EINVAL
    assert lp(M=1, V=131072, ld=131072, n=5, ws=P + 8) == EALIGN


def test_head_refusals():
    assert head(B=None) == EINVAL and head(X=None) == EINVAL and head(ws=None) == EINVAL
    assert head(B=P + 8) == EALIGN and head(X=P + 8) == EALIGN and head(ws=P + 8) == EALIGN
    assert head(fmt=6) == ENOTSUP and head(fmt=99) == EINVAL
    assert head(K=255) == ESHAPE and head(M=-1) == ESHAPE and head(M=65537) == ESHAPE and head(N=0) == ESHAPE
    assert head(t=None) == EINVAL and head(n=65) == ESHAPE and head(ids=None) == EINVAL
    need = ql.head_workspace_bytes("q4k", 4, 100, 256, 2)
    assert need >= 4 * 4 * 100 and head(wsb=need - 1) == EINVAL
    assert head(M=0) == OK


def test_workspace_sizes():
    """Zero for shapes the calls refuse; the head keeps at most 2^26 logits."""
    assert ql.moe_workspace_bytes("q4k", "q4k", 4, 8, 2, 500, 256) == 0
    assert ql.moe_workspace_bytes("q8k", "q4k", 4, 8, 2, 512, 256) == 0
    assert ql.moe_workspace_bytes("q4k", "q4k", 0, 8, 2, 512, 256) == 0
    assert ql.head_workspace_bytes("q4k", 65536, 131072, 4096) <= (4 << 26) + (1 << 20)
    assert ql.head_workspace_bytes("q4k", 4, 100, 255) == 0
    assert ql.logprobs_workspace_bytes(0, 100, 2) == 0 and ql.logprobs_workspace_bytes(4, 100, 65) == 0


def test_wrappers_check_tensors():
    """Host tensors, wrong shapes and wrong types are refused by name."""
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="logits must be a device tensor"):
        ql.moe_route(x, 2)
    with pytest.raises(ValueError, match="2-D"):
        ql.moe_route(x[0], 2)
    with pytest.raises(ValueError, match="bias"):
        ql.moe_route(x, 2, score="sigmoid", bias=torch.zeros(15))
    with pytest.raises(ValueError, match="ids must be of shape"):
        ql.moe_route(x, 2, ids=torch.zeros(4, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        ql.logprobs(x)
    with pytest.raises(ValueError, match="contiguous rows"):
        ql.logprobs(x.t())
    b = torch.zeros(ql.blocks_bytes("q4k", 2 * 256, 256), dtype=torch.uint8)
    X, ids, w = torch.zeros(3, 256, dtype=torch.bfloat16), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    with pytest.raises(ValueError, match="gate_blocks is too small"):
        ql.qmatmul_moe("q4k", b[:-16], b, b, X, ids, w, 2, 256)
    with pytest.raises(ValueError, match="down_blocks is too small"):
        ql.qmatmul_moe("q4k", b, b, b, X, ids, w, 2, 256, fmt_down="q8_0")
    with pytest.raises(ValueError, match="ids and weights"):
        ql.qmatmul_moe("q4k", b, b, b, X, ids[:2], w, 2, 256)
    with pytest.raises(ValueError, match="device tensor"):
        ql.qmatmul_moe("q4k", b, b, b, X, ids, w, 2, 256)
    with pytest.raises(ValueError, match="blocks is too small"):
        ql.qmatmul_logprobs("q4k", b, X, 1000)
    with pytest.raises(ValueError, match="X must be a device tensor"):
        ql.qmatmul_logprobs("q4k", b, X, 512, torch.zeros(3, dtype=torch.int32))


def test_python_constants_match():
    assert ctypes.sizeof(ctypes.c_void_p) == 8
    assert ql.MAX_TOP_N == 64 and ql.SCORE == {"softmax": 0, "sigmoid": 1}


def test_moe_size_limit():
    """T * top_k * F and T * top_k * K up to 2^36: one more token is refused
    before any launch, with or without a size for its workspace."""
    size = ql.lib().qmatmul_moe_workspace_bytes
    assert size(0, 0, 32768, 16, 32, 1 << 16, 32) > 0            # 2^36 values of H
    assert size(0, 0, 32769, 16, 32, 1 << 16, 32) == 0
    assert size(0, 0, 32769, 8, 32, 32, 1 << 16) == 0
    assert moe(fmt=0, fd=0, T=32769, E=16, k=32, F=1 << 16, K=32) == ESHAPE
    assert moe(fmt=0, fd=0, T=32769, E=8, k=32, F=32, K=1 << 16) == ESHAPE
