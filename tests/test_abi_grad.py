"""Argument checks of the gradient and cross-entropy calls: every refusal
happens before anything is launched, so no GPU is needed.  Pointers are made-up
aligned addresses that no refused call may touch."""
import pytest
import torch

import ggml_block_quant_amd as ql

P = 0x10000  # aligned, never read
OK, EINVAL, ESHAPE, EALIGN, ENOTSUP = ql.Q_OK, ql.Q_EINVAL, ql.Q_ESHAPE, ql.Q_EALIGN, ql.Q_ENOTSUP
BIG = 1 << 45


def grad(**kw):
    a = dict(fmt=1, B=P, dY=P, dt=0, dX=P, M=4, N=100, K=256, ws=P, wsb=BIG)
    a.update(kw)
    return ql.lib().qmatmul_grad(*a.values(), None)


def glu(**kw):
    a = dict(fmt=1, g=P, u=P, X=P, dH=P, dt=0, dX=P, dG=P, dU=P, M=4, F=100, K=256, act=0, ws=P, wsb=BIG)
    a.update(kw)
    return ql.lib().qmatmul_glu_grad(*a.values(), None)


def xent(**kw):
    a = dict(fmt=1, B=P, X=P, M=4, N=100, K=256, t=P, w=P, loss=P, lse=P, dX=P, ws=P, wsb=BIG)
    a.update(kw)
    return ql.lib().qmatmul_xent(*a.values(), None)


@pytest.mark.parametrize("call,size,names,rows", (
    (grad, lambda M: ql.grad_workspace_bytes("q4k", M, 100, 256), ("B", "dY", "dX"), "N"),
    (glu, lambda M: ql.glu_grad_workspace_bytes("q4k", M, 100, 256), ("g", "u", "X", "dH", "dX"), "F"),
    (xent, lambda M: ql.xent_workspace_bytes("q4k", M, 100, 256), ("B", "X"), "N")))
def test_refusals(call, size, names, rows):
    for n in names:
        assert call(**{n: None}) == EINVAL or (call is xent and n == "dX"), n
        assert call(**{n: P + 8}) == EALIGN, n
    assert call(fmt=6) == ENOTSUP and call(fmt=11) == ENOTSUP and call(fmt=13) == EINVAL and call(fmt=-1) == EINVAL
    assert call(K=255) == ESHAPE and call(K=288) == ESHAPE and call(K=0) == ESHAPE and call(fmt=0, K=48) == ESHAPE
    assert call(M=-1) == ESHAPE and call(M=65537) == ESHAPE
    assert call(**{rows: 0}) == ESHAPE and call(**{rows: (1 << 24) + 1}) == ESHAPE
    assert call(M=65536, K=1 << 20, **{rows: 1 << 24}) == ESHAPE  # elements over 2^40
    assert call(ws=None) == EINVAL and call(ws=P + 8) == EALIGN
    need = size(4)
    assert need > 0 and call(wsb=need - 1) == EINVAL and call(wsb=0) == EINVAL
    assert call(M=0, ws=None, wsb=0) == OK  # nothing to do


def test_more_refusals():
    assert grad(dt=2) == EINVAL and grad(dt=-1) == EINVAL
    assert glu(dt=2) == EINVAL and glu(act=3) == EINVAL and glu(act=-1) == EINVAL
    assert glu(dG=P + 8) == EALIGN and glu(dU=P + 8) == EALIGN
    for n in ("t", "w", "loss", "lse"):
        assert xent(**{n: P + 2}) == EALIGN, n
    assert xent(t=None) == EINVAL and xent(loss=None) == EINVAL
    assert xent(dX=P + 8) == EALIGN
    # the loss alone needs less, and its size does not do for the gradient
    a, b = ql.xent_workspace_bytes("q4k", 4, 100, 256, grad=False), ql.xent_workspace_bytes("q4k", 4, 100, 256)
    assert 0 < a < b and xent(wsb=a) == EINVAL and xent(dX=None, wsb=a - 1) == EINVAL


MS = (*range(1, 70), 127, 128, 129, 171, 255, 256, 257, 511, 512, 513, 1023, 1024, 2047, 2048, 2049, 4095, 4096, 4097, 65536)


@pytest.mark.parametrize("fmt", ("q4k", "q8_0", "fp8"))
def test_workspaces_grow_with_the_rows_and_stay_bounded(fmt):
    for N in (1, 100, 127, 4096, 14336, 131072, 1 << 20, 1 << 24):
        for K in (256, 4096, 14336):
            for size in (ql.grad_workspace_bytes, ql.glu_grad_workspace_bytes, ql.xent_workspace_bytes,
                         lambda *a: ql.xent_workspace_bytes(*a, grad=False)):
                v = [size(fmt, M, N, K) for M in MS]
                assert v == sorted(v) and v[0] > 0, (N, K)
                # the chunks' values, the splits' sums, the rows at once of the
                # narrow sides
                assert v[-1] <= 12 * max(1 << 27, 32 * (N + 64)) + 4 * 32768 * (K + 64) + (1 << 24), (N, K, v[-1])
    for f in (ql.grad_workspace_bytes, ql.glu_grad_workspace_bytes, ql.xent_workspace_bytes):
        assert f("q4k", 4, 100, 255) == 0 and f("q4k", 0, 100, 256) == 0 and f("q8k", 4, 100, 256) == 0
        assert f("q4k", 65537, 100, 256) == 0


def test_wrappers_check_tensors():
    """Host tensors, wrong shapes and wrong types are refused by name."""
    N, K, M = 40, 256, 3
    b = torch.zeros(ql.blocks_bytes("q4k", N, K), dtype=torch.uint8)
    X, d, t = torch.zeros((M, K), dtype=torch.bfloat16), torch.zeros((M, N)), torch.zeros(M, dtype=torch.int32)
    with pytest.raises(ValueError, match="2-D"):
        ql.qmatmul_grad("q4k", b, d[0], K)
    with pytest.raises(ValueError, match="dY must be torch.float32 or torch.bfloat16"):
        ql.qmatmul_grad("q4k", b, d.double(), K)
    with pytest.raises(ValueError, match="too small"):
        ql.qmatmul_grad("q4k", b[:-16], d, K)
    with pytest.raises(ValueError, match="dY must be a device tensor"):
        ql.qmatmul_grad("q4k", b, d, K)
    with pytest.raises(ValueError, match="dH must be of shape"):
        ql.qmatmul_glu_grad("q4k", b, b, X, d[:2])
    with pytest.raises(ValueError, match="up_blocks is too small"):
        ql.qmatmul_glu_grad("q4k", b, b[:-16], X, d)
    with pytest.raises(ValueError, match="dH must be torch.float32 or torch.bfloat16"):
        ql.qmatmul_glu_grad("q4k", b, b, X, d.half())
    with pytest.raises(ValueError, match="X must be a device tensor"):
        ql.qmatmul_glu_grad("q4k", b, b, X, d)
    with pytest.raises(ValueError, match="targets must be of shape"):
        ql.qmatmul_xent("q4k", b, X, N, t[:2])
    with pytest.raises(ValueError, match="weights must be of shape"):
        ql.qmatmul_xent("q4k", b, X, N, t, weights=torch.zeros(2))
    with pytest.raises(ValueError, match="blocks is too small"):
        ql.qmatmul_xent("q4k", b, X, N + 1, t)
    with pytest.raises(ValueError, match="X must be a device tensor"):
        ql.qmatmul_xent("q4k", b, X, N, t)
    assert ql.GRAD_TYPE == {torch.float32: 0, torch.bfloat16: 1}
