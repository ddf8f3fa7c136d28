"""Workspaces of the log-probability calls: one sized for the largest batch
serves every smaller one."""
import numpy as np
import pytest
import torch

import ggml_block_quant_amd as ql
import synth
from gpu_util import to_dev_bf16

MS = (*range(1, 70), 127, 128, 171, 255, 256, 257, 511, 512, 513, 1023, 1024, 1366, 2047, 2048, 2049, 4095, 4096, 4097, 65536)
VS = (1, 100, 4092, 4093, 4094, 8189, 8190, 32003, 61437, 61438, 65533, 126973, 126974, 131072, 131073, 262144, 1 << 20, 1 << 24)


@pytest.mark.parametrize("top", (0, 1, 8, 20, 64))
def test_sizes_grow_with_the_rows(top):
    for V in VS:
        size = [ql.logprobs_workspace_bytes(M, V, top) for M in MS]
        assert size == sorted(size), V
        assert size[-1] <= 8190 * (16 + 8 * top)  # two parts of 4095 rows
        if top:
            fewer = [ql.logprobs_workspace_bytes(M, V, top - 1) for M in MS]
            assert all(a <= b for a, b in zip(fewer, size)), V
    for N in (100, 32003, 131072, 262144):
        size = [ql.head_workspace_bytes("q4k", M, N, 256, top) for M in MS]
        assert size == sorted(size), N


@pytest.mark.gpu
@pytest.mark.parametrize("V,top", ((32003, 20), (131072, 64), (131072, 0), (200001, 3)))
def test_one_workspace_for_every_batch(V, top):
    """The size of 600 rows, and NaN patterns around it, for batches of every
    split into parts."""
    most = 600
    n = ql.logprobs_workspace_bytes(most, V, top)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
    x = torch.randn((most, V), device="cuda", generator=torch.Generator("cuda").manual_seed(V))
    t = torch.arange(most, dtype=torch.int32, device="cuda") * 7
    for M in (600, 512, 511, 300, 256, 255, 171, 64, 17, 16, 2, 1):
        a = ql.logprobs(x[:M], t[:M], top, workspace=ws[:n])
        b = ql.logprobs(x[:M], t[:M], top)
        for u, v in zip(a, b):
            assert (u is None and v is None) or torch.equal(u, v)
        lse = torch.logsumexp(x[:M].double(), 1)
        want = x[:M].double().gather(1, t[:M, None].long())[:, 0] - lse
        # lse: the exponents' rounding and sums of up to V / 256 terms a thread
        assert ((a.logprob.double() - want).abs() <= (72 + V / 256 + 20 + 3 * 32) * 2.0 ** -24).all()
    assert (ws[n:] == 255).all()


@pytest.mark.gpu
def test_one_workspace_for_every_batch_of_a_head():
    N, K, top, most = 70001, 256, 20, 1100
    blocks = ql.isq("q4k", to_dev_bf16(synth.weights_bf16(66000, N, K)))
    X = to_dev_bf16(synth.activations_bf16(66001, most, K))
    t = torch.from_numpy(np.arange(most, dtype=np.int32) * 63).cuda()
    ws = torch.full((ql.head_workspace_bytes("q4k", most, N, K, top),), 255, dtype=torch.uint8, device="cuda")
    for M in (1100, 900, 769, 768, 511, 255, 9, 1):
        a = ql.qmatmul_logprobs("q4k", blocks, X[:M], N, t[:M], top, workspace=ws)
        b = ql.qmatmul_logprobs("q4k", blocks, X[:M], N, t[:M], top)
        for u, v in zip(a, b):
            assert torch.equal(u, v)
