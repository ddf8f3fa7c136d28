"""The cross entropy over a quantized head (qmatmul_xent) where a pass over a
row takes several workgroups: heads some of whose rows are not finite."""
import numpy as np
import pytest
import torch

import ggml_block_quant_amd as ql
import oracle
import synth
from grad_util import FMTS
from gpu_util import to_dev_bf16
from test_moe_precision import pack

pytestmark = pytest.mark.gpu


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
