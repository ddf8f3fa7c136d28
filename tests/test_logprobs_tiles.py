"""Log probabilities around the first tile boundary (4096 logits, counted from
the 16-byte boundary at or below the row's start), rows at every alignment.

Bar: as in test_parity_logprobs, with the number of terms one thread adds: a
workgroup of 256 threads walks a part of a row, so at most V / 256 + 16 of them
(one part a row; several parts have fewer)."""
import numpy as np
import pytest
import torch

import ggml_block_quant_amd as ql
from test_parity_logprobs import U, close, want

pytestmark = pytest.mark.gpu


def check(got, x, t, top, label):
    V = x.shape[1]
    ref = want(x, t, top)
    part = (2 * 32 + 4 + V / 256 + 16 + 20 + 3 * np.log(V + 1)) * U
    assert np.array_equal(got.rank.cpu().numpy(), ref["rank"]), label
    close(got.logprob, ref["logprob"], part, label)
    close(got.entropy, ref["entropy"], part * min(32, np.log(V) + 1), label)
    if top:
        assert np.array_equal(got.top_ids.cpu().numpy(), ref["top_ids"]), label
        close(got.top_logprobs, ref["top_logprobs"], part, label)


@pytest.mark.parametrize("V", (*range(4092, 4100), 8188, 8189, 8192, 8195))
@pytest.mark.parametrize("M", (5, 520))
def test_tile_boundaries_at_every_alignment(V, M):
    """M = 520: one part a row; 5: a part per tile.  The best logits stand at the
    boundary; what lies between the rows (NaN) belongs to none."""
    rng = np.random.default_rng(V + M)
    x = (rng.standard_normal((M, V)) * 3).astype(np.float32)
    x[:, 4090:4100] += 12
    x[0::5, V - 1] = 40
    x[1::5, :V - 1] = -np.inf
    x[2::5] = 1.5
    t = rng.integers(0, V, M).astype(np.int32)
    t[::2] = V - 1
    for start in range(4):
        for gap in (0, 1, 6):
            ld = V + gap
            buf = torch.full((start + M * ld,), float("nan"), device="cuda")
            view = buf[start:].as_strided((M, V), (ld, 1))
            view.copy_(torch.from_numpy(x))
            for top in (0, 6):
                check(ql.logprobs(view, torch.from_numpy(t).cuda(), top), x, t, top, f"V={V} M={M} start={start} ld={ld} top={top}")
