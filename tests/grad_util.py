"""The gradients' definitions in 64 bits and the bounds that their kernels are
held to, shared by the GPU tests of the gradients and the cross entropy.

Roundings, relative to the value (half a step, torch.finfo(t).eps / 2): a weight
or a gradient to fp16 2^-11 (the latter also 2^-39 of its row's largest: half of
fp16's smallest step, 2^-25, over a row that is scaled to 2^14 or more), an fp32
sum of n terms n * 2^-24 of the magnitudes summed, bf16 results 2^-8 (and half
of their smallest step, 2^-134)."""
import torch

import oracle
import synth

E16, U, EB = 2.0 ** -11, 2.0 ** -24, 2.0 ** -8
FMTS = ("q8_0", "q4k", "q6k", "q5k", "q3k", "q2k", "q4_0", "q4_1", "q5_0", "q5_1", "fp8")


def weights(fmt, seed, N, K, outliers=False):
    """(bf16 bits, values in 64 bits on the device) of a [N][K] weight."""
    w = synth.weights_bf16(seed, N, K, outliers=outliers)
    if fmt == "fp8":
        W = oracle.dequant_fp8(oracle.quantize_fp8(w))
    else:
        W = oracle.dequant(fmt, oracle.quantize(fmt, w), N, K)
    return w, torch.from_numpy(W).cuda()


def rounded(y, tol):
    """The bound of a value within tol of y after its rounding to bf16."""
    return tol + EB * (y.abs() + tol) + 2.0 ** -134


def within(got, want, tol, label):
    got, want = got.double(), want.double()
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(int(v) for v in torch.nonzero(bad)[0])
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {float(got[i])} for "
                             f"{float(want[i])}, bound {float(tol[i]):.3e}")


def back(A, W, extra=None):
    """A . W in 64 bits and the bound of the kernels' sums of it; extra: a bound
    of A's own errors (A's roundings here are those of the product alone)."""
    n = A.shape[1]
    y = A @ W
    a = A.abs() if extra is None else A.abs() + extra
    tol = (2 * E16 + E16 ** 2 + (n + 8) * U) * (a @ W.abs())
    tol = tol + 2.0 ** -39 * a.amax(1, keepdim=True) * W.abs().sum(0, keepdim=True) * 1.001
    if extra is not None:
        tol = tol + extra @ W.abs()
    return y, tol


def forward(X, W, pair=False):
    """X . W^T in 64 bits and the bound of the kernels' sums: one fp16 a weight,
    or a pair (2^-22: its low half is an fp16 of what the high half leaves, down
    to fp16's smallest step, 2^-25 of a weight's unit)."""
    den = X.abs() @ W.abs().t()
    n = X.shape[1]
    tol = ((2.0 ** -22 if pair else E16) + (2 * n + 8) * U) * den
    tol = tol + 2.0 ** -39 * X.abs().amax(1, keepdim=True) * W.abs().sum(1)[None] * 1.001
    if pair:
        tol = tol + 2.0 ** -25 * X.abs().sum(1, keepdim=True)
    return X @ W.t(), tol
