"""Block-quantized linear layers on AMD MI355X (gfx950).

A thin Python binding over the C ABI of ``libqlinear.so`` (declared in
``include/qlinear.h``): in-situ quantization of bf16 weights into Q8_0, Q4K
or Q6K blocks (and Q5K, Q3K, Q2K, Q4_0, Q4_1, Q5_0, Q5_1), the fused
dequantize-matmul that consumes them, the gated feed-forward projection, the
mixture-of-experts layer and its router, the quantized embedding lookup, the
output head's log probabilities, and the gradients through frozen quantized
weights (linear layer, gated projection, the head's cross entropy).  Every
step of the computation runs in the library's HIP kernels; this module only
checks tensors and passes pointers, sizes and the current HIP stream.
PyTorch provides device memory and streams.

Formats and policy follow page "Quantization types" (mistral.rs reference):
sections "Numeric shorthands", "Sensitive tensor precision", "Q*K family"
and "Legacy GGML types".
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# QLINEAR_LIB names another build of the same library (the host-sanitizer
# build of tests/sanitize_host.py); there is no other implementation
LIB_PATH = os.environ.get("QLINEAR_LIB") or os.path.join(_HERE, "libqlinear.so")

FMT = {"q8_0": 0, "q4k": 1, "q6k": 2, "q2k": 3, "q3k": 4, "q5k": 5, "q8k": 6,
       "q4_0": 7, "q4_1": 8, "q5_0": 9, "q5_1": 10, "q8_1": 11, "fp8": 12}
FMT_NAME = {v: k for k, v in FMT.items()}
PATH = {"auto": 0, "gemv": 1, "mfma_bf16": 2, "mfma_i8": 3, "mfma_fp8": 4}
ACT = {"silu": 0, "relu": 1, "sigmoid": 2}
SCORE = {"softmax": 0, "sigmoid": 1}
GRAD_TYPE = {torch.float32: 0, torch.bfloat16: 1}  # QTYPE_F32, QTYPE_BF16
MAX_TOP_N = 64  # QLINEAR_MAX_TOP_N

Q_OK, Q_EINVAL, Q_ESHAPE, Q_EALIGN, Q_ENOTSUP, Q_EHIP, Q_ESCRATCH = 0, -1, -2, -3, -4, -5, -6
STATIC_SCRATCH_BYTES = 32 << 20  # QLINEAR_STATIC_SCRATCH_BYTES

# every symbol include/qlinear.h declares, with its ctypes signature
_P, _I64, _INT, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
_IP = ctypes.POINTER(ctypes.c_int)
SIGNATURES = {
    "q_blocks_bytes": (_SZ, [_INT, _I64, _I64]),
    "isq_quantize": (_INT, [_INT, _P, _I64, _I64, _P, _P]),
    "q_act_quantize": (_INT, [_P, _I64, _I64, _P, _P]),
    "qmatmul": (_INT, [_INT, _P, _P, _P, _I64, _I64, _I64, _P]),
    "qmatmul_workspace_bytes": (_SZ, [_INT, _INT, _I64, _I64]),
    "qmatmul_ex": (_INT, [_INT, _P, _P, _P, _I64, _I64, _I64, _INT, _P, _SZ, _P]),
    "qmatmul_static": (_INT, [_INT, _P, _P, _P, _I64, _I64, _I64, _INT, _P]),
    "q_embed": (_INT, [_INT, _P, _I64, _I64, _P, _I64, _P, _P]),
    "qmatmul_glu_workspace_bytes": (_SZ, [_INT, _I64, _I64, _I64]),
    "qmatmul_glu": (_INT, [_INT, _P, _P, _P, _P, _I64, _I64, _I64, _INT, _P, _SZ, _P]),
    "q_moe_route": (_INT, [_P, _I64, _I64, _INT, _INT, _P, _INT, ctypes.c_float, _P, _P, _P]),
    "qmatmul_moe_workspace_bytes": (_SZ, [_INT, _INT, _I64, _I64, _INT, _I64, _I64]),
    "qmatmul_moe": (_INT, [_INT, _P, _P, _INT, _P, _P, _P, _P, _P, _I64, _I64, _INT, _I64, _I64, _INT, _P, _SZ, _P]),
    "q_logprobs_workspace_bytes": (_SZ, [_I64, _I64, _INT]),
    "q_logprobs": (_INT, [_P, _I64, _I64, _I64, _P, _INT, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "qmatmul_logprobs_workspace_bytes": (_SZ, [_INT, _I64, _I64, _I64, _INT]),
    "qmatmul_logprobs": (_INT, [_INT, _P, _P, _I64, _I64, _I64, _P, _INT, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "qmatmul_grad_workspace_bytes": (_SZ, [_INT, _I64, _I64, _I64]),
    "qmatmul_grad": (_INT, [_INT, _P, _P, _INT, _P, _I64, _I64, _I64, _P, _SZ, _P]),
    "qmatmul_glu_grad_workspace_bytes": (_SZ, [_INT, _I64, _I64, _I64]),
    "qmatmul_glu_grad": (_INT, [_INT, _P, _P, _P, _P, _INT, _P, _P, _P, _I64, _I64, _I64, _INT, _P, _SZ, _P]),
    "qmatmul_xent_workspace_bytes": (_SZ, [_INT, _I64, _I64, _I64, _INT]),
    "qmatmul_xent": (_INT, [_INT, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "q_dequantize": (_INT, [_INT, _P, _I64, _I64, _P, _P]),
    "isq_resolve_level": (_INT, [_INT, _IP]),
    "isq_sensitive_fmt": (_INT, [_INT, _IP]),
    "isq_tensor_fmt": (_INT, [_INT, _INT, _INT, _IP]),
    "q_fmt_supported": (_INT, [_INT]),
    "q_fmt_name": (ctypes.c_char_p, [_INT]),
    "q_strerror": (ctypes.c_char_p, [_INT]),
    "q_probe_read": (_INT, [_P, _I64, _P, _P]),
    "q_probe_mfma": (_INT, [_P, _I64, _P]),
    "q_probe_mfma_flops": (_I64, [_I64]),
    "q_probe_mix": (_INT, [_P, _I64, _INT, _INT, _P]),
    "q_probe_mix_valu": (_I64, [_I64, _INT]),
}


class QLinearError(RuntimeError):
    """A call into libqlinear returned an error status."""

    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status} ({strerror(status)})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library.  Raises ImportError if it has not been built:
    there is no fallback implementation."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run `python -m ggml_block_quant_amd.build` "
                              "or __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().q_strerror(status).decode()


def _fmt(fmt) -> int:
    return FMT[fmt] if isinstance(fmt, str) else int(fmt)


def _check(fn: str, status: int):
    if status != Q_OK:
        raise QLinearError(fn, status)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    """The current device's current stream.  The raw getter, where torch has
    it, costs a fortieth of building a Stream object (0.07 against 2.8 us)."""
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _dev(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _shaped(t, name: str, shape):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be of shape {tuple(shape)}, got {tuple(t.shape)}")


def _out(t, name: str, shape, dtype, like: torch.Tensor) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _shaped(t, name, shape)
    return t


def _blocks_fit(t: torch.Tensor, name: str, fmt: int, N: int, K: int):
    """A block buffer at least as long as its [N][K] weight needs (a shape the
    format does not take has no size here; the call reports it)."""
    if t.numel() * t.element_size() < lib().q_blocks_bytes(fmt, N, K):
        raise ValueError(f"{name} is too small for [{N}][{K}]")


def _ptr(t, name: str, dtype, dev: int):
    """The address of a contiguous tensor of that type on device ``dev`` (None
    for none)."""
    if t is None:
        return None
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        raise ValueError(f"{name} is on {t.device}, other tensors of the call on device {dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _device_of(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.get_device()


def _call(fn: str, dev: int, *args):
    """A library call with device ``dev`` current, on its current stream."""
    if dev == torch.cuda.current_device():
        st = getattr(_lib, fn)(*args, _stream())
    else:
        with torch.cuda.device(dev):
            st = getattr(_lib, fn)(*args, _stream())
    if st != Q_OK:
        raise QLinearError(fn, st)


# ----------------------------------------------------------------------------
# host-side helpers (no GPU needed)
# ----------------------------------------------------------------------------

def blocks_bytes(fmt, N: int, K: int) -> int:
    return int(lib().q_blocks_bytes(_fmt(fmt), N, K))


def workspace_bytes(fmt, path, M: int, K: int) -> int:
    p = PATH[path] if isinstance(path, str) else int(path)
    return int(lib().qmatmul_workspace_bytes(_fmt(fmt), p, M, K))


def resolve_level(level: int) -> str:
    out = ctypes.c_int()
    _check("isq_resolve_level", lib().isq_resolve_level(level, ctypes.byref(out)))
    return FMT_NAME[out.value]


def sensitive_fmt(model_default) -> str:
    out = ctypes.c_int()
    _check("isq_sensitive_fmt", lib().isq_sensitive_fmt(_fmt(model_default), ctypes.byref(out)))
    return FMT_NAME[out.value]


def tensor_fmt(level: int, is_embedding_or_head: bool, explicit=None) -> str:
    out = ctypes.c_int()
    e = -1 if explicit is None else _fmt(explicit)
    _check("isq_tensor_fmt", lib().isq_tensor_fmt(level, int(bool(is_embedding_or_head)), e, ctypes.byref(out)))
    return FMT_NAME[out.value]


def fmt_supported(fmt) -> bool:
    return bool(lib().q_fmt_supported(_fmt(fmt)))


# ----------------------------------------------------------------------------
# device calls
# ----------------------------------------------------------------------------

def isq(fmt, W: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Quantize bf16 weights W [N][K] (device) into a uint8 block buffer."""
    if W.dim() != 2:
        raise ValueError("W must be 2-D [N][K]")
    N, K = W.shape
    nbytes = blocks_bytes(fmt, N, K)
    if nbytes == 0:
        raise QLinearError("q_blocks_bytes", Q_ESHAPE)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    elif out.numel() < nbytes or out.dtype != torch.uint8:
        raise ValueError("out is too small or not uint8")
    _check("isq_quantize", lib().isq_quantize(_fmt(fmt), _dev(W, "W", torch.bfloat16), N, K,
                                              _dev(out, "out"), _stream()))
    return out


def act_quantize(X: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Quantize bf16 activations X [M][K] to Q8_0 blocks (codes then scales)."""
    M, K = X.shape
    nbytes = blocks_bytes("q8_0", M, K)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=X.device)
    _check("q_act_quantize", lib().q_act_quantize(_dev(X, "X", torch.bfloat16), M, K,
                                                  _dev(out, "out"), _stream()))
    return out


def qmatmul(fmt, blocks: torch.Tensor, X: torch.Tensor, N: int, path="auto",
            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Y = X . deq(W)^T as fp32 [M][N] for X bf16 [M][K] and the blocks of a
    [N][K] weight.  ``path``: auto | gemv | mfma_bf16 | mfma_i8 | mfma_fp8."""
    if X.dim() != 2:
        raise ValueError("X must be 2-D [M][K]")
    M, K = X.shape
    p = PATH[path] if isinstance(path, str) else int(path)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=X.device)
    ws_ptr, ws_bytes = None, 0
    need = workspace_bytes(fmt, p, M, K)
    if need:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
        ws_ptr, ws_bytes = _dev(workspace, "workspace"), workspace.numel()
    _check("qmatmul_ex", lib().qmatmul_ex(_fmt(fmt), _dev(blocks, "blocks", torch.uint8),
                                          _dev(X, "X", torch.bfloat16), _dev(out, "Y", torch.float32),
                                          M, N, K, p, ws_ptr, ws_bytes, _stream()))
    return out


def qmatmul_static(fmt, blocks: torch.Tensor, X: torch.Tensor, N: int, path="auto",
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """As ``qmatmul``, with no workspace: the int8 and FP8 paths keep X's
    activation blocks in the library's fixed per-GPU buffer (calls that
    overlap in time on one GPU race on it).  With ``out`` given, the call
    itself allocates nothing."""
    if X.dim() != 2:
        raise ValueError("X must be 2-D [M][K]")
    M, K = X.shape
    p = PATH[path] if isinstance(path, str) else int(path)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=X.device)
    _check("qmatmul_static", lib().qmatmul_static(_fmt(fmt), _dev(blocks, "blocks", torch.uint8),
                                                  _dev(X, "X", torch.bfloat16), _dev(out, "Y", torch.float32),
                                                  M, N, K, p, _stream()))
    return out


def glu_workspace_bytes(fmt, M: int, F: int, K: int) -> int:
    return lib().qmatmul_glu_workspace_bytes(_fmt(fmt), M, F, K)


def qmatmul_glu(fmt, gate_blocks: torch.Tensor, up_blocks: torch.Tensor, X: torch.Tensor, F: int,
                act="silu", out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """H = act(X . deq(Wg)^T) * (X . deq(Wu)^T) as fp32 [M][F] for the blocks
    of the [F][K] gate and up weights; ``act``: silu | relu | sigmoid."""
    if X.dim() != 2:
        raise ValueError("X must be 2-D [M][K]")
    M, K = X.shape
    if out is None:
        out = torch.empty((M, F), dtype=torch.float32, device=X.device)
    ws_ptr, ws_bytes = None, 0
    need = glu_workspace_bytes(fmt, M, F, K)
    if need:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
        ws_ptr, ws_bytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    a = ACT[act] if isinstance(act, str) else int(act)
    _check("qmatmul_glu", lib().qmatmul_glu(_fmt(fmt), _dev(gate_blocks, "gate_blocks", torch.uint8),
                                            _dev(up_blocks, "up_blocks", torch.uint8),
                                            _dev(X, "X", torch.bfloat16), _dev(out, "H", torch.float32),
                                            M, F, K, a, ws_ptr, ws_bytes, _stream()))
    return out


def embed(fmt, blocks: torch.Tensor, N: int, K: int, ids: torch.Tensor,
          out: torch.Tensor | None = None) -> torch.Tensor:
    """Rows ``ids`` (int32, device) of the quantized [N][K] table, dequantized
    exactly to fp32 [len(ids)][K]; ids outside [0, N) give zero rows.  The
    same blocks serve ``qmatmul`` as a tied output head."""
    if ids.dim() != 1:
        raise ValueError("ids must be 1-D")
    n = ids.numel()
    if out is None:
        out = torch.empty((n, K), dtype=torch.float32, device=blocks.device)
    if n == 0:
        return out
    _check("q_embed", lib().q_embed(_fmt(fmt), _dev(blocks, "blocks", torch.uint8), N, K,
                                    _dev(ids, "ids", torch.int32), n, _dev(out, "out", torch.float32),
                                    _stream()))
    return out


def moe_route(logits: torch.Tensor, top_k: int, score="softmax", bias: torch.Tensor | None = None, renorm: bool = True,
              scale: float = 1.0, ids: torch.Tensor | None = None, weights: torch.Tensor | None = None):
    """A router's choice from its fp32 logits [T][E]: (ids int32 [T][top_k],
    weights fp32 [T][top_k]).  ``score``: softmax | sigmoid; ``bias`` [E]
    (sigmoid only) takes part in the choice; ``renorm``: weights divided by
    their sum.  Logits of -inf are never chosen (id -1, weight 0)."""
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D [T][E]")
    T, E = logits.shape
    _shaped(bias, "bias", (E,))
    ids = _out(ids, "ids", (T, top_k), torch.int32, logits)
    weights = _out(weights, "weights", (T, top_k), torch.float32, logits)
    sc = SCORE[score] if isinstance(score, str) else int(score)
    dev = _device_of(logits, "logits")
    args = (_ptr(logits, "logits", torch.float32, dev), T, E, top_k, sc, _ptr(bias, "bias", torch.float32, dev),
            1 if renorm else 0, scale, _ptr(ids, "ids", torch.int32, dev), _ptr(weights, "weights", torch.float32, dev))
    if T:
        lib()
        _call("q_moe_route", dev, *args)
    return ids, weights


def moe_workspace_bytes(fmt, fmt_down, T: int, E: int, top_k: int, F: int, K: int) -> int:
    return int(lib().qmatmul_moe_workspace_bytes(_fmt(fmt), _fmt(fmt_down), T, E, top_k, F, K))


def qmatmul_moe(fmt, gate_blocks: torch.Tensor, up_blocks: torch.Tensor, down_blocks: torch.Tensor, X: torch.Tensor,
                ids: torch.Tensor, weights: torch.Tensor, E: int, F: int, act="silu", fmt_down=None,
                out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Mixture-of-experts layer as fp32 [T][K]: sum over j of weights[t][j] *
    Wd[e] . (act(Wg[e] . x) * (Wu[e] . x)), e = ids[t][j], for the blocks of the
    experts' stacked [E*F][K] gate and up weights (``fmt``) and [E*K][F] down
    weights (``fmt_down``, by default ``fmt``).  ids outside [0, E) add nothing.
    How the values between the two weights are held, and the accuracy that
    follows, is stated at qmatmul_moe in include/qlinear.h."""
    if X.dim() != 2 or ids.dim() != 2:
        raise ValueError("X must be 2-D [T][K] and ids 2-D [T][top_k]")
    T, K = X.shape
    k = ids.shape[1]
    if ids.shape[0] != T or weights.shape != ids.shape:
        raise ValueError("ids and weights must be [T][top_k]")
    f, fd = _fmt(fmt), _fmt(fmt if fmt_down is None else fmt_down)
    _blocks_fit(gate_blocks, "gate_blocks", f, E * F, K)
    _blocks_fit(up_blocks, "up_blocks", f, E * F, K)
    _blocks_fit(down_blocks, "down_blocks", fd, E * K, F)
    out = _out(out, "Y", (T, K), torch.float32, X)
    a = ACT[act] if isinstance(act, str) else int(act)
    if workspace is None:
        need = lib().qmatmul_moe_workspace_bytes(f, fd, T, E, k, F, K)
        workspace = X.new_empty(need, dtype=torch.uint8) if need else None
    dev, u8 = _device_of(X, "X"), torch.uint8
    args = (f, _ptr(gate_blocks, "gate_blocks", u8, dev), _ptr(up_blocks, "up_blocks", u8, dev), fd,
            _ptr(down_blocks, "down_blocks", u8, dev), _ptr(X, "X", torch.bfloat16, dev),
            _ptr(ids, "ids", torch.int32, dev), _ptr(weights, "weights", torch.float32, dev),
            _ptr(out, "Y", torch.float32, dev), T, E, k, F, K, a, _ptr(workspace, "workspace", u8, dev),
            0 if workspace is None else workspace.numel())
    if T:
        _call("qmatmul_moe", dev, *args)
    return out


class LogProbs(NamedTuple):
    """Results of ``logprobs``: logprob and rank [M] (None without targets),
    entropy [M], top_ids and top_logprobs [M][top] (None for top = 0)."""
    logprob: torch.Tensor | None
    rank: torch.Tensor | None
    entropy: torch.Tensor | None
    top_ids: torch.Tensor | None
    top_logprobs: torch.Tensor | None


def _logprob_out(out, M, targets, top, like, dev):
    """The results' tensors and the addresses of targets and results."""
    f, i = torch.float32, torch.int32
    if out is None:
        given = targets is not None
        out = LogProbs(like.new_empty(M, dtype=f) if given else None, like.new_empty(M, dtype=i) if given else None,
                       like.new_empty(M, dtype=f), like.new_empty((M, top), dtype=i) if top else None,
                       like.new_empty((M, top), dtype=f) if top else None)
    else:
        for t, name, shape in ((out.logprob, "logprob", (M,)), (out.rank, "rank", (M,)), (out.entropy, "entropy", (M,)),
                               (out.top_ids, "top_ids", (M, top)), (out.top_logprobs, "top_logprobs", (M, top))):
            _shaped(t, name, shape)
    _shaped(targets, "targets", (M,))
    return out, (_ptr(targets, "targets", i, dev), top, _ptr(out.logprob, "logprob", f, dev), _ptr(out.rank, "rank", i, dev),
                 _ptr(out.entropy, "entropy", f, dev), _ptr(out.top_ids, "top_ids", i, dev),
                 _ptr(out.top_logprobs, "top_logprobs", f, dev))


def logprobs_workspace_bytes(M: int, V: int, top: int = 0) -> int:
    """Bytes of a workspace for ``logprobs`` of up to M rows of V logits and up
    to ``top`` alternatives."""
    return int(lib().q_logprobs_workspace_bytes(M, V, top))


def logprobs(logits: torch.Tensor, targets: torch.Tensor | None = None, top: int = 0, out: LogProbs | None = None,
             workspace: torch.Tensor | None = None) -> LogProbs:
    """Log probability and rank of ``targets`` (int32 [M]; outside [0, V): not
    scored, 0), entropy and the ``top`` most probable tokens of each row of
    fp32 logits [M][V] (rows may be apart: any stride of at least V along M).
    -inf masks a token.  ``out``: a LogProbs whose tensors are overwritten
    (those that are None are not computed)."""
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be 2-D [M][V] with contiguous rows")
    M, V = logits.shape
    dev = _device_of(logits, "logits")
    if logits.dtype is not torch.float32:
        raise ValueError(f"logits must be torch.float32, got {logits.dtype}")
    out, args = _logprob_out(out, M, targets, top, logits, dev)
    if workspace is None:
        need = lib().q_logprobs_workspace_bytes(M, V, top)
        workspace = logits.new_empty(need, dtype=torch.uint8) if need else None
    ws = _ptr(workspace, "workspace", torch.uint8, dev)
    if M:
        lib()
        _call("q_logprobs", dev, logits.data_ptr(), M, V, logits.stride(0) if M > 1 else V, *args, ws,
              0 if workspace is None else workspace.numel())
    return out


def head_workspace_bytes(fmt, M: int, N: int, K: int, top: int = 0) -> int:
    """Bytes of a workspace for ``qmatmul_logprobs`` of up to M rows and up
    to ``top`` alternatives on an [N][K] head."""
    return int(lib().qmatmul_logprobs_workspace_bytes(_fmt(fmt), M, N, K, top))


def qmatmul_logprobs(fmt, blocks: torch.Tensor, X: torch.Tensor, N: int, targets: torch.Tensor | None = None,
                     top: int = 0, out: LogProbs | None = None, workspace: torch.Tensor | None = None) -> LogProbs:
    """``logprobs`` of the logits X . deq(W)^T of a quantized [N][K] output
    head, for X bf16 [M][K], without holding the M x N logits (at most 2^26 of
    them at a time, in the workspace)."""
    if X.dim() != 2:
        raise ValueError("X must be 2-D [M][K]")
    M, K = X.shape
    f = _fmt(fmt)
    _blocks_fit(blocks, "blocks", f, N, K)
    dev = _device_of(X, "X")
    out, args = _logprob_out(out, M, targets, top, X, dev)
    if workspace is None:
        need = lib().qmatmul_logprobs_workspace_bytes(f, M, N, K, top)
        workspace = X.new_empty(need, dtype=torch.uint8) if need else None
    ws = _ptr(workspace, "workspace", torch.uint8, dev)
    b, x = _ptr(blocks, "blocks", torch.uint8, dev), _ptr(X, "X", torch.bfloat16, dev)
    if M:
        _call("qmatmul_logprobs", dev, f, b, x, M, N, K, *args, ws, 0 if workspace is None else workspace.numel())
    return out


# ----------------------------------------------------------------------------
# gradients through frozen quantized weights
# ----------------------------------------------------------------------------

def _grad_type(t: torch.Tensor, name: str) -> int:
    if t.dtype not in GRAD_TYPE:
        raise ValueError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")
    return GRAD_TYPE[t.dtype]


def grad_workspace_bytes(fmt, M: int, N: int, K: int) -> int:
    """Bytes of a workspace for ``qmatmul_grad`` of up to M rows."""
    return int(lib().qmatmul_grad_workspace_bytes(_fmt(fmt), M, N, K))


def qmatmul_grad(fmt, blocks: torch.Tensor, dY: torch.Tensor, K: int, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of ``qmatmul``'s result with respect to X: dX = dY . deq(W) as
    bf16 [M][K], for dY fp32 or bf16 [M][N] and the blocks of the [N][K]
    weight.  The accuracy is stated at qmatmul_grad in include/qlinear.h."""
    if dY.dim() != 2:
        raise ValueError("dY must be 2-D [M][N]")
    M, N = dY.shape
    f, t = _fmt(fmt), _grad_type(dY, "dY")
    _blocks_fit(blocks, "blocks", f, N, K)
    dev, u8, bf = _device_of(dY, "dY"), torch.uint8, torch.bfloat16
    out = _out(out, "dX", (M, K), bf, dY)
    if workspace is None:
        workspace = dY.new_empty(lib().qmatmul_grad_workspace_bytes(f, M, N, K), dtype=u8)
    args = (f, _ptr(blocks, "blocks", u8, dev), _ptr(dY, "dY", dY.dtype, dev), t, _ptr(out, "dX", bf, dev), M, N, K,
            _ptr(workspace, "workspace", u8, dev), workspace.numel())
    if M:
        _call("qmatmul_grad", dev, *args)
    return out


class GluGrad(NamedTuple):
    """Results of ``qmatmul_glu_grad``, bf16: dX [M][K]; dG and dU [M][F]
    (None where not wanted)."""
    dX: torch.Tensor
    dG: torch.Tensor | None
    dU: torch.Tensor | None


def glu_grad_workspace_bytes(fmt, M: int, F: int, K: int) -> int:
    """Bytes of a workspace for ``qmatmul_glu_grad`` of up to M rows."""
    return int(lib().qmatmul_glu_grad_workspace_bytes(_fmt(fmt), M, F, K))


def qmatmul_glu_grad(fmt, gate_blocks: torch.Tensor, up_blocks: torch.Tensor, X: torch.Tensor, dH: torch.Tensor,
                     act="silu", parts: bool = False, out: GluGrad | None = None,
                     workspace: torch.Tensor | None = None) -> GluGrad:
    """Backward pass of ``qmatmul_glu`` from X bf16 [M][K] and dH fp32 or bf16
    [M][F]: dX = dG . deq(Wg) + dU . deq(Wu) with dG = dH * U * act'(G) and dU =
    dH * act(G); G and U are computed again.  ``parts``: dG and dU are wanted
    too.  ``out``: a GluGrad whose tensors are overwritten (dG and dU that are
    None are not stored)."""
    if X.dim() != 2 or dH.dim() != 2:
        raise ValueError("X must be 2-D [M][K] and dH 2-D [M][F]")
    M, K = X.shape
    F = dH.shape[1]
    _shaped(dH, "dH", (M, F))
    f, t = _fmt(fmt), _grad_type(dH, "dH")
    _blocks_fit(gate_blocks, "gate_blocks", f, F, K)
    _blocks_fit(up_blocks, "up_blocks", f, F, K)
    dev, u8, bf = _device_of(X, "X"), torch.uint8, torch.bfloat16
    if out is None:
        out = GluGrad(X.new_empty((M, K), dtype=bf), X.new_empty((M, F), dtype=bf) if parts else None,
                      X.new_empty((M, F), dtype=bf) if parts else None)
    else:
        for v, name, shape in ((out.dX, "dX", (M, K)), (out.dG, "dG", (M, F)), (out.dU, "dU", (M, F))):
            _shaped(v, name, shape)
    a = ACT[act] if isinstance(act, str) else int(act)
    if workspace is None:
        workspace = X.new_empty(lib().qmatmul_glu_grad_workspace_bytes(f, M, F, K), dtype=u8)
    args = (f, _ptr(gate_blocks, "gate_blocks", u8, dev), _ptr(up_blocks, "up_blocks", u8, dev), _ptr(X, "X", bf, dev),
            _ptr(dH, "dH", dH.dtype, dev), t, _ptr(out.dX, "dX", bf, dev), _ptr(out.dG, "dG", bf, dev),
            _ptr(out.dU, "dU", bf, dev), M, F, K, a, _ptr(workspace, "workspace", u8, dev), workspace.numel())
    if M:
        _call("qmatmul_glu_grad", dev, *args)
    return out


class Xent(NamedTuple):
    """Results of ``qmatmul_xent``: loss [M] fp32, lse [M] fp32, dX [M][K] bf16
    (lse and dX None where not wanted)."""
    loss: torch.Tensor
    lse: torch.Tensor | None
    dX: torch.Tensor | None


def xent_workspace_bytes(fmt, M: int, N: int, K: int, grad: bool = True) -> int:
    """Bytes of a workspace for ``qmatmul_xent`` of up to M rows."""
    return int(lib().qmatmul_xent_workspace_bytes(_fmt(fmt), M, N, K, 1 if grad else 0))


def qmatmul_xent(fmt, blocks: torch.Tensor, X: torch.Tensor, N: int, targets: torch.Tensor,
                 weights: torch.Tensor | None = None, grad: bool = True, out: Xent | None = None,
                 workspace: torch.Tensor | None = None) -> Xent:
    """Softmax cross entropy of ``targets`` (int32 [M]; outside [0, N): not
    scored, loss 0) behind a quantized [N][K] output head, for X bf16 [M][K],
    and its gradient dX = weights[m] * (softmax - onehot) . deq(W) (``weights``:
    fp32 [M], by default 1; they enter dX alone), without holding the logits.
    ``grad=False``: the loss alone.  ``out``: an Xent whose tensors are
    overwritten (lse and dX that are None are not computed)."""
    if X.dim() != 2:
        raise ValueError("X must be 2-D [M][K]")
    M, K = X.shape
    f = _fmt(fmt)
    _blocks_fit(blocks, "blocks", f, N, K)
    _shaped(targets, "targets", (M,))
    _shaped(weights, "weights", (M,))
    dev, u8, bf, f32 = _device_of(X, "X"), torch.uint8, torch.bfloat16, torch.float32
    if out is None:
        out = Xent(X.new_empty(M, dtype=f32), X.new_empty(M, dtype=f32), X.new_empty((M, K), dtype=bf) if grad else None)
    else:
        for v, name, shape in ((out.loss, "loss", (M,)), (out.lse, "lse", (M,)), (out.dX, "dX", (M, K))):
            _shaped(v, name, shape)
    if workspace is None:
        workspace = X.new_empty(lib().qmatmul_xent_workspace_bytes(f, M, N, K, 0 if out.dX is None else 1), dtype=u8)
    args = (f, _ptr(blocks, "blocks", u8, dev), _ptr(X, "X", bf, dev), M, N, K, _ptr(targets, "targets", torch.int32, dev),
            _ptr(weights, "weights", f32, dev), _ptr(out.loss, "loss", f32, dev), _ptr(out.lse, "lse", f32, dev),
            _ptr(out.dX, "dX", bf, dev), _ptr(workspace, "workspace", u8, dev), workspace.numel())
    if M:
        _call("qmatmul_xent", dev, *args)
    return out


def dequantize(fmt, blocks: torch.Tensor, N: int, K: int) -> torch.Tensor:
    """Test aid: exact fp32 [N][K] values of a block buffer."""
    out = torch.empty((N, K), dtype=torch.float32, device=blocks.device)
    _check("q_dequantize", lib().q_dequantize(_fmt(fmt), _dev(blocks, "blocks", torch.uint8), N, K,
                                              _dev(out, "W"), _stream()))
    return out


# ----------------------------------------------------------------------------
# measurement aids (the benchmark's ceilings; not part of the computation)
# ----------------------------------------------------------------------------

def probe_read(buf: torch.Tensor, sink: torch.Tensor):
    """Read every byte of device tensor ``buf`` once (streaming-read ceiling)."""
    n = buf.numel() * buf.element_size()
    _check("q_probe_read", lib().q_probe_read(_dev(buf, "buf"), n, _dev(sink, "sink", torch.float32), _stream()))


def probe_mfma(iters: int, sink: torch.Tensor) -> int:
    """A loop of bf16 MFMAs with no memory traffic; returns its FLOP count."""
    _check("q_probe_mfma", lib().q_probe_mfma(_dev(sink, "sink", torch.float32), iters, _stream()))
    return int(lib().q_probe_mfma_flops(iters))


def probe_mix(iters: int, mode: int, waves_per_simd: int, sink: torch.Tensor):
    """The MFMA loop with 16 fp32 fmas per MFMA, waves_per_simd waves on
    each SIMD: mode 0 MFMAs only, 1 fmas only, 2 both interleaved; returns
    (MFMA FLOP, wave-level fma instructions) of the call."""
    _check("q_probe_mix", lib().q_probe_mix(_dev(sink, "sink", torch.float32), iters, mode, waves_per_simd,
                                            _stream()))
    fmas = int(lib().q_probe_mix_valu(iters, waves_per_simd))
    flops = fmas // 16 * 32 * 32 * 16 * 2 if mode != 1 else 0
    return flops, (fmas if mode != 0 else 0)
