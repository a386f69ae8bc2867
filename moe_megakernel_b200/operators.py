"""Operators around the MoE layer: products grouped by expert, the dense layer
and its gradients, and the orthogonalised update of weight gradients.

Argument checks and marshalling over the C entry points of the same names
(include/moe_b200.h); every step runs in the library's CUDA kernels. Tensors
are bf16 or fp16 on one CUDA device, the last index contiguous, rows a multiple
of 8 elements apart, no extent above 2**30. Work is enqueued on `stream` (default: the current stream
of the tensors' device); nothing synchronises. With a `stream` of its own a call
takes the tensors that it makes (results and scratch) from the allocator on that
stream; its inputs have to be ready there, and a result that another stream goes
on with needs what any tensor needs there: that stream waits, and
``Tensor.record_stream`` if the result may be dropped before that work is done.
`error_word`, an int32 tensor of one element, receives the call's device error
code (0 = none). Results carry no autograd history, whether the inputs require
gradients or not: ``linear_backward``, ``grouped_matmul_wgrad`` and the transposed
``grouped_matmul`` are the backward passes.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence, Union

import torch

from . import MOE_ERR_UNSUPPORTED_SHAPE, MoEError, _counts, load_library

DTYPE_CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
#: Newton-Schulz coefficients (a, b, c) of the quintic a t + b t^3 + c t^5 that drives singular values towards 1.
QUINTIC = (3.4445, -4.7750, 2.0315)


def _tensor(t, name: str, dims: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dims:
        raise ValueError(f"{name}: expected {dims} dimensions, got shape {tuple(t.shape)}")


def _like(t, name: str, shape, dtype, device):
    """Shape, type and device of a tensor; its last index must be contiguous."""
    if (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype == dtype and t.device == device
            and (t.stride(-1) == 1 or shape[-1] <= 1)):
        return
    _tensor(t, name, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    _last(t, name)


def _last(t, name: str):
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the last index must be contiguous")


def _whole(t, name: str, shape, dtype, device):
    _like(t, name, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _pitch(t, name: str) -> int:
    """Row pitch in elements of a [rows, width] tensor; a single row has its own width."""
    rows, width = t.shape
    ld = t.stride(0) if rows > 1 else width
    if rows > 1 and (ld < width or ld % 8):
        raise ValueError(f"{name}: rows must be a multiple of 8 elements apart and not overlap (stride {ld})")
    return ld


def _half(t, name: str) -> int:
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"{name}: expected bfloat16 or float16, got {t.dtype}")
    return DTYPE_CODES[t.dtype]


def _cuda(t, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device, got {t.device}")


def _activation(name) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation: expected one of {sorted(k for k in ACTIVATIONS if k)} or None, got {name!r}")
    return ACTIVATIONS[name]


def _address(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _error_word(t, device):
    if t is not None:
        _whole(t, "error_word", (1,), torch.int32, device)
    return _address(t)


def _raw_stream(stream, device) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    if stream.device != device:
        raise ValueError(f"stream: expected a stream of {device}, got one of {stream.device}")
    return stream.cuda_stream


def _call(name: str, device, *args):
    """The C entry point `name`, with the tensors' device as the current one."""
    f = getattr(load_library(), name)
    if torch._C._cuda_getDevice() == device.index:
        rc = f(*args)
    else:
        with torch.cuda.device(device):
            rc = f(*args)
    if rc:
        raise MoEError(rc, name)


def _new(like, shape, stream, dtype=None):
    """A tensor beside ``like`` from the allocator, for work on ``stream``: taken on that stream, so that
    the memory held nothing which work still queued on another one reads, and so that it is reused only
    behind that stream's work (and belongs to the graph when captured)."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _workspace(nbytes: int, like, stream):
    return _new(like, (nbytes,), stream, torch.uint8) if nbytes else None


def _apart(out, name: str, *inputs):
    """A given result that starts where an input does would be written while the kernel still reads it."""
    if out.numel() and any(t is not None and t.data_ptr() == out.data_ptr() for t in inputs):
        raise ValueError(f"{name} overlaps an input")


def _offsets(offsets, device):
    _tensor(offsets, "offsets", 1)
    groups = offsets.shape[0] - 1
    if groups < 1:
        raise ValueError("offsets: expected groups + 1 >= 2 values")
    _whole(offsets, "offsets", (groups + 1,), torch.int32, device)
    return groups


def grouped_matmul(x: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor, transpose: bool = False,
                   y: Optional[torch.Tensor] = None, error_word: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """y[r] = x[r] @ W[e] for offsets[e] <= r < offsets[e+1]; with ``transpose`` x[r] @ W[e].T.

    x [rows, K], W [groups, K, N] contiguous ([groups, N, K] with ``transpose``), offsets int32
    [groups + 1] on the device, not decreasing (``MoEPlan.routing``'s expert_offset fits; sizes
    need no padding). Rows outside the groups are left as they were in a given y (which overlaps
    no input), undefined in a new one. At most 1024 groups; K and N multiples of 8."""
    _tensor(x, "x", 2)
    _tensor(W, "W", 3)
    dt = _half(x, "x")
    rows, K = x.shape
    dev = x.device
    groups = _offsets(offsets, dev)
    N = W.shape[1] if transpose else W.shape[2]
    _last(x, "x")
    _whole(W, "W", (groups, N, K) if transpose else (groups, K, N), x.dtype, dev)
    _counts("moe_grouped_matmul", rows, groups, K, N)
    _cuda(x, "x")
    if y is None:
        y = _new(x, (rows, N), stream)
    else:
        _like(y, "y", (rows, N), x.dtype, dev)
        _apart(y, "y", x, W)
    _call("moe_grouped_matmul", dev, x.data_ptr(), _pitch(x, "x"), W.data_ptr(), offsets.data_ptr(), rows, groups, K, N,
          1 if transpose else 0, dt, y.data_ptr(), _pitch(y, "y"), _error_word(error_word, dev),
          _raw_stream(stream, dev))
    return y


def grouped_matmul_wgrad(x: torch.Tensor, dy: torch.Tensor, offsets: torch.Tensor,
                         dW: Optional[torch.Tensor] = None, error_word: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """dW[e] = x[rows of e].T @ dy[rows of e], [groups, K, N]; zeros for an empty group.
    (``grouped_matmul(dy, W, offsets, transpose=True)`` is the input gradient.)"""
    _tensor(x, "x", 2)
    _tensor(dy, "dy", 2)
    dt = _half(x, "x")
    rows, K = x.shape
    N = dy.shape[1]
    dev = x.device
    groups = _offsets(offsets, dev)
    _last(x, "x")
    _like(dy, "dy", (rows, N), x.dtype, dev)
    _counts("moe_grouped_matmul_wgrad", rows, groups, K, N)
    _cuda(x, "x")
    if dW is None:
        dW = _new(x, (groups, K, N), stream)
    else:
        _whole(dW, "dW", (groups, K, N), x.dtype, dev)
        _apart(dW, "dW", x, dy)
    _call("moe_grouped_matmul_wgrad", dev, x.data_ptr(), _pitch(x, "x"), dy.data_ptr(), _pitch(dy, "dy"),
          offsets.data_ptr(), rows, groups, K, N, dt, dW.data_ptr(), _error_word(error_word, dev),
          _raw_stream(stream, dev))
    return dW


def linear(x: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None, activation: Optional[str] = None,
           residual: Optional[torch.Tensor] = None, save_preact: bool = False, y: Optional[torch.Tensor] = None,
           preact: Optional[torch.Tensor] = None, error_word: Optional[torch.Tensor] = None, stream=None):
    """act(x @ W + bias) + residual in one kernel: x [T, K], W [K, N], bias [N], residual [T, N].

    activation: None, "relu", "gelu" (erf), "gelu_tanh" or "silu". With ``save_preact`` (or a
    given ``preact``) returns (y, z), z = x @ W + bias as linear_backward takes it. y may be the
    residual itself; given results overlap nothing else."""
    _tensor(x, "x", 2)
    _tensor(W, "W", 2)
    dt, act = _half(x, "x"), _activation(activation)
    T, K = x.shape
    N = W.shape[1]
    dev = x.device
    _last(x, "x")
    _whole(W, "W", (K, N), x.dtype, dev)
    _counts("moe_linear", T, K, N)
    if bias is not None:
        _whole(bias, "bias", (N,), x.dtype, dev)
    if residual is not None:
        _like(residual, "residual", (T, N), x.dtype, dev)
    _cuda(x, "x")
    if y is None:
        y = _new(x, (T, N), stream)
    else:
        _like(y, "y", (T, N), x.dtype, dev)
        _apart(y, "y", x, W, bias, preact)
        if residual is not None and residual.data_ptr() == y.data_ptr() and residual.stride() != y.stride() and T > 1:
            raise ValueError("y overlaps the residual, in rows of another pitch")
    if preact is not None:
        _like(preact, "preact", (T, N), x.dtype, dev)
        _apart(preact, "preact", x, W, bias, residual)
    elif save_preact:
        preact = _new(x, (T, N), stream)
    _call("moe_linear", dev, x.data_ptr(), _pitch(x, "x"), W.data_ptr(), _address(bias), _address(residual),
          0 if residual is None else _pitch(residual, "residual"), T, K, N, act, dt, y.data_ptr(), _pitch(y, "y"),
          _address(preact), 0 if preact is None else _pitch(preact, "preact"), _error_word(error_word, dev),
          _raw_stream(stream, dev))
    return y if preact is None else (y, preact)


def linear_backward(dy: torch.Tensor, x: torch.Tensor, W: torch.Tensor, preact: Optional[torch.Tensor] = None,
                    activation: Optional[str] = None, input_grad: bool = True, weight_grad: bool = True,
                    bias_grad: bool = False, error_word: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of ``linear`` for the upstream dy [T, N]: dict of dx [T, K], dW [K, N] and
    dbias [N] (None where not asked for). preact: the z that linear returned, needed with an
    activation. The residual's gradient is dy itself."""
    _tensor(dy, "dy", 2)
    _tensor(x, "x", 2)
    _tensor(W, "W", 2)
    dt, act = _half(x, "x"), _activation(activation)
    T, K = x.shape
    N = W.shape[1]
    dev = x.device
    _last(x, "x")
    _whole(W, "W", (K, N), x.dtype, dev)
    _like(dy, "dy", (T, N), x.dtype, dev)
    _counts("moe_linear_backward", T, K, N)
    if act and preact is None:
        raise ValueError("preact is needed with an activation")
    z = preact if act else None
    if z is not None:
        _like(z, "preact", (T, N), x.dtype, dev)
    _cuda(x, "x")
    lib = load_library()
    dx = _new(x, (T, K), stream) if input_grad else None
    dW = _new(x, (K, N), stream) if weight_grad else None
    dbias = _new(x, (N,), stream) if bias_grad else None
    nbytes = lib.moe_linear_backward_workspace_bytes(T, N, act, 1 if bias_grad else 0)
    ws = _workspace(nbytes, x, stream)
    _call("moe_linear_backward", dev, dy.data_ptr(), _pitch(dy, "dy"), x.data_ptr(), _pitch(x, "x"), W.data_ptr(),
          _address(z), 0 if z is None else _pitch(z, "preact"), T, K, N, act, dt, _address(dx), K, _address(dW),
          _address(dbias), _address(ws), nbytes, _error_word(error_word, dev), _raw_stream(stream, dev))
    return dict(dx=dx, dW=dW, dbias=dbias)


@functools.lru_cache(maxsize=64)
def _schedule(steps: int, coeffs: tuple):
    """The steps' coefficients as the C array [steps, 3] (read during the call only)."""
    rows = list(coeffs) if coeffs and isinstance(coeffs[0], tuple) else [coeffs] * steps
    if len(rows) != steps or any(not isinstance(r, tuple) or len(r) != 3 for r in rows):
        raise ValueError("coeffs: expected (a, b, c), or one such triple for each step")
    return (ctypes.c_float * (3 * steps))(*[float(v) for r in rows for v in r])


def orthogonalize(G: torch.Tensor, steps: int = 5,
                  coeffs: Union[Sequence[float], Sequence[Sequence[float]]] = QUINTIC, eps: float = 1e-7,
                  out: Optional[torch.Tensor] = None, error_word: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Newton-Schulz orthogonalisation of G [m, n] or of every matrix of G [batch, m, n]
    (weight gradients: ``MoEPlan.backward``'s dW1, dW3, dW2, ``grouped_matmul_wgrad``'s or
    ``linear_backward``'s dW). X = G / (|G|_F + eps), then ``steps`` times
    X <- a X + (b A + c A A) X with A = X X^T (the short side inside). G bf16 or fp32 of any size
    and row pitch; returns bf16 of G's shape (out may be a bf16 G itself). coeffs: one (a, b, c) for all
    steps, or one per step. The entries of A and b A + c A A have to stay below 32 in magnitude (with
    QUINTIC they stay below 7): they pass through fp16, and larger ones give infinities or NaN."""
    if not isinstance(G, torch.Tensor):
        raise TypeError("G must be a torch.Tensor")
    if G.dim() not in (2, 3) or G.shape[-1] < 1 or G.shape[-2] < 1:
        raise ValueError(f"G: expected [m, n] or [batch, m, n], got {tuple(G.shape)}")
    if G.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"G: expected bfloat16 or float32, got {G.dtype}")
    if steps < 1:
        raise ValueError("steps must be at least 1")
    batch, m, n = G.shape if G.dim() == 3 else (1, *G.shape)
    _counts("moe_orthogonalize", batch, m, n)
    if steps > 64:
        raise MoEError(MOE_ERR_UNSUPPORTED_SHAPE, "moe_orthogonalize")
    flat = _schedule(steps, tuple(tuple(c) if isinstance(c, (list, tuple)) else c for c in coeffs))
    _last(G, "G")
    _cuda(G, "G")
    dev = G.device
    if out is None:
        out = _new(G, G.shape, stream, torch.bfloat16)
    else:
        _like(out, "out", tuple(G.shape), torch.bfloat16, dev)

    def pitches(t, name):
        t = t if t.dim() == 3 else t.unsqueeze(0)
        ld = t.stride(1) if t.shape[1] > 1 else t.shape[2]
        bs = t.stride(0) if t.shape[0] > 1 else ld * t.shape[1]
        if ld < t.shape[2] or (t.shape[0] > 1 and bs < ld * (t.shape[1] - 1) + t.shape[2]):
            raise ValueError(f"{name}: rows or matrices overlap")
        return ld, bs

    lib = load_library()
    nbytes = lib.moe_orthogonalize_workspace_bytes(batch, m, n)
    ws = _workspace(nbytes, G, stream)
    _call("moe_orthogonalize", dev, G.data_ptr(), *pitches(G, "G"), batch, m, n, DTYPE_CODES[G.dtype], steps, flat, eps,
          out.data_ptr(), *pitches(out, "out"), _address(ws), nbytes, _error_word(error_word, dev),
          _raw_stream(stream, dev))
    return out
