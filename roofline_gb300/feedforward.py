"""The gated feed-forward layer on torch tensors: the block and its gradients,
products with 4-bit weights for a few tokens, and gradient clipping.

Argument marshalling only, like ``gemm``: everything is computed by the
kernels of libgb300gemm.so (see include/gb300_gemm.h for the formulas and the
rules of each call).  Tensors are torch CUDA tensors, float32 or bfloat16.
"""
from __future__ import annotations

import ctypes
from array import array

import torch

from . import gemm
from .gemm import GemmError, OK, OP_N, OP_T

DT_F32 = 0
DT_BF16 = 1
ACT_SILU = 0
ACT_GELU = 1
ACT_GELU_TANH = 2
ACT_RELU = 3
ACTS = {"silu": ACT_SILU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH, "relu": ACT_RELU}


def _act(act) -> int:
    if isinstance(act, str):
        if act not in ACTS:
            raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACTS)}")
        return ACTS[act]
    return int(act)


_DTYPES = {torch.float32: DT_F32, torch.bfloat16: DT_BF16}


def _dtype(t) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"dtype {t.dtype}: float32 or bfloat16 wanted")
    return d


def _rows(t, name, rows, cols, dtype, device):
    """Leading dimension of a row-major rows x cols matrix."""
    if t.shape != (rows, cols) or t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name} must be {rows} x {cols}, {dtype}, on CUDA device {device}: got "
                         f"{tuple(t.shape)}, {t.dtype}, {t.device}")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    # the row stride of a one-row matrix is never used
    return (s0 if rows > 1 else cols) or 1


def _first(t, name):
    """(rows, cols, leading dimension, dtype code, device index) of the matrix that sets them."""
    device = t.get_device()
    if device < 0 or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    rows, cols = t.shape
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    # the row stride of a one-row matrix is never used
    return rows, cols, (s0 if rows > 1 else cols) or 1, _dtype(t), device


def _weight(t, name, D, F, dtype, device):
    """{op: ld} of the ways a D x F weight can be read: row-major is op N,
    ``W.t()`` of a stored F x D matrix op T (one row or column may be either)."""
    if t.shape != (D, F) or t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name} must be {D} x {F}, {dtype}, on CUDA device {device}: got "
                         f"{tuple(t.shape)}, {t.dtype}, {t.device}")
    s0, s1 = t.stride()
    ops = {}
    if s1 == 1 or F <= 1:
        ops[OP_N] = (s0 if D > 1 else F) or 1
    if s0 == 1 or D <= 1:
        ops[OP_T] = (s1 if F > 1 else D) or 1
    if not ops:
        raise ValueError(f"{name} must have a unit row or column stride")
    return ops


def _weights(Wg, Wu, D, dtype, device):
    """(F, op, ld of Wg, ld of Wu)."""
    if Wg.dim() != 2:
        raise ValueError("Wg must be a 2-D tensor")
    F = Wg.shape[1]
    g, u = _weight(Wg, "Wg", D, F, dtype, device), _weight(Wu, "Wu", D, F, dtype, device)
    for op in (OP_N, OP_T):
        if op in g and op in u:
            return F, op, g[op], u[op]
    raise ValueError("Wg and Wu must be stored in the same order")


def _matrix(rows, cols, dtype, device, order=OP_N, pad=False):
    """A new rows x cols matrix, row-major or (OP_T) the transpose of one;
    ``pad``: with rows on 16-byte boundaries."""
    ld = -(-cols // 8) * 8 if pad else cols
    return torch.empty_strided((rows, cols), (ld, 1) if order == OP_N else (1, rows), dtype=dtype,
                               device=device)


def _stream(stream, device, *new):
    """The handle to launch on.  Tensors made here on torch's current stream
    and used on another are told so, for the caching allocator."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    for t in new:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


def _workspace(w):
    return (None, 0) if w is None else (w.data_ptr(), w.numel() * w.element_size())


def _lib():
    return gemm._lib or gemm.load()


def _check(rc, what):
    if rc != OK:
        raise GemmError(rc, what)


def gated_ff(X, Wg, Wu, act="silu", save=False, out=None, stream=None, workspace=None):
    """H = act(X @ Wg) * (X @ Wu): X is M x D, the weights D x F (a stored
    F x D weight is passed as ``W.t()``, without a copy).  Returns H, or with
    ``save`` (H, G, U), where G = X @ Wg and U = X @ Wu, in float32, are what
    ``gated_ff_backward`` reads.  ``workspace``: as for ``gemm.matmul``
    (``gated_ff_workspace`` bytes)."""
    M, D, ldx, dt, dev = _first(X, "X")
    dtype, device = X.dtype, X.device
    F, op, ldwg, ldwu = _weights(Wg, Wu, D, dtype, dev)
    H = _matrix(M, F, dtype, device) if out is None else out
    ldh = (F or 1) if out is None else _rows(out, "out", M, F, dtype, dev)
    G = U = g = u = None
    if save:
        G = _matrix(M, F, torch.float32, device, pad=True)
        U = _matrix(M, F, torch.float32, device, pad=True)
        g, u = G.data_ptr(), U.data_ptr()
    lds = -(-(F or 1) // 8) * 8
    ws, wsb = _workspace(workspace)
    rc = _lib().gated_ff(dt, _act(act), op, M, D, F, X.data_ptr(), ldx, Wg.data_ptr(), ldwg,
                         Wu.data_ptr(), ldwu, H.data_ptr(), ldh, g, lds, u, lds, ws, wsb,
                         _stream(stream, dev, None if out is not None else H, G, U))
    _check(rc, "gated_ff")
    return (H, G, U) if save else H


def gated_ff_backward(dH, X, Wg, Wu, G, U, act="silu", need_dx=True, need_dw=True, stream=None,
                      workspace=None):
    """(dX, dWg, dWu) of ``gated_ff`` from dH and the saved G and U.  The
    weights' gradients are stored as the weights are (for a weight passed as
    ``W.t()``, dWg.t() is the contiguous F x D gradient of W).  What is not
    needed is None."""
    M, D, ldx, dt, dev = _first(X, "X")
    dtype, device = X.dtype, X.device
    F, op, ldwg, ldwu = _weights(Wg, Wu, D, dtype, dev)
    ldh = _rows(dH, "dH", M, F, dtype, dev)
    ldg = _rows(G, "G", M, F, torch.float32, dev)
    ldu = _rows(U, "U", M, F, torch.float32, dev)
    dX = dWg = dWu = dx = dg = du = None
    if need_dx:
        dX = _matrix(M, D, dtype, device)
        dx = dX.data_ptr()
    if need_dw:
        dWg, dWu = _matrix(D, F, dtype, device, op), _matrix(D, F, dtype, device, op)
        dg, du = dWg.data_ptr(), dWu.data_ptr()
    ldw = (F if op == OP_N else D) or 1
    ws, wsb = _workspace(workspace)
    if need_dx or need_dw:
        rc = _lib().gated_ff_backward(
            dt, _act(act), op, M, D, F, dH.data_ptr(), ldh, X.data_ptr(), ldx, Wg.data_ptr(),
            ldwg, Wu.data_ptr(), ldwu, G.data_ptr(), ldg, U.data_ptr(), ldu, dx, D or 1, dg, ldw,
            du, ldw, ws, wsb, _stream(stream, dev, dX, dWg, dWu))
        _check(rc, "gated_ff_backward")
    return dX, dWg, dWu


def gated_ff_workspace(M, D, F, dtype, op_w=OP_N, backward=False, aligned=False) -> int:
    """Scratch bytes a call of these sizes may need (dtype: DT_F32 or DT_BF16)."""
    out = ctypes.c_uint64(0)
    _check(_lib().gated_ff_workspace(1 if backward else 0, dtype, op_w, M, D, F,
                                          1 if aligned else 0, ctypes.byref(out)),
           "gated_ff_workspace")
    return out.value


def _q4_side(q, s, z, N, K, groups, dtype, device, name):
    """(ldq, address of the zero points) of one quantised matrix, checked."""
    width = (K + 1) // 2
    if q.shape != (N, width) or q.dtype is not torch.uint8 or q.get_device() != device:
        raise ValueError(f"{name} must be {N} x {width}, uint8, on CUDA device {device}")
    ldq, one = q.stride()
    if one != 1 and width > 1:
        raise ValueError(f"{name} must have unit column stride")
    for t in (s,) if z is None else (s, z):
        if (t.shape != (N, groups) or t.dtype is not dtype or t.get_device() != device or
                not t.is_contiguous()):
            raise ValueError(f"scales and zeros of {name} must be {N} x {groups}, contiguous, "
                             f"{dtype}, on CUDA device {device}")
    return (ldq if N > 1 else width) or 1, None if z is None else z.data_ptr()


def q4_matmul(X, Wq, scales, zeros=None, group=128, out=None, stream=None):
    """Y = X @ W.t() with W (N x K) in 4-bit codes: Wq uint8 N x ceil(K/2), the
    even column's code in the low half of each byte; W(n,k) =
    scales(n, k // group) * (code - zeros(n, k // group)), zeros 8 when None."""
    M, K, ldx, dt, dev = _first(X, "X")
    if group <= 0 or Wq.dim() != 2:
        raise ValueError("group must be positive and Wq a 2-D tensor")
    N, dtype = Wq.shape[0], X.dtype
    ldq, z = _q4_side(Wq, scales, zeros, N, K, -(-K // group), dtype, dev, "Wq")
    if out is None:
        Y, ldy = torch.empty((M, N), dtype=dtype, device=X.device), N or 1
    else:
        Y, ldy = out, _rows(out, "out", M, N, dtype, dev)
    rc = _lib().q4_matmul(dt, M, N, K, X.data_ptr(), ldx, Wq.data_ptr(), ldq, scales.data_ptr(), z,
                          group, Y.data_ptr(), ldy,
                          _stream(stream, dev, None if out is not None else Y))
    if rc:
        _check(rc, "q4_matmul")
    return Y


def q4_gated(X, Wq_g, scales_g, Wq_u, scales_u, zeros_g=None, zeros_u=None, group=128,
             act="silu", out=None, stream=None):
    """H = act(X @ Wg.t()) * (X @ Wu.t()), both weights in the format of ``q4_matmul``."""
    M, K, ldx, dt, dev = _first(X, "X")
    if group <= 0 or Wq_g.dim() != 2:
        raise ValueError("group must be positive and Wq_g a 2-D tensor")
    N, dtype, groups = Wq_g.shape[0], X.dtype, -(-K // group)
    ldg, zg = _q4_side(Wq_g, scales_g, zeros_g, N, K, groups, dtype, dev, "Wq_g")
    ldu, zu = _q4_side(Wq_u, scales_u, zeros_u, N, K, groups, dtype, dev, "Wq_u")
    if out is None:
        H, ldh = torch.empty((M, N), dtype=dtype, device=X.device), N or 1
    else:
        H, ldh = out, _rows(out, "out", M, N, dtype, dev)
    rc = _lib().q4_gated(dt, _act(act), M, N, K, X.data_ptr(), ldx, Wq_g.data_ptr(), ldg,
                         scales_g.data_ptr(), zg, Wq_u.data_ptr(), ldu, scales_u.data_ptr(), zu,
                         group, H.data_ptr(), ldh,
                         _stream(stream, dev, None if out is not None else H))
    if rc:
        _check(rc, "q4_gated")
    return H


def _tensors(ts, name):
    """(device, addresses, sizes, dtype codes) of a list of contiguous CUDA tensors."""
    if not all(map(torch.Tensor.is_contiguous, ts)):
        raise ValueError(f"{name} must be contiguous tensors")
    devices = set(map(torch.Tensor.get_device, ts))
    if len(devices) > 1 or -1 in devices:
        raise ValueError(f"{name} must be CUDA tensors of one device")
    try:
        dts = [_DTYPES[t.dtype] for t in ts]
    except KeyError as e:
        raise ValueError(f"dtype {e.args[0]} in {name}: float32 or bfloat16 wanted") from None
    return (devices.pop() if devices else None, array("Q", map(torch.Tensor.data_ptr, ts)),
            array("q", map(torch.Tensor.numel, ts)), array("i", dts))


def _norm_clip(grads, max_norm, outs, stream, workspace):
    device, ptrs, sizes, dts = _tensors(grads, "grads")
    optrs = None
    if outs is grads:
        optrs = ptrs
    elif outs is not None:
        odev, optrs, osizes, odts = _tensors(outs, "out")
        if odev != device or osizes != sizes or odts != dts:
            raise ValueError("out must match grads in number, sizes, dtypes and device")
    if device is None:
        device = torch.cuda.current_device()
    norm = torch.empty((), dtype=torch.float32, device=f"cuda:{device}")
    at = lambda a: None if a is None else a.buffer_info()[0]  # noqa: E731
    ws, wsb = _workspace(workspace)
    _check(_lib().grad_norm_clip(len(ptrs), at(dts), at(ptrs), at(optrs), at(sizes),
                                 float(max_norm), norm.data_ptr(), ws, wsb,
                                 _stream(stream, device, norm)), "grad_norm_clip")
    return norm


def grad_norm(grads, stream=None, workspace=None):
    """sqrt of the sum of squares over all tensors, as a 0-d float32 tensor."""
    return _norm_clip(list(grads), 0.0, None, stream, workspace)


def clip_grad_norm(grads, max_norm, out=None, stream=None, workspace=None):
    """Scales every tensor by min(1, max_norm / (norm + 1e-6)) and returns the
    norm before clipping.  In place, or into the tensors ``out``."""
    grads = list(grads)
    return _norm_clip(grads, max_norm, grads if out is None else list(out), stream, workspace)
