"""The gated feed-forward layer on torch tensors: the block and its gradients,
products with 4-bit weights for a few tokens, and gradient clipping.

Argument marshalling only, like ``gemm``: everything is computed by the
kernels of libgb300gemm.so (see include/gb300_gemm.h for the formulas and the
rules of each call).  Tensors are torch CUDA tensors, float32 or bfloat16.
"""
from __future__ import annotations

import ctypes

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


_DTYPES = {}


def _dtype(t) -> int:
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: DT_F32, torch.bfloat16: DT_BF16})
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"dtype {t.dtype}: float32 or bfloat16 wanted")
    return d


def _rows(t, name, like=None, shape=None, dtype=None):
    """Leading dimension of a row-major 2-D CUDA tensor."""
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    if like is not None and (t.dtype != (dtype or like.dtype) or t.device != like.device):
        raise ValueError(f"{name} must be {dtype or like.dtype} on the first operand's device")
    r, c = t.shape
    if shape is not None and (r, c) != shape:
        raise ValueError(f"{name} is {r} x {c}, {shape[0]} x {shape[1]} wanted")
    s0, s1 = t.stride()
    if s1 != 1 and c > 1:
        raise ValueError(f"{name} must have unit column stride")
    # the row stride of a one-row matrix is never used
    return max(s0 if r > 1 else c, 1)


def _weight(t, name, like, D, F):
    """{op: ld} of the ways a D x F weight can be read: row-major is op N,
    ``W.t()`` of a stored F x D matrix op T (one row or column may be either)."""
    if not t.is_cuda or t.dim() != 2 or t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must be a 2-D CUDA tensor of the first operand's dtype and device")
    if tuple(t.shape) != (D, F):
        raise ValueError(f"{name} is {tuple(t.shape)}, {(D, F)} wanted")
    s0, s1 = t.stride()
    ops = {}
    if s1 == 1 or F <= 1:
        ops[OP_N] = max(s0 if D > 1 else F, 1)
    if s0 == 1 or D <= 1:
        ops[OP_T] = max(s1 if F > 1 else D, 1)
    if not ops:
        raise ValueError(f"{name} must have a unit row or column stride")
    return ops


def _weights(Wg, Wu, like, D, F):
    g, u = _weight(Wg, "Wg", like, D, F), _weight(Wu, "Wu", like, D, F)
    for op in (OP_N, OP_T):
        if op in g and op in u:
            return op, g[op], u[op]
    raise ValueError("Wg and Wu must be stored in the same order")


def _stream(stream, *new):
    """The handle to launch on.  Tensors made here on torch's current stream
    and used on another are told so, for the caching allocator."""
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    for t in new:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


def _workspace(w):
    return (None, 0) if w is None else (w.data_ptr(), w.numel() * w.element_size())


def _check(rc, what):
    if rc != OK:
        raise GemmError(rc, what)


def gated_ff(X, Wg, Wu, act="silu", save=False, out=None, stream=None, workspace=None):
    """H = act(X @ Wg) * (X @ Wu): X is M x D, the weights D x F (a stored
    F x D weight is passed as ``W.t()``, without a copy).  Returns H, or with
    ``save`` (H, G, U), where G = X @ Wg and U = X @ Wu, in float32, are what
    ``gated_ff_backward`` reads.  ``workspace``: as for ``gemm.matmul``
    (``gated_ff_workspace`` bytes)."""
    import torch
    M, D = X.shape
    F = Wg.shape[1]
    dt, ldx = _dtype(X), _rows(X, "X")
    op, ldg, ldu = _weights(Wg, Wu, X, D, F)
    H = torch.empty((M, F), dtype=X.dtype, device=X.device) if out is None else out
    ldh = F if out is None else _rows(out, "out", X, (M, F))
    G = U = None
    if save:
        G = torch.empty((M, F), dtype=torch.float32, device=X.device)
        U = torch.empty((M, F), dtype=torch.float32, device=X.device)
    ws, wsb = _workspace(workspace)
    _check(gemm.load().gated_ff(
        dt, _act(act), op, M, D, F, X.data_ptr(), ldx, Wg.data_ptr(), ldg, Wu.data_ptr(), ldu,
        H.data_ptr(), max(ldh, 1), G.data_ptr() if save else None, max(F, 1),
        U.data_ptr() if save else None, max(F, 1), ws, wsb,
        _stream(stream, None if out is not None else H, G, U)), "gated_ff")
    return (H, G, U) if save else H


def gated_ff_backward(dH, X, Wg, Wu, G, U, act="silu", need_dx=True, need_dw=True, stream=None,
                      workspace=None):
    """(dX, dWg, dWu) of ``gated_ff`` from dH and the saved G and U.  The
    weights' gradients are stored as the weights are (for a weight passed as
    ``W.t()``, dWg.t() is the contiguous F x D gradient of W).  What is not
    needed is None."""
    import torch
    M, D = X.shape
    F = Wg.shape[1]
    dt, ldx = _dtype(X), _rows(X, "X")
    op, ldg, ldu = _weights(Wg, Wu, X, D, F)
    lds = [_rows(dH, "dH", X, (M, F)), _rows(G, "G", X, (M, F), torch.float32),
           _rows(U, "U", X, (M, F), torch.float32)]
    dX = dWg = dWu = None
    if need_dx:
        dX = torch.empty((M, D), dtype=X.dtype, device=X.device)
    if need_dw:
        shape = (D, F) if op == OP_N else (F, D)
        dWg = torch.empty(shape, dtype=X.dtype, device=X.device)
        dWu = torch.empty(shape, dtype=X.dtype, device=X.device)
    ldw = max(F if op == OP_N else D, 1)
    ws, wsb = _workspace(workspace)
    if need_dx or need_dw:
        _check(gemm.load().gated_ff_backward(
            dt, _act(act), op, M, D, F, dH.data_ptr(), lds[0], X.data_ptr(), ldx, Wg.data_ptr(),
            ldg, Wu.data_ptr(), ldu, G.data_ptr(), lds[1], U.data_ptr(), lds[2],
            dX.data_ptr() if need_dx else None, max(D, 1), dWg.data_ptr() if need_dw else None,
            ldw, dWu.data_ptr() if need_dw else None, ldw, ws, wsb,
            _stream(stream, dX, dWg, dWu)), "gated_ff_backward")
    if need_dw and op == OP_T:
        dWg, dWu = dWg.t(), dWu.t()
    return dX, dWg, dWu


def gated_ff_workspace(M, D, F, dtype, op_w=OP_N, backward=False, aligned=False) -> int:
    """Scratch bytes a call of these sizes may need (dtype: DT_F32 or DT_BF16)."""
    out = ctypes.c_uint64(0)
    _check(gemm.load().gated_ff_workspace(1 if backward else 0, dtype, op_w, M, D, F,
                                          1 if aligned else 0, ctypes.byref(out)),
           "gated_ff_workspace")
    return out.value


def _q4_side(q, s, z, like, K, group, name):
    """(q, ldq, s, z) addresses of one quantised matrix, checked against K and group."""
    N = q.shape[0]
    if not q.is_cuda or q.dim() != 2 or q.element_size() != 1 or q.shape[1] != (K + 1) // 2:
        raise ValueError(f"{name} must be an N x {(K + 1) // 2} uint8 CUDA tensor")
    if q.shape[1] > 1 and q.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    groups = -(-K // group)
    for t, what in ((s, "scales"), (z, "zeros")):
        if t is not None and (t.dtype != like.dtype or not t.is_cuda or
                              tuple(t.shape) != (N, groups) or not t.is_contiguous()):
            raise ValueError(f"{what} of {name} must be contiguous, {N} x {groups}, of X's dtype")
    ldq = q.stride(0) if N > 1 else q.shape[1]
    return q.data_ptr(), max(ldq, 1), s.data_ptr(), None if z is None else z.data_ptr()


def q4_matmul(X, Wq, scales, zeros=None, group=128, out=None, stream=None):
    """Y = X @ W.t() with W (N x K) in 4-bit codes: Wq uint8 N x ceil(K/2), the
    even column's code in the low half of each byte; W(n,k) =
    scales(n, k // group) * (code - zeros(n, k // group)), zeros 8 when None."""
    import torch
    M, K = X.shape
    N = Wq.shape[0]
    if group <= 0:
        raise ValueError("group must be positive")
    w = _q4_side(Wq, scales, zeros, X, K, group, "Wq")
    Y = torch.empty((M, N), dtype=X.dtype, device=X.device) if out is None else out
    ldy = max(N, 1) if out is None else _rows(out, "out", X, (M, N))
    _check(gemm.load().q4_matmul(_dtype(X), M, N, K, X.data_ptr(), _rows(X, "X"), *w, group,
                                 Y.data_ptr(), ldy, _stream(stream, None if out is not None else Y)),
           "q4_matmul")
    return Y


def q4_gated(X, Wq_g, scales_g, Wq_u, scales_u, zeros_g=None, zeros_u=None, group=128,
             act="silu", out=None, stream=None):
    """H = act(X @ Wg.t()) * (X @ Wu.t()), both weights in the format of ``q4_matmul``."""
    import torch
    M, K = X.shape
    N = Wq_g.shape[0]
    if group <= 0:
        raise ValueError("group must be positive")
    if Wq_u.shape[0] != N:
        raise ValueError("Wq_g and Wq_u must have the same number of rows")
    g = _q4_side(Wq_g, scales_g, zeros_g, X, K, group, "Wq_g")
    u = _q4_side(Wq_u, scales_u, zeros_u, X, K, group, "Wq_u")
    H = torch.empty((M, N), dtype=X.dtype, device=X.device) if out is None else out
    ldh = max(N, 1) if out is None else _rows(out, "out", X, (M, N))
    _check(gemm.load().q4_gated(_dtype(X), _act(act), M, N, K, X.data_ptr(), _rows(X, "X"), *g,
                                *u, group, H.data_ptr(), ldh,
                                _stream(stream, None if out is not None else H)), "q4_gated")
    return H


def _tensors(ts, name):
    """(addresses, sizes, dtypes) of a list of contiguous CUDA tensors."""
    for t in ts:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous CUDA tensors")
    return [t.data_ptr() for t in ts], [t.numel() for t in ts], [_dtype(t) for t in ts]


def _norm_clip(grads, max_norm, outs, stream, workspace):
    import torch
    n = len(grads)
    ptrs, sizes, dts = _tensors(grads, "grads")
    optrs = None
    if outs is not None:
        if outs is grads:
            optrs = ptrs
        else:
            optrs, osizes, odts = _tensors(outs, "out")
            if osizes != sizes or odts != dts:
                raise ValueError("out must match grads in number, sizes and dtypes")
    device = grads[0].device if n else "cuda"
    norm = torch.empty((), dtype=torch.float32, device=device)
    vp, i64 = ctypes.c_void_p * n, ctypes.c_int64 * n
    ws, wsb = _workspace(workspace)
    _check(gemm.load().grad_norm_clip(n, (ctypes.c_int * n)(*dts), vp(*ptrs),
                                      None if optrs is None else vp(*optrs), i64(*sizes),
                                      float(max_norm), norm.data_ptr(), ws, wsb,
                                      _stream(stream, norm)), "grad_norm_clip")
    return norm


def grad_norm(grads, stream=None, workspace=None):
    """sqrt of the sum of squares over all tensors, as a 0-d float32 tensor."""
    return _norm_clip(grads, 0.0, None, stream, workspace)


def clip_grad_norm(grads, max_norm, out=None, stream=None, workspace=None):
    """Scales every tensor by min(1, max_norm / (norm + 1e-6)) and returns the
    norm before clipping.  In place, or into the tensors ``out``."""
    grads = list(grads)
    return _norm_clip(grads, max_norm, grads if out is None else list(out), stream, workspace)
