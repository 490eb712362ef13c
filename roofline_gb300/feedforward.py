"""The gated feed-forward layer on torch tensors: the block and its gradients,
products with 4-bit weights for a few tokens, and gradient clipping.

Argument marshalling only, like ``gemm``: everything is computed by the
kernels of libgb300gemm.so (see include/gb300_gemm.h for the formulas and the
rules of each call).  Tensors are torch CUDA tensors, float32 or bfloat16.
The checks of the tensors are native (csrc/torch_binding.cpp); a tensor of
the wrong shape, type, device or storage raises ValueError, what the library
refuses raises ``gemm.GemmError``.

``stream``: the torch.cuda.Stream to launch on (None: torch's current one).  As
with torch's own operators its order with the streams that made the inputs, or
that use the outputs, is the caller's part; new outputs are of the given
stream's memory, so nothing before the call uses them.

No call records a graph for autograd: outputs require no gradient, whatever the
inputs do.  What is written in place or into ``out`` counts as modified.

``workspace``: optional contiguous CUDA tensor used as scratch
(``gated_ff_workspace`` or ``grad_norm_workspace`` bytes, which no other work
uses at the time).  Without one a call takes its own from torch's allocator, on
the stream that it runs on: calls on several streams share nothing, and a
captured graph keeps its own.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

from . import build as _build
from . import gemm
from .gemm import GemmError, OK, OP_N

DT_F32 = 0
DT_BF16 = 1
ACT_SILU = 0
ACT_GELU = 1
ACT_GELU_TANH = 2
ACT_RELU = 3
ACTS = {"silu": ACT_SILU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH, "relu": ACT_RELU}

_module = None


def _native():
    """The native module (loaded once).  Raises if it has not been built."""
    global _module
    if _module is None:
        if not os.path.exists(_build.BINDING):
            raise RuntimeError(f"{_build.BINDING} is missing: build it with "
                               "`python -m roofline_gb300.build` (there is no CPU fallback)")
        import torch  # noqa: F401  (the module's own libraries)
        gemm.load()
        spec = importlib.util.spec_from_file_location("_ff_native", _build.BINDING)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _module = module
    return _module


def _act(act) -> int:
    code = ACTS.get(act, act)
    if isinstance(code, str):
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACTS)}")
    return code


def _handle(stream):
    """The handle of the stream to launch on; None for torch's current one."""
    return None if stream is None else stream.cuda_stream


def gated_ff(X, Wg, Wu, act="silu", save=False, out=None, stream=None, workspace=None):
    """H = act(X @ Wg) * (X @ Wu): X is M x D, the weights D x F (a stored
    F x D weight is passed as ``W.t()``, without a copy).  Returns H, or with
    ``save`` (H, G, U), where G = X @ Wg and U = X @ Wu, in float32, are what
    ``gated_ff_backward`` reads."""
    return (_module or _native()).gated_ff(X, Wg, Wu, _act(act), bool(save), out, _handle(stream),
                                           workspace)


def gated_ff_backward(dH, X, Wg, Wu, G, U, act="silu", need_dx=True, need_dw=True, stream=None,
                      workspace=None):
    """(dX, dWg, dWu) of ``gated_ff`` from dH and the saved G and U.  The
    weights' gradients are stored as the weights are (for a weight passed as
    ``W.t()``, dWg.t() is the contiguous F x D gradient of W).  What is not
    needed is None."""
    return (_module or _native()).gated_ff_backward(dH, X, Wg, Wu, G, U, _act(act), bool(need_dx),
                                                    bool(need_dw), _handle(stream), workspace)


def gated_ff_workspace(M, D, F, dtype, op_w=OP_N, backward=False, aligned=False) -> int:
    """Scratch bytes a call of these sizes may need (dtype: DT_F32 or DT_BF16)."""
    out = ctypes.c_uint64(0)
    rc = gemm.load().gated_ff_workspace(1 if backward else 0, dtype, op_w, M, D, F,
                                        1 if aligned else 0, ctypes.byref(out))
    if rc != OK:
        raise GemmError(rc, "gated_ff_workspace")
    return out.value


def q4_matmul(X, Wq, scales, zeros=None, group=128, out=None, stream=None):
    """Y = X @ W.t() with W (N x K) in 4-bit codes: Wq uint8 N x ceil(K/2), the
    even column's code in the low half of each byte; W(n,k) =
    scales(n, k // group) * (code - zeros(n, k // group)), zeros 8 when None."""
    return (_module or _native()).q4_matmul(X, Wq, scales, zeros, group, out, _handle(stream))


def q4_gated(X, Wq_g, scales_g, Wq_u, scales_u, zeros_g=None, zeros_u=None, group=128,
             act="silu", out=None, stream=None):
    """H = act(X @ Wg.t()) * (X @ Wu.t()), both weights in the format of ``q4_matmul``."""
    return (_module or _native()).q4_gated(X, Wq_g, scales_g, zeros_g, Wq_u, scales_u, zeros_u,
                                           group, _act(act), out, _handle(stream))


def grad_norm(grads, stream=None, workspace=None):
    """sqrt of the sum of squares over all tensors, as a 0-d float32 tensor."""
    return (_module or _native()).grad_norm_clip(list(grads), None, 0.0, _handle(stream),
                                                 workspace)


def grad_norm_workspace(count) -> int:
    """Scratch bytes of ``grad_norm`` and ``clip_grad_norm`` of `count` tensors."""
    return int(gemm.load().grad_norm_clip_workspace(count))


def clip_grad_norm(grads, max_norm, out=None, stream=None, workspace=None):
    """Scales every tensor by min(1, max_norm / (norm + 1e-6)) and returns the
    norm before clipping.  In place, or into the tensors ``out``.  Tensors are
    dense in any order of their dimensions (as ``gated_ff_backward`` returns the
    gradients of a weight passed as ``W.t()``); an ``out`` has its gradient's."""
    grads = list(grads)
    return (_module or _native()).grad_norm_clip(grads, grads if out is None else list(out),
                                                 max_norm, _handle(stream), workspace)
