"""Operators around a language model's products: the norm before them, in their types or in 8 bits, and the loss over
the vocabulary behind them, with their gradients; and the adapters of many requests beside one.

A binding over the C ABI of ``include/fp4g_lm.h`` in the manner of the package's other
functions: each has the name of its C entry point, checks its torch arguments, runs on the
current stream of their GPU and raises ``Fp4GemmError`` on a non-zero status.  The checks and
the calls are compiled (``binding/lm_binding.cpp``).

Layouts (contiguous, all on one GPU):
  rms_norm           : X [rows, K] float32 or bfloat16, weight [K] float32 or bfloat16 -> Y like X
  rms_norm_quantize  : the same -> codes [rows, K] int8 or uint8 (E4M3), scales [rows] float32
  rms_norm_backward  : the gradients of rms_norm
  cross_entropy_gemm           : X [M, K], W [V, K] bfloat16, target [M] int64 -> loss [M] float32
  cross_entropy_gemm_backward  : the gradients of cross_entropy_gemm, bfloat16
  adapter_gemm       : base [M, N] float32 or bfloat16, X [M, K], A [L, R, K], B [L, N, R] bfloat16, index [M] int32
                       -> D like base
K of the loss and K and R of the adapters are multiples of 8.  rms_norm and cross_entropy_gemm take part in autograd, in
reverse mode (a forward-mode tangent raises NotImplementedError); the results of the other functions carry no graph.  The functions themselves may be captured into a graph at any time; a backward pass of autograd
only while no eager graph of the same leaves is alive, as everywhere in torch.
"""
from __future__ import annotations

import ctypes
import functools
import importlib

import torch

import block_scaled_precision_e2m1_amd as _base

LM_SYMBOLS = ("rms_norm", "rms_norm_quantize", "rms_norm_backward_workspace_size", "rms_norm_backward",
              "cross_entropy_gemm_workspace_size", "cross_entropy_gemm", "cross_entropy_gemm_backward_workspace_size",
              "cross_entropy_gemm_backward", "adapter_gemm_workspace_size", "adapter_gemm")

__all__ = [*LM_SYMBOLS, "LM_SYMBOLS"]


@functools.lru_cache(maxsize=None)
def _library():
    lib = _base.load_library()
    i64, p, c_int, size, f64 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_double
    psize = ctypes.POINTER(size)
    args = {
        "rms_norm": [i64, i64, p, c_int, p, p, c_int, f64, p, p, p],
        "rms_norm_quantize": [i64, i64, p, c_int, p, p, c_int, f64, p, p, p, c_int, p, p],
        "rms_norm_backward_workspace_size": [i64, i64, c_int, psize],
        "rms_norm_backward": [i64, i64, p, p, c_int, p, c_int, f64, p, p, p, p, size, p],
        "cross_entropy_gemm_workspace_size": [i64, i64, i64, psize],
        "cross_entropy_gemm": [i64, i64, i64, p, p, p, i64, p, p, p, size, p],
        "cross_entropy_gemm_backward_workspace_size": [i64, i64, i64, psize, psize],
        "cross_entropy_gemm_backward": [i64, i64, i64, p, p, p, p, i64, p, p, p, p, size, p],
        "adapter_gemm_workspace_size": [i64, i64, i64, i64, i64, psize],
        "adapter_gemm": [i64, i64, i64, i64, i64, p, p, p, p, p, p, p, c_int, p, size, p],
    }
    for name, a in args.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = a, c_int
    return lib


_native = None


def _binding():
    """The compiled binding (binding/lm_binding.cpp); raises if the package is not built."""
    global _native
    if _native is None:
        _library()
        try:
            _native = importlib.import_module("block_scaled_precision_e2m1_amd._lm_binding")
        except ImportError as e:
            raise ImportError("_lm_binding.so is not built or does not fit this torch; run "
                              "`python -c 'import __graft_entry__ as g; g.build()'`") from e
    return _native


def _query(name, *sizes, results=1):
    n = [ctypes.c_size_t(0) for _ in range(results)]
    _base._raise_on(name, getattr(_library(), name)(*sizes, *map(ctypes.byref, n)))
    return tuple(int(v.value) for v in n) if results > 1 else int(n[0].value)


def _no_second(what):
    raise RuntimeError(f"{what} has no second derivatives")


class _NormGradients(torch.autograd.Function):
    """rms_norm_backward within a backward pass.  Where that is recorded itself (create_graph), a second derivative
    raises: without this it would vanish."""

    @staticmethod
    def forward(ctx, dY, X, weight, eps, dH, want_dw):
        return _binding().rms_norm_backward(dY, X, weight, eps, dH, want_dw, None)

    @staticmethod
    def backward(ctx, *_):
        _no_second("rms_norm")


class _RmsNorm(torch.autograd.Function):
    """rms_norm with its gradient, from the rows that were normed."""

    @staticmethod
    def forward(ctx, X, weight, eps, residual):
        r = _binding().rms_norm(X, weight, eps, residual, None, None)
        ctx.save_for_backward(X if residual is None else r[1], weight)
        ctx.eps = eps
        ctx.set_materialize_grads(False)
        return r

    @staticmethod
    def backward(ctx, dY, dH=None):
        if dY is None:                       # the sum alone was used
            return dH, None, None, dH if ctx.needs_input_grad[3] else None
        rows, weight = ctx.saved_tensors
        dX, dW = _NormGradients.apply(dY.contiguous(), rows, weight, ctx.eps,
                                      None if dH is None else dH.contiguous(), ctx.needs_input_grad[1])
        return (dX if ctx.needs_input_grad[0] else None, dW, None, dX if ctx.needs_input_grad[3] else None)


def rms_norm(X, weight=None, eps=1e-6, residual=None, out=None, sum_out=None):
    """The root-mean-square norm of each row: Y = X / sqrt(mean(X^2) + eps) * weight.  With a residual (like X), of
    H = X + residual, rounded to its type, and (Y, H) is returned.  `out` may be X or the residual, `sum_out` (for H)
    too.

    Differentiable in X, weight and residual (then without `out` and `sum_out`)."""
    r = (_native or _binding()).rms_norm(X, weight, eps, residual, out, sum_out)
    return _RmsNorm.apply(X, weight, eps, residual) if r is None else r


def rms_norm_quantize(X, weight=None, eps=1e-6, residual=None, codes="int8", keep=False, sum_out=None):
    """The same norm as codes with one scale for each row, as w8a8_gemm (codes="int8", int8) and w4a8_gemm
    (codes="e4m3", uint8) take them: (codes [rows, K], scales [rows] float32), then H where there is a residual, then
    with keep=True the rows themselves, Y.  Not differentiable."""
    return (_native or _binding()).rms_norm_quantize(X, weight, eps, residual, codes, keep, sum_out)


def rms_norm_backward_workspace_size(rows, K, dtype=torch.bfloat16) -> int:
    """Bytes of workspace rms_norm_backward takes for rows of this type on the current device."""
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"dtype must be torch.float32 or torch.bfloat16, got {dtype}")
    return _query("rms_norm_backward_workspace_size", rows, K,
                  _base.IN_BF16 if dtype == torch.bfloat16 else _base.IN_F32)


def rms_norm_backward(dY, X, weight=None, eps=1e-6, dH=None, workspace=None):
    """The gradients (dX like X, dW like weight or None) of rms_norm for the incoming dY and, where H was used further
    on, dH, both like X.  X: the rows that were normed (H where there was a residual, whose gradient is dX too).
    `workspace` (uint8) needs rms_norm_backward_workspace_size bytes; None allocates them.  Nothing is recorded: the
    results carry no graph."""
    return (_native or _binding()).rms_norm_backward(dY, X, weight, eps, dH, True, workspace)


class _LossGradients(torch.autograd.Function):
    """cross_entropy_gemm_backward within a backward pass; as _NormGradients."""

    @staticmethod
    def forward(ctx, dL, X, W, target, lse, ignore_index, want_dx, want_dw):
        return _binding().cross_entropy_gemm_backward(dL, X, W, target, lse, ignore_index, want_dx, want_dw, None)

    @staticmethod
    def backward(ctx, *_):
        _no_second("cross_entropy_gemm")


class _CrossEntropyGemm(torch.autograd.Function):
    """cross_entropy_gemm with its gradient, from the lse that it keeps."""

    @staticmethod
    def forward(ctx, X, W, target, ignore_index, workspace):
        loss, lse = _binding().cross_entropy_gemm(X, W, target, ignore_index, True, workspace)
        ctx.save_for_backward(X, W, target, lse)
        ctx.ignore_index = ignore_index
        ctx.mark_non_differentiable(lse)
        ctx.set_materialize_grads(False)
        return loss, lse

    @staticmethod
    def backward(ctx, dL, _):
        if dL is None:
            return (None,) * 5
        dX, dW = _LossGradients.apply(dL.contiguous(), *ctx.saved_tensors, ctx.ignore_index, *ctx.needs_input_grad[:2])
        return dX, dW, None, None, None


def cross_entropy_gemm_workspace_size(M, V, K) -> int:
    """Bytes of workspace cross_entropy_gemm takes for these sizes on the current device."""
    return _query("cross_entropy_gemm_workspace_size", M, V, K)


def cross_entropy_gemm_backward_workspace_size(M, V, K):
    """(bytes cross_entropy_gemm_backward can use, bytes it needs at least) on the current device."""
    return _query("cross_entropy_gemm_backward_workspace_size", M, V, K, results=2)


def cross_entropy_gemm(X, W, target, ignore_index=-100, save=False, workspace=None):
    """The softmax cross entropy of each row of X [M, K] against its target token, over the vocabulary's W [V, K] and
    without the logits X W^T in memory: loss [M] float32 = log sum exp(X W^T) - (X W^T)[target].  Rows whose target is
    ignore_index have loss 0 and take no part.  With save=True returns (loss, lse): lse [M] float32, which
    cross_entropy_gemm_backward takes.  `workspace` (uint8) needs cross_entropy_gemm_workspace_size bytes; None
    allocates them.

    Differentiable in X and W; lse carries no graph."""
    r = (_native or _binding()).cross_entropy_gemm(X, W, target, ignore_index, save, workspace)
    if r is None:
        r = _CrossEntropyGemm.apply(X, W, target, ignore_index, workspace)
        return r if save else r[0]
    return r


def cross_entropy_gemm_backward(dL, X, W, target, lse, ignore_index=-100, workspace=None):
    """The gradients (dX [M, K], dW [V, K], bfloat16) of cross_entropy_gemm for the incoming dL [M] float32, with lse as
    cross_entropy_gemm(..., save=True) returned it.  `workspace` (uint8) needs the second of
    cross_entropy_gemm_backward_workspace_size's values; None allocates the first.  Nothing is recorded: the results
    carry no graph."""
    return (_native or _binding()).cross_entropy_gemm_backward(dL, X, W, target, lse, ignore_index, True, True, workspace)


def adapter_gemm_workspace_size(M, N, K, R, L) -> int:
    """Bytes of workspace adapter_gemm takes for these sizes on the current device."""
    return _query("adapter_gemm_workspace_size", M, N, K, R, L)


def adapter_gemm(base, X, A, B, index, scales=None, out=None, workspace=None):
    """Low-rank adapters of many requests beside a projection that they share and that has given `base` [M, N] (of any of
    the package's products): D[m] = base[m] + scales[i] * B[i] (A[i] X[m]) with i = index[m], for A [L, R, K], B [L, N, R]
    and scales [L] float32 (None: 1).  A row whose index is outside 0 .. L-1 (-1, say) keeps its base.  Adapters of
    a lower rank than R are filled up with zeros.  `out` may be base itself.  `workspace` (uint8) needs
    adapter_gemm_workspace_size bytes; None allocates them.  Not differentiable."""
    return (_native or _binding()).adapter_gemm(base, X, A, B, index, scales, out, workspace)
