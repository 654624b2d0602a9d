"""Feed-forward operators: int8 activations and products, and the gated block in int8 and bf16.

A binding over the C ABI of ``include/fp4g_ffn.h`` in the manner of the package's other
functions: each has the name of its C entry point, checks its torch arguments, runs on the
current stream of their GPU and raises ``Fp4GemmError`` on a non-zero status.  The checks and
the calls are compiled (``binding/ffn_binding.cpp``): a decode step's kernels take a few
microseconds, less than the same checks take in Python.

Layouts (contiguous, all on one GPU):
  int8_quantize        : X [rows, K] float32 or bfloat16 -> codes [rows, K] int8, scales [rows] float32
  w8a8_gemm            : A [M, K] int8, sa [M] float32, B [N, K] int8, sb [N] float32 -> D [M, N]
  w8a8_gated_gemm      : A, sa as above; Bg, Bu [N, K] int8, sg, su [N] float32 -> D [M, N]
  gated_gemm           : X [M, K], Wg, Wu [N, K] bfloat16 -> H [M, N] bfloat16
  gated_gemm_backward  : the gradients of gated_gemm, bfloat16
K is a multiple of 16 for int8 operands and of 8 for bf16; M and N are free, but for
gated_gemm_backward's N of at most 2^21.  gated_gemm takes part in autograd; the results of the
other functions carry no graph.
"""
from __future__ import annotations

import ctypes
import functools
import importlib

import torch

import block_scaled_precision_e2m1_amd as _base

__all__ = ["int8_quantize", "w8a8_gemm_workspace_size", "w8a8_gemm", "w8a8_gated_gemm_workspace_size",
           "w8a8_gated_gemm", "gated_gemm_workspace_size", "gated_gemm", "gated_gemm_backward_workspace_size",
           "gated_gemm_backward", "FFN_SYMBOLS"]

FFN_SYMBOLS = ("int8_quantize", "w8a8_gemm_workspace_size", "w8a8_gemm", "w8a8_gated_gemm_workspace_size",
               "w8a8_gated_gemm", "gated_gemm_workspace_size", "gated_gemm", "gated_gemm_backward_workspace_size",
               "gated_gemm_backward")


@functools.lru_cache(maxsize=None)
def _library():
    lib = _base.load_library()
    i64, p, c_int, size = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    psize = ctypes.POINTER(size)
    args = {
        "int8_quantize": [i64, i64, p, c_int, p, p, p],
        "w8a8_gemm": [i64, i64, i64, p, p, p, p, p, c_int, p, size, p],
        "w8a8_gated_gemm": [i64, i64, i64, p, p, p, p, p, p, c_int, p, c_int, p, size, p],
        "gated_gemm": [i64, i64, i64, p, p, p, c_int, p, p, p, p, size, p],
        "gated_gemm_backward": [i64, i64, i64, p, p, p, p, p, p, c_int, p, p, p, p, size, p],
        "w8a8_gemm_workspace_size": [i64, i64, i64, psize],
        "w8a8_gated_gemm_workspace_size": [i64, i64, i64, psize],
        "gated_gemm_workspace_size": [i64, i64, i64, psize],
        "gated_gemm_backward_workspace_size": [i64, i64, i64, psize, psize],
    }
    for name, a in args.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = a, c_int
    return lib


_native = None


def _binding():
    """The compiled binding (binding/ffn_binding.cpp); raises if the package is not built."""
    global _native
    if _native is None:
        _library()
        try:
            _native = importlib.import_module("block_scaled_precision_e2m1_amd._ffn_binding")
        except ImportError as e:
            raise ImportError("_ffn_binding.so is not built or does not fit this torch; run "
                              "`python -c 'import __graft_entry__ as g; g.build()'`") from e
    return _native


def _query(name, *mnk):
    n = [ctypes.c_size_t(0) for _ in range(2 if "backward" in name else 1)]
    st = getattr(_library(), name)(*mnk, *map(ctypes.byref, n))
    _base._raise_on(name, st)
    return tuple(int(v.value) for v in n) if len(n) > 1 else int(n[0].value)


def w8a8_gemm_workspace_size(M, N, K) -> int:
    """Bytes of workspace w8a8_gemm can use for these sizes on the current device."""
    return _query("w8a8_gemm_workspace_size", M, N, K)


def w8a8_gated_gemm_workspace_size(M, N, K) -> int:
    """Bytes of workspace w8a8_gated_gemm can use for these sizes on the current device."""
    return _query("w8a8_gated_gemm_workspace_size", M, N, K)


def gated_gemm_workspace_size(M, N, K) -> int:
    """Bytes of workspace gated_gemm can use for these sizes on the current device."""
    return _query("gated_gemm_workspace_size", M, N, K)


def gated_gemm_backward_workspace_size(M, N, K):
    """(bytes gated_gemm_backward can use, bytes it needs at least) on the current device."""
    return _query("gated_gemm_backward_workspace_size", M, N, K)


def int8_quantize(X, codes=None, scales=None):
    """Row quantizer: X [rows, K] float32 or bfloat16 (K % 16 == 0) -> (codes [rows, K] int8,
    scales [rows] float32), scale = max|x| / 127, codes rounded to nearest, ties to even."""
    return (_native or _binding()).int8_quantize(X, codes, scales)


def w8a8_gemm(A, sa, B, sb, out=None, out_dtype=torch.bfloat16, workspace=None):
    """int8 GEMM with a scale for each token and each channel: D = (A B^T) * sa[:, None] *
    sb[None, :], exact sums.  `workspace` (uint8) may hold the partial sums of a K split;
    None allocates what the library can use."""
    return (_native or _binding()).w8a8_gemm(A, sa, B, sb, out, out_dtype, workspace)


def w8a8_gated_gemm(A, sa, Bg, sg, Bu, su, act="silu", out=None, out_dtype=torch.bfloat16, workspace=None):
    """The gated half of a feed-forward block in int8: D = act(g) * u with g and u the
    w8a8_gemm of A with Bg, sg and with Bu, su.  act: "silu", "gelu" or "gelu_tanh"."""
    return (_native or _binding()).w8a8_gated_gemm(A, sa, Bg, sg, Bu, su, act, out, out_dtype, workspace)


class _Gradients(torch.autograd.Function):
    """gated_gemm_backward within a backward pass.  Where that is recorded itself (create_graph), a second
    derivative raises: without this it would vanish."""

    @staticmethod
    def forward(ctx, dH, X, Wg, Wu, G, U, act):
        return _binding().gated_gemm_backward(dH, X, Wg, Wu, G, U, act, None)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("gated_gemm has no second derivatives")


class _GatedGemm(torch.autograd.Function):
    """gated_gemm with its gradient, from the G and U that it keeps."""

    @staticmethod
    def forward(ctx, X, Wg, Wu, act, out, workspace):
        H, G, U = _binding().gated_gemm(X, Wg, Wu, act, True, out, workspace)
        ctx.save_for_backward(X, Wg, Wu, G, U)
        ctx.act = act
        ctx.mark_non_differentiable(G, U)
        ctx.set_materialize_grads(False)
        if out is not None:
            ctx.mark_dirty(out)
        return H, G, U

    @staticmethod
    def backward(ctx, dH, dG, dU):
        if dH is None:
            return (None,) * 6
        grads = _Gradients.apply(dH.contiguous(), *ctx.saved_tensors, ctx.act)
        return *(d if wanted else None for d, wanted in zip(grads, ctx.needs_input_grad)), None, None, None


def gated_gemm(X, Wg, Wu, act="silu", save=False, out=None, workspace=None):
    """The gated half of a feed-forward block in bf16: H = act(X Wg^T) * (X Wu^T), fp32 sums,
    one rounding.  With save=True returns (H, G, U): G and U [M, N] float32 are the two
    products, which gated_gemm_backward takes.

    Differentiable in X, Wg and Wu: where one of them requires a gradient, G and U are kept for
    the backward pass, and H carries the graph (G and U do not)."""
    r = (_native or _binding()).gated_gemm(X, Wg, Wu, act, save, out, workspace)
    if r is None:
        r = _GatedGemm.apply(X, Wg, Wu, act, out, workspace)
        return r if save else r[0]
    return r


def gated_gemm_backward(dH, X, Wg, Wu, G, U, act="silu", workspace=None):
    """The gradients (dX [M, K], dWg [N, K], dWu [N, K], bfloat16) of gated_gemm for the
    incoming dH [M, N] bfloat16, with G and U as gated_gemm(..., save=True) returned them.
    `workspace` (uint8) needs the second of gated_gemm_backward_workspace_size's values; None
    allocates the first.  Nothing is recorded: the results carry no graph."""
    return (_native or _binding()).gated_gemm_backward(dH, X, Wg, Wu, G, U, act, workspace)
