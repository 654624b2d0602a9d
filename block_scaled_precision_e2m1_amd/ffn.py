"""Feed-forward operators: int8 activations and products, and the gated block in int8 and bf16.

A binding over the C ABI of ``include/fp4g_ffn.h`` in the manner of the package's other
functions: each has the name of its C entry point, checks its torch arguments, runs on the
current stream of their GPU and raises ``Fp4GemmError`` on a non-zero status.

Layouts (contiguous, all on one GPU):
  int8_quantize        : X [rows, K] float32 or bfloat16 -> codes [rows, K] int8, scales [rows] float32
  w8a8_gemm            : A [M, K] int8, sa [M] float32, B [N, K] int8, sb [N] float32 -> D [M, N]
  w8a8_gated_gemm      : A, sa as above; Bg, Bu [N, K] int8, sg, su [N] float32 -> D [M, N]
  gated_gemm           : X [M, K], Wg, Wu [N, K] bfloat16 -> H [M, N] bfloat16
  gated_gemm_backward  : the gradients of gated_gemm, bfloat16
K is a multiple of 16 for int8 operands and of 8 for bf16; M and N are free.
"""
from __future__ import annotations

import ctypes
import functools

import torch

import block_scaled_precision_e2m1_amd as _base

__all__ = ["int8_quantize", "w8a8_gemm_workspace_size", "w8a8_gemm", "w8a8_gated_gemm_workspace_size",
           "w8a8_gated_gemm", "gated_gemm_workspace_size", "gated_gemm", "gated_gemm_backward_workspace_size",
           "gated_gemm_backward", "FFN_SYMBOLS"]

FFN_SYMBOLS = ("int8_quantize", "w8a8_gemm_workspace_size", "w8a8_gemm", "w8a8_gated_gemm_workspace_size",
               "w8a8_gated_gemm", "gated_gemm_workspace_size", "gated_gemm", "gated_gemm_backward_workspace_size",
               "gated_gemm_backward")

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
_F32, _BF16, _I8 = torch.float32, torch.bfloat16, torch.int8


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


def _need(t, name, dtype, shape, device):
    """t is a contiguous tensor of this type and shape on this device; the package's errors if not."""
    if (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        return
    _base._check(t, name, dtype, shape, device)


def _matrix(t, name, dtypes):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.device


def _result(out, name, dtype, shape, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(out, name, dtype, shape, device)
    return out


def _out(out, M, N, out_dtype, device):
    if out is not None:
        out_dtype = out.dtype if isinstance(out, torch.Tensor) else out_dtype
    if out_dtype is not _BF16 and out_dtype is not _F32:
        raise TypeError("out must be float32 or bfloat16")
    return _result(out, "out", out_dtype, (M, N), device), int(out_dtype is _BF16)


def _act(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def _space(workspace, nbytes, device):
    """(pointer, bytes, tensor) of the caller's workspace or of a new one of `nbytes`."""
    if workspace is None:
        if not nbytes:
            return None, 0, None
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    else:
        _need(workspace, "workspace", torch.uint8, (workspace.numel(),), device)
    return workspace.data_ptr() or None, workspace.numel(), workspace


def _stream(device):
    return torch.cuda.current_stream(device).cuda_stream


# The sizes depend on the device only through its number of compute units.
@functools.lru_cache(maxsize=4096)
def _sizes(name, device, *mnk):
    with torch.cuda.device(device):
        return _query(name, *mnk)


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
    device = _matrix(X, "X", (_BF16, _F32))
    rows, K = X.shape
    if K % 16:
        raise ValueError(f"K={K} must be a multiple of 16")
    codes = _result(codes, "codes", _I8, (rows, K), device)
    scales = _result(scales, "scales", _F32, (rows,), device)
    st = _library().int8_quantize(rows, K, X.data_ptr(), int(X.dtype is _BF16), codes.data_ptr(), scales.data_ptr(),
                                  _stream(device))
    if st:
        _base._raise_on("int8_quantize", st)
    return codes, scales


def _int8_operands(A, sa, weights):
    device = _matrix(A, "A", (_I8,))
    M, K = A.shape
    if K % 16:
        raise ValueError(f"K={K} must be a multiple of 16")
    N = None
    for name, B, sname, sb in weights:
        if N is None:
            _matrix(B, name, (_I8,))
            N = B.shape[0]
        _need(B, name, _I8, (N, K), device)
        _need(sb, sname, _F32, (N,), device)
    _need(sa, "sa", _F32, (M,), device)
    return device, M, N, K


def w8a8_gemm(A, sa, B, sb, out=None, out_dtype=torch.bfloat16, workspace=None):
    """int8 GEMM with a scale for each token and each channel: D = (A B^T) * sa[:, None] *
    sb[None, :], exact sums.  `workspace` (uint8) may hold the partial sums of a K split;
    None allocates what the library can use."""
    device, M, N, K = _int8_operands(A, sa, (("B", B, "sb", sb),))
    D, dt = _out(out, M, N, out_dtype, device)
    nbytes = _sizes("w8a8_gemm_workspace_size", device, M, N, K) if workspace is None else 0
    ptr, size, _keep = _space(workspace, nbytes, device)
    st = _library().w8a8_gemm(M, N, K, A.data_ptr(), sa.data_ptr(), B.data_ptr(), sb.data_ptr(), D.data_ptr(), dt, ptr,
                              size, _stream(device))
    if st:
        _base._raise_on("w8a8_gemm", st)
    return D


def w8a8_gated_gemm(A, sa, Bg, sg, Bu, su, act="silu", out=None, out_dtype=torch.bfloat16, workspace=None):
    """The gated half of a feed-forward block in int8: D = act(g) * u with g and u the
    w8a8_gemm of A with Bg, sg and with Bu, su.  act: "silu", "gelu" or "gelu_tanh"."""
    device, M, N, K = _int8_operands(A, sa, (("Bg", Bg, "sg", sg), ("Bu", Bu, "su", su)))
    code = _act(act)
    D, dt = _out(out, M, N, out_dtype, device)
    nbytes = _sizes("w8a8_gated_gemm_workspace_size", device, M, N, K) if workspace is None else 0
    ptr, size, _keep = _space(workspace, nbytes, device)
    st = _library().w8a8_gated_gemm(M, N, K, A.data_ptr(), sa.data_ptr(), Bg.data_ptr(), sg.data_ptr(), Bu.data_ptr(),
                                    su.data_ptr(), code, D.data_ptr(), dt, ptr, size, _stream(device))
    if st:
        _base._raise_on("w8a8_gated_gemm", st)
    return D


def _bf16_operands(X, Wg, Wu):
    device = _matrix(X, "X", (_BF16,))
    _matrix(Wg, "Wg", (_BF16,))
    M, K = X.shape
    N = Wg.shape[0]
    if K % 8:
        raise ValueError(f"K={K} must be a multiple of 8")
    _need(Wg, "Wg", _BF16, (N, K), device)
    _need(Wu, "Wu", _BF16, (N, K), device)
    return device, M, N, K


def gated_gemm(X, Wg, Wu, act="silu", save=False, out=None, workspace=None):
    """The gated half of a feed-forward block in bf16: H = act(X Wg^T) * (X Wu^T), fp32 sums,
    one rounding.  With save=True returns (H, G, U): G and U [M, N] float32 are the two
    products, which gated_gemm_backward takes."""
    device, M, N, K = _bf16_operands(X, Wg, Wu)
    code = _act(act)
    H = _result(out, "out", _BF16, (M, N), device)
    G = U = None
    if save:
        G = torch.empty((M, N), dtype=_F32, device=device)
        U = torch.empty((M, N), dtype=_F32, device=device)
    nbytes = _sizes("gated_gemm_workspace_size", device, M, N, K) if workspace is None else 0
    ptr, size, _keep = _space(workspace, nbytes, device)
    st = _library().gated_gemm(M, N, K, X.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), code, H.data_ptr(),
                               G.data_ptr() if save else None, U.data_ptr() if save else None, ptr, size,
                               _stream(device))
    if st:
        _base._raise_on("gated_gemm", st)
    return (H, G, U) if save else H


def gated_gemm_backward(dH, X, Wg, Wu, G, U, act="silu", workspace=None):
    """The gradients (dX [M, K], dWg [N, K], dWu [N, K], bfloat16) of gated_gemm for the
    incoming dH [M, N] bfloat16, with G and U as gated_gemm(..., save=True) returned them.
    `workspace` (uint8) needs the second of gated_gemm_backward_workspace_size's values; None
    allocates the first."""
    device, M, N, K = _bf16_operands(X, Wg, Wu)
    code = _act(act)
    _need(dH, "dH", _BF16, (M, N), device)
    _need(G, "G", _F32, (M, N), device)
    _need(U, "U", _F32, (M, N), device)
    dX = torch.empty((M, K), dtype=_BF16, device=device)
    dWg = torch.empty((N, K), dtype=_BF16, device=device)
    dWu = torch.empty((N, K), dtype=_BF16, device=device)
    nbytes = _sizes("gated_gemm_backward_workspace_size", device, M, N, K)[0] if workspace is None else 0
    ptr, size, _keep = _space(workspace, nbytes, device)
    st = _library().gated_gemm_backward(M, N, K, dH.data_ptr(), X.data_ptr(), Wg.data_ptr(), Wu.data_ptr(),
                                        G.data_ptr(), U.data_ptr(), code, dX.data_ptr(), dWg.data_ptr(),
                                        dWu.data_ptr(), ptr, size, _stream(device))
    if st:
        _base._raise_on("gated_gemm_backward", st)
    return dX, dWg, dWu
