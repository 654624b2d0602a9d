"""Forward-mode tangents are refused, not dropped: by every operator that says whether it can be differentiated."""
import pytest
import torch
import torch.autograd.forward_ad as forward

import block_scaled_precision_e2m1_amd as fp4

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


def calls():
    """(function, its tensors by name, the other arguments) of every operator with every tensor that could carry a tangent."""
    rn = lambda t, *s: torch.randn(*s, device=DEV).to(t)  # noqa: E731
    rows, k, n, r = 6, 64, 40, 8
    norm = {"X": rn(F32, rows, k), "weight": rn(F32, k), "residual": rn(F32, rows, k)}
    target, index = torch.arange(rows, device=DEV), torch.zeros(rows, dtype=torch.int32, device=DEV)
    return [
        (fp4.rms_norm, dict(norm), {}),
        (fp4.rms_norm, {**norm, "out": rn(F32, rows, k), "sum_out": rn(F32, rows, k)}, {}),
        (fp4.rms_norm_quantize, {**norm, "sum_out": rn(F32, rows, k)}, {}),
        (fp4.cross_entropy_gemm, {"X": rn(BF, rows, k), "W": rn(BF, n, k)}, {"target": target}),
        (fp4.adapter_gemm, {"base": rn(F32, rows, n), "X": rn(BF, rows, k), "A": rn(BF, 1, r, k), "B": rn(BF, 1, n, r),
                            "scales": rn(F32, 1), "out": rn(F32, rows, n)}, {"index": index}),
        (fp4.gated_gemm, {"X": rn(BF, rows, k), "Wg": rn(BF, n, k), "Wu": rn(BF, n, k), "out": rn(BF, rows, n)}, {}),
    ]


@pytest.mark.parametrize("at", range(6))
def test_tangents_are_refused(at):
    f, tensors, rest = calls()[at]
    f(**tensors, **rest)
    with forward.dual_level():
        f(**tensors, **rest)                       # without tangents nothing is refused
        for name, t in tensors.items():
            dual = forward.make_dual(t, torch.ones_like(t))
            with pytest.raises(NotImplementedError, match="forward-mode"):
                f(**{**tensors, name: dual}, **rest)
            with torch.no_grad(), pytest.raises(NotImplementedError, match="forward-mode"):   # which turns off reverse mode alone
                f(**{**tensors, name: dual}, **rest)
            with forward._set_fwd_grad_enabled(False):
                f(**{**tensors, name: dual}, **rest)
    torch.cuda.synchronize(DEV)


def test_with_reverse_mode_at_once():
    f, tensors, rest = calls()[0]
    with forward.dual_level(), pytest.raises(NotImplementedError, match="forward-mode"):
        f(**{**tensors, "X": forward.make_dual(tensors["X"], tensors["X"]), "weight": tensors["weight"].clone().requires_grad_()})
