"""What an incoming gradient of infinity gives: the formula's infinities, whichever terms P is kept in."""
import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("m", [2, 100, 128, 129, 200])
@pytest.mark.parametrize("big", [float("inf"), 3.4e38])
def test_infinite_gradients(m, big):
    """Two tokens of equal logits, p = 1/2, and one row whose dL is infinite or nearly: its P is -dL / 2 at its token and dL / 2
    at the other.  With x > 0 dW is infinite with it, and so is dX where W has one sign for each sign of P; the other rows
    stay finite."""
    v, k = 2, 24
    x = torch.full((m, k), 0.5, device=DEV)
    w = torch.zeros(v, k, device=DEV)
    w[:, 0], w[:, 1] = torch.tensor([1.0, -1.0], device=DEV), torch.tensor([-1.0, 1.0], device=DEV)
    t = torch.zeros(m, dtype=torch.int64, device=DEV)
    dl = torch.ones(m, device=DEV)
    dl[m - 1] = big
    print(f"case cross_entropy_gemm_backward {m}x{v}x{k} dL {big}", flush=True)
    x, w = x.bfloat16(), w.bfloat16()
    _, lse = fp4.cross_entropy_gemm(x, w, t, save=True)
    dx, dw = fp4.cross_entropy_gemm_backward(dl, x, w, t, lse)
    torch.cuda.synchronize(DEV)
    assert torch.isfinite(dx[:-1].float()).all()
    if big == float("inf"):
        assert (dw[0] == -big).all() and (dw[1] == big).all()
        assert dx[-1, 0] == -big and dx[-1, 1] == big
    else:   # P = -+1.7e38, and dX = -+3.4e38, which rounds to bf16 within its range or to infinity
        assert torch.isfinite(dw.float()).all() and (dw[0].float() < -8e37).all() and (dw[1].float() > 8e37).all()
        assert dx[-1, 0] < -3e38 and dx[-1, 1] > 3e38
