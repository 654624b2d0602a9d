"""Every tile of the loss's products, without and with a K split, on whole vocabularies and on pieces."""
import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4
from tests import loss_plans as plans
from tests.test_gpu_loss import DEV, check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ignored", [0.0, 0.6])
@pytest.mark.parametrize("size", [p[0] for p in plans.SIZES])
def test_tiles(size, ignored):
    print(f"case cross_entropy_gemm {size} {plans.products(*size)} ignored {ignored}", flush=True)
    check(*inputs(*size, 31, ignored))


@pytest.mark.parametrize("size", [p[0] for p in plans.SIZES if p[0][1] <= 5200])
def test_pieces(size):
    """dX's sums kept over pieces of 64 columns, and over a few of them."""
    m, v, k = size
    most, least = fp4.cross_entropy_gemm_backward_workspace_size(m, v, k)
    x, w, t, dl = inputs(m, v, k, 32, 0.3)
    for room in sorted({least, least + (most - least) // 3}):
        print(f"case cross_entropy_gemm_backward {size} workspace {room}", flush=True)
        check(x, w, t, dl, torch.full((room,), 255, dtype=torch.uint8, device=DEV))
