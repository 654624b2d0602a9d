"""Gradients of a mean: one dL for all rows, of which each row's P is mostly made."""
import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4
from tests.test_gpu_loss import B, DEV, check, formula, inputs

pytestmark = pytest.mark.gpu


def errors(x, w, t, dl):
    _, _, dx, dw = check(x, w, t, dl)
    _, _, _, rx, _, rw, _ = formula(x, w, t, dl)
    return [((g.double() - r).norm() / r.norm()).item() for g, r in zip((dx, dw), (rx, rw))]


def unsure(m, v, k, seed):
    """Rows that know little of their tokens: p is about 1 / V, and P at the wanted token -dL."""
    x, w, t, dl = inputs(m, v, k, seed, 0.0, 0.1)
    return (0.1 * x.float()).bfloat16(), w, t, dl


@pytest.mark.parametrize("m,v,k", [(230, 3000, 264), (1020, 2000, 264), (4080, 2000, 520), (4095, 20000, 264), (9000, 3000, 264)])
@pytest.mark.parametrize("dl", [1.0, 1.00390625, 1.33, 1.9, -1.0039])
def test_a_mean_has_the_precision_of_its_results(m, v, k, dl):
    """P's wanted entries are dL but for p, below 2^-9, and dL is rounded to nothing: what is left of P's roundings is that
    of the other entries, each 2^-9 of 1 / V or so.  The gradients are off by their own rounding: at most 2^-8 of each value, and
    of values spread over a binade less than 0.6 of that in the norm."""
    print(f"case cross_entropy_gemm_backward {m}x{v}x{k} dL {dl} / {m}", flush=True)
    x, w, t, _ = unsure(m, v, k, 80)
    for e in errors(x, w, t, torch.full((m,), dl / m, device=DEV)):
        assert e < 0.6 * B, e


@pytest.mark.parametrize("top", [2.0 ** -149, 2.0 ** -127, 2.0 ** -126, 1.5 * 2.0 ** -126, 1.5 * 2.0 ** 125, 2.0 ** 126, 1.5 * 2.0 ** 126])
@pytest.mark.parametrize("m", [100, 300, 5000])
def test_the_ends_of_the_range(m, top):
    """The largest |dL| at and past the ends of what is scaled: results are those of the formula, where bf16's normal numbers hold them."""
    print(f"case cross_entropy_gemm_backward {m}x600x72 largest dL {top}", flush=True)
    x, w, t, dl = inputs(m, 600, 72, 81)
    dl = dl * 0
    dl[::2] = 2.0 ** -100 if top > 1 else top / 8
    dl[5] = -top
    t[5] = 3
    x[5], w = x[5] * 2.0 ** -8, (w.float() * 2.0 ** -2).bfloat16()
    _, lse = fp4.cross_entropy_gemm(x, w, t, save=True)
    dx, dw = fp4.cross_entropy_gemm_backward(dl, x, w, t, lse)
    torch.cuda.synchronize(DEV)
    _, _, _, rx, tx, rw, tw = formula(x, w, t, dl)
    # below the smallest normal number, 2^-126, an entry of P or a result may be lost whole
    assert ((dx.double() - rx).abs() <= tx + 2.0 ** -125 * (1 + w.double().abs().sum(0))).all()
    assert ((dw.double() - rw).abs() <= tw + 2.0 ** -125 * (1 + x.double().abs().sum(0))).all()


def test_rows_that_take_no_part_do_not_scale():
    """What dL holds there, infinities and NaN and the largest numbers among it, changes no bit."""
    for m in (300, 5000):
        x, w, t, dl = inputs(m, 700, 72, 82, 0.5)
        loss, lse = fp4.cross_entropy_gemm(x, w, t, save=True)
        want = fp4.cross_entropy_gemm_backward(dl, x, w, t, lse)
        none = torch.nonzero(t == -100)[:, 0]
        other = dl.clone()
        other[none] = torch.tensor([float("nan"), float("inf"), -3e38, 1.1, 0.0], device=DEV).repeat(none.numel() // 5 + 1)[:none.numel()]
        got = fp4.cross_entropy_gemm_backward(other, x, w, t, lse)
        torch.cuda.synchronize(DEV)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("m", [3, 300])
def test_results_next_to_the_largest_number(m):
    """A gradient that fp32 and bf16 hold, made of sums that no scaling may take past it: dX = -+1.8 * 2^126."""
    v, k = 2, 24
    x, w = torch.full((m, k), 0.5, device=DEV), torch.zeros(v, k, device=DEV)
    w[0, 0], w[1, 0] = 1.0, -1.125
    x[:, 1], w[0, 1], w[1, 1] = 0.5, -1.0, 1.125                 # the logits are 0
    t = torch.zeros(m, dtype=torch.int64, device=DEV)
    dl = torch.zeros(m, device=DEV)
    dl[1] = 1.7 * 2.0 ** 126
    x, w = x.bfloat16(), w.bfloat16()
    _, lse = fp4.cross_entropy_gemm(x, w, t, save=True)
    dx, dw = fp4.cross_entropy_gemm_backward(dl, x, w, t, lse)
    torch.cuda.synchronize(DEV)
    want = -0.5 * 1.7 * 2.0 ** 126 * 2.125
    assert abs(dx[1, 0].double().item() / want - 1) <= 3 * B and abs(dx[1, 1].double().item() / want + 1) <= 3 * B
    assert torch.isfinite(dx.float()).all() and torch.isfinite(dw.float()).all()
