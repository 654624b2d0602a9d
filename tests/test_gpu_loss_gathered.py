"""The loss's edge cases where its forward pass gathers the rows that take part, as it does for large products."""
import ctypes

import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4
from tests.ffn_plans import internal
from tests.test_gpu_loss import DEV, U, check, close, formula, inputs

pytestmark = pytest.mark.gpu

# Rows counted by every workgroup, and in chunks of 1024 (more than 4096).
SIZES = [(300, 30000, 1024), (5000, 2000, 1024)]


def gathers(m, v, k):
    return internal("_ZN4fp4g12loss_gathersElll", ctypes.c_bool, 3)(m, v, k)


@pytest.fixture(params=SIZES, ids=str)
def size(request):
    assert gathers(*request.param)
    print(f"case cross_entropy_gemm {request.param}", flush=True)
    return request.param


def test_the_border():
    assert not gathers(64, 1 << 20, 4096) and gathers(65, 1 << 20, 4096) and not gathers(8192, 1024, 1024)


def test_no_row_takes_part(size):
    """With a token of the vocabulary as the one that is ignored."""
    x, w, t, dl = inputs(*size, 50)
    t[:] = 7
    loss, lse = fp4.cross_entropy_gemm(x, w, t, ignore_index=7, save=True)
    dx, dw = fp4.cross_entropy_gemm_backward(dl, x, w, t, lse, ignore_index=7)
    torch.cuda.synchronize(DEV)
    assert not loss.any() and not lse.any() and not dx.any() and not dw.any()


def test_an_ignored_token_of_the_vocabulary(size):
    x, w, t, dl = inputs(*size, 51, 0.0)
    t[::3] = 7
    loss, lse = fp4.cross_entropy_gemm(x, w, t, ignore_index=7, save=True)
    got = fp4.cross_entropy_gemm_backward(dl, x, w, t, lse, ignore_index=7)
    torch.cuda.synchronize(DEV)
    t[t == 7] = -100
    rl, rs, tol, rx, tx, rw, tw = formula(x, w, t, dl)
    for a, b, c, name in ((loss, rl, tol, "loss"), (lse, rs, tol, "lse"), (got[0], rx, tx, "dX"), (got[1], rw, tw, "dW")):
        close(a, b, c, name)


@pytest.mark.parametrize("keep", [1, 2, 70, 129])
def test_few_rows_take_part(size, keep):
    """The last row among them: the others are far apart."""
    m = size[0]
    x, w, t, dl = inputs(*size, 52, 0.0)
    out = torch.ones(m, dtype=torch.bool, device=DEV)
    out[torch.linspace(m - 1, m // 7, keep, device=DEV).long()] = False
    t[out] = -100
    check(x, w, t, dl)


def test_targets_outside_the_vocabulary(size):
    m, v, k = size
    x, w, t, dl = inputs(*size, 53, 0.2)
    for at, bad in ((3, v), (4, -1), (5, 1 << 40), (m - 1, -(1 << 33))):
        t[at] = bad
    loss, lse = fp4.cross_entropy_gemm(x, w, t, save=True)
    dx, dw = fp4.cross_entropy_gemm_backward(dl, x, w, t, lse)
    torch.cuda.synchronize(DEV)
    bad = torch.zeros(m, dtype=torch.bool, device=DEV)
    bad[[3, 4, 5, m - 1]] = True
    assert torch.isnan(loss[bad]).all() and torch.isfinite(lse).all()
    assert torch.isnan(dx[bad]).all() and torch.isnan(dw).all()
    assert torch.isfinite(dx[~bad].float()).all()
    t[bad] = -100                      # what the others give is theirs alone
    rl, _, tol, *_ = formula(x, w, t, dl)
    close(loss[~bad], rl[~bad], tol[~bad], "loss")


def test_infinities_stay_in_their_rows(size):
    m = size[0]
    x, w, t, dl = inputs(*size, 54, 0.3)
    t[5], t[m - 2] = 1, 2
    x[5, 3], x[m - 2, 1] = float("inf"), float("nan")
    loss = fp4.cross_entropy_gemm(x, w, t)
    torch.cuda.synchronize(DEV)
    bad = torch.zeros(m, dtype=torch.bool, device=DEV)
    bad[[5, m - 2]] = True
    assert torch.isnan(loss[bad]).all() and torch.isfinite(loss[~bad]).all()


def test_logits_of_minus_infinity(size):
    """A token that is ruled out has probability 0; where it is the wanted one the loss is infinite."""
    m, v, k = size
    x, w, t, dl = inputs(*size, 55, 0.1)
    x[:, 0] = 1
    w[:, 0] = 0
    w[256:512, 0] = float("-inf")      # whole tiles of them
    t[(t >= 256) & (t < 512)] = 3
    t[9] = 300
    loss, lse = fp4.cross_entropy_gemm(x, w, t, save=True)
    torch.cuda.synchronize(DEV)
    there = torch.ones(v, dtype=torch.bool, device=DEV)
    there[256:512] = False
    some = t != -100
    some[9] = False
    z = x.double() @ w[there].double().t()
    tol = 2 * (k + 8) * U * (x.double().abs() @ w[there].double().abs().t()).amax(1) + (v / 1024 + 200) * U * (1 + z.abs().amax(1))
    assert loss[9] == float("inf") and torch.isfinite(loss[some]).all()
    close(lse[some], torch.logsumexp(z, 1)[some], tol[some], "lse")


def test_replayed_with_other_rows(size):
    """A captured call in whose replays other rows take part, none among them."""
    x, w, t, dl = inputs(*size, 56, 0.5)
    others = [t, torch.full_like(t, -100), inputs(*size, 57, 0.9)[2]]
    live = t.clone()

    def calls():
        loss, lse = fp4.cross_entropy_gemm(x, w, live, save=True)
        return loss, lse, *fp4.cross_entropy_gemm_backward(dl, x, w, live, lse)

    want = []
    for o in others:
        live.copy_(o)
        want.append([r.clone() for r in calls()])
    torch.cuda.synchronize(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for rep in range(6):
        live.copy_(others[rep % 3])
        for r in held:
            r.fill_(1)
        graph.replay()
        torch.cuda.synchronize(DEV)
        for a, b in zip(held, want[rep % 3]):
            assert torch.equal(a, b), rep
        fp4.cross_entropy_gemm(x, w, t)
        torch.cuda.synchronize(DEV)
