"""Few rows that take part among many: P is kept in two terms by the rows that there are, not by all rows of the call."""
import pytest
import torch

import block_scaled_precision_e2m1_amd as fp4
from tests.test_gpu_loss import B, DEV, check, formula, gen, inputs

pytestmark = pytest.mark.gpu


def few(m, v, k, keep, seed):
    x, w, t, dl = inputs(m, v, k, seed, 0.0)
    t[torch.randperm(m, generator=gen(seed + 1), device=DEV)[keep:]] = -100
    return x, w, t, dl


@pytest.mark.parametrize("m,v,k,keep", [(4096, 2000, 256, 1), (4096, 2000, 256, 3), (600, 3000, 136, 20), (200, 900, 264, 100),
                                        (129, 900, 264, 128), (5000, 2000, 1024, 65), (9000, 40000, 264, 40),
                                        (2100, 300, 72, 128)])
def test_gradients_are_off_by_their_own_rounding_alone(m, v, k, keep):
    """As where these rows are all of the call: at most 2^-8 of each value where P's two terms keep 2^-16, and of values
    spread over a binade less than 0.6 of that in the norm."""
    print(f"case cross_entropy_gemm_backward {m}x{v}x{k}, {keep} rows", flush=True)
    for seed in (60, 62, 64):
        x, w, t, dl = few(m, v, k, keep, seed)
        _, _, dx, dw = check(x, w, t, dl)
        _, _, _, rx, _, rw, _ = formula(x, w, t, dl)
        for got, want in ((dx, rx), (dw, rw)):
            e = ((got.double() - want).norm() / want.norm()).item()
            assert e < 0.6 * B, (seed, e)


@pytest.mark.parametrize("keep", [0, 1, 127, 128, 129, 200])
@pytest.mark.parametrize("m,v,k", [(300, 2000, 136), (1500, 5200, 72)])
def test_pieces_and_workspaces_at_the_border(m, v, k, keep):
    """On each side of 128 rows, for the whole vocabulary and for pieces of it, in a workspace of just the size that is asked
    for and full of NaN."""
    x, w, t, dl = few(m, v, k, keep, 70)
    most, least = fp4.cross_entropy_gemm_backward_workspace_size(m, v, k)
    for room in sorted({least, least + (most - least) // 3, most}):
        print(f"case cross_entropy_gemm_backward {m}x{v}x{k}, {keep} rows, workspace {room}", flush=True)
        space = torch.full((room + 64,), 255, dtype=torch.uint8, device=DEV)
        check(x, w, t, dl, space[:room])
        assert (space[room:] == 255).all()


def test_a_replay_crosses_the_border():
    """One captured call, replayed with more rows and with fewer."""
    m, v, k = 300, 2000, 136
    x, w, t, dl = inputs(m, v, k, 71, 0.0)
    others = [few(m, v, k, n, 71)[2] for n in (128, 300, 5, 129)]
    live = t.clone()

    def calls():
        loss, lse = fp4.cross_entropy_gemm(x, w, live, save=True)
        return fp4.cross_entropy_gemm_backward(dl, x, w, live, lse)

    want = []
    for o in others:
        live.copy_(o)
        want.append([r.clone() for r in calls()])
    torch.cuda.synchronize(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for rep in range(8):
        live.copy_(others[rep % 4])
        for r in held:
            r.fill_(1)
        graph.replay()
        torch.cuda.synchronize(DEV)
        assert all(torch.equal(a, b) for a, b in zip(held, want[rep % 4])), rep
        fp4.cross_entropy_gemm(x, w, t)
        torch.cuda.synchronize(DEV)
