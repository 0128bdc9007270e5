"""An infinity in an element that is not rotated changes no other element but through the
row's norm; one that is rotated changes its pair's."""
import math

import pytest
import torch

import __graft_entry__
import exact_attention_blackwell_tiled_gb300 as fa
from test_norm_rope import _rows, partner_sum, plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _case(D, rot, seed):
    gen = torch.Generator().manual_seed(seed)
    x, dy = _rows(D, 1, D, gen), _rows(D, 1, D, gen)  # row d: the infinity in element d
    w = 1 + torch.rand(D, generator=gen)
    pos = torch.randint(1, 50, (D,), generator=gen)
    cos, sin = fa.rope_table(50, rot)
    return x, dy, w, pos, cos, sin


@pytest.mark.parametrize("D,rot", [(64, 16), (64, 48), (128, 16), (128, 64), (128, 112), (128, 128), (64, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inf", [math.inf, -math.inf])
def test_in_the_input(D, rot, interleaved, inf):
    x, dy, w, pos, cos, sin = _case(D, rot, D + rot)
    x[torch.arange(D), 0, torch.arange(D)] = inf
    y, _ = fa.norm_rope_fwd(x.cuda(), x.cuda(), w.cuda(), w.cuda(), cos, sin, pos.int().cuda(),
                            interleaved=interleaved)
    want = plain(x, w, pos, rot, interleaved)["y"]  # NaN at the infinity (and its pair), 0 elsewhere
    assert torch.equal(torch.isnan(y).cpu(), torch.isnan(want))
    assert bool((y.cpu()[~torch.isnan(want)] == 0).all())


@pytest.mark.parametrize("D,rot", [(64, 16), (64, 48), (128, 16), (128, 64), (128, 112), (128, 128), (64, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inf", [math.inf, -math.inf])
def test_in_the_gradient(D, rot, interleaved, inf):
    """The weights' gradients of elements that no infinity reaches stay finite, and right.  (To
    plain's bound comes the rotation of dy, whose two terms may cancel: two products and a sum
    of 2^-24 and the tables' 2^-25 err by less than 2^-22 of |dy_a| + |dy_b|.)"""
    x, dy, w, pos, cos, sin = _case(D, rot, D + rot + 1)
    for d in sorted({0, 9, rot - 1, min(rot, D - 1), D - 9, D - 1}):
        bad = dy.clone()
        bad[d, 0, d] = inf
        g = fa.norm_rope_bwd(x.cuda(), x.cuda(), w.cuda(), w.cuda(), cos, sin, pos.int().cuda(),
                             bad.cuda(), bad.cuda(), interleaved=interleaved)
        r = plain(x, w, pos, rot, interleaved, dy=bad)
        clean = plain(x, w, pos, rot, interleaved, dy=dy)
        u = x.double() / (x.double().square().mean(-1, keepdim=True) + 1e-6).sqrt()
        tol = clean["dw_tol"] + 2.0 ** -22 * (partner_sum(dy.double(), rot, interleaved) * u.abs()).sum((0, 1))
        for dw in g[2:]:
            dw = dw.cpu().double()
            reached = ~torch.isfinite(r["dw"])
            assert int(reached.sum()) == (2 if d < rot else 1)
            assert torch.equal(~torch.isfinite(dw), reached)
            assert bool(((dw - clean["dw"]).abs() <= tol)[~reached].all())
        for dx, ref in ((g[0], r), (g[1], r)):
            dx = dx.cpu().double()
            rest = torch.arange(D) != d
            over = (dx - ref["dx"]).abs() - ref["dx_tol"]
            assert bool((over[rest] <= 0).all())
            assert not bool(torch.isfinite(dx[d]).any())
