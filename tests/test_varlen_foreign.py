"""Infinities and NaN in other sequences' rows, before the first and behind the last,
change no bit of a sequence's results, under every mask and scale."""
import pytest
import torch

import __graft_entry__
import exact_attention_blackwell_tiled_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("lens", [[33, 1, 129, 7, 200], [128, 64, 256, 63, 65], [3, 500, 17, 255, 1]],
                         ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("scale", [None, 0.0, -0.2])
@pytest.mark.parametrize("window", [(-1, 0), (-1, -1), (20, 3), (5, -1)], ids=lambda w: "%d,%d" % w)
@pytest.mark.parametrize("D", [64, 128])
def test_foreign_rows(D, window, scale, lens):
    first, tail = 2, 40
    cu = torch.tensor([first, *lens]).cumsum(0)
    T = int(cu[-1]) + tail
    gen = torch.Generator().manual_seed(T)
    t = [torch.randn(T, h, D, generator=gen).to(torch.bfloat16).cuda() for h in (4, 2, 2, 4)]
    cud = cu.to(torch.int32).cuda()

    def run(fill):
        q, k, v, do = (x.clone() for x in t)
        for x in (q, k, v, do):
            for b in (1, 3):  # every other sequence, and the rows of none
                x[cu[b]:cu[b + 1]] = fill
            x[:first] = fill
            x[cu[-1]:] = fill
        o, lse = fa.fwd_varlen(q, k, v, cud, scale=scale, window=window)
        grads = fa.bwd_varlen(q, k, v, o, do, lse, cud, scale=scale, window=window, deterministic=True)
        return o, lse.T, *grads

    clean = run(0.5)
    for fill in (float("nan"), float("inf"), float("-inf")):
        for a, b in zip(clean, run(fill)):
            for s in (0, 2, 4):
                x, y = a[cu[s]:cu[s + 1]], b[cu[s]:cu[s + 1]]
                assert torch.equal(x, y) and bool(torch.isfinite(y.float()).all())
    assert fa.fwd_status() == fa.FA_OK
