"""Windows wider than any sequence, up to the widest an int holds: every distance lies
inside, in the forward and in the gradients."""
import pytest
import torch

import __graft_entry__
import exact_attention_blackwell_tiled_gb300 as fa
import oracle
import synth
from packed_reference import assert_within, packed
from parity_helpers import assert_fwd_rows, assert_grad_close

pytestmark = pytest.mark.gpu

WIDEST = 2 ** 31 - 1
WINDOWS = [(WIDEST, 0), (-1, WIDEST), (WIDEST, WIDEST), (WIDEST - 200, 3), (40, WIDEST - 300)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", WINDOWS, ids=lambda w: "%d,%d" % w)
def test_packed(D, window):
    gen = torch.Generator().manual_seed(12)
    bounds = [(0, 150), (150, 151), (151, 530)]
    q, k, v, do = (torch.randn(530, h, D, generator=gen).to(torch.bfloat16) for h in (4, 2, 2, 4))
    ref = packed(q, k, v, bounds, window=window, do=do)
    qd, kd, vd, dod = (x.cuda() for x in (q, k, v, do))
    cu = torch.tensor([0, 150, 151, 530], dtype=torch.int32, device="cuda")
    o, lse = fa.fwd_varlen(qd, kd, vd, cu, window=window)
    assert_within(o, ref["o"], ref["o_tol"], "o")
    assert_within(lse, ref["lse"], ref["lse_tol"], "lse")
    for det in (False, True):
        grads = fa.bwd_varlen(qd, kd, vd, o, dod, lse, cu, window=window, deterministic=det)
        for g, n in zip(grads, ("dq", "dk", "dv")):
            assert_within(g, ref[n], ref[n + "_tol"], f"{n} det={det}")
    assert fa.fwd_status() == fa.FA_OK


@pytest.mark.parametrize("Sq,Sk", [(300, 300), (130, 500), (500, 130)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", WINDOWS, ids=lambda w: "%d,%d" % w)
def test_dense(D, window, Sq, Sk):
    """fwd, the split form and both backward modes; the oracle gets the window cut to the
    rows there are."""
    w = synth.Workload("wide", 1, 4, 2, Sq, Sk, D, False, 8, with_do=True)
    q, k, v, do = synth.make_inputs(w, with_do=True)
    wl, wr = (x if x < 0 else min(x, Sq + Sk) for x in window)
    o_r, lse_r = oracle.fwd_mod(q, k, v, w.softmax_scale, wl, wr)
    qd, kd, vd, dod = (x.cuda() for x in (q, k, v, do))
    kw = dict(scale=w.softmax_scale, window=window)
    o, lse = fa.fwd(qd, kd, vd, **kw)
    assert_fwd_rows(o, lse, o_r, lse_r, "forward")
    assert_fwd_rows(*fa.fwd(qd, kd, vd, n_splits=2, **kw), o_r, lse_r, "split")
    grads_r = oracle.bwd_mod(q, k, v, do, w.softmax_scale, wl, wr)
    for det in (False, True):
        for g, r, n in zip(fa.bwd(qd, kd, vd, o, dod, lse, deterministic=det, **kw), grads_r,
                           ("dq", "dk", "dv")):
            assert_grad_close(g, r, f"{n} det={det}")
    assert fa.fwd_status() == fa.FA_OK
