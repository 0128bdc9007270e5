"""Rows behind the sinks count for no query whose own window begins past their tile, also
where a unit's two query tiles differ in that: the first one's window begins in the
sequence's first tile of keys, the second one's behind it."""
import math

import pytest
import torch

import __graft_entry__
import exact_attention_blackwell_tiled_gb300 as fa
from packed_reference import assert_within
from sink_reference import packed_sinks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (4, 2)])  # (an even group: two heads a unit)
@pytest.mark.parametrize("n,wl,far", [(700, 200, 384), (640, 129, 384), (1100, 450, 640), (512, 255, 384), (300, 0, 128)])
@pytest.mark.parametrize("sinks", [4, 40, 128])
@pytest.mark.parametrize("scale", [None, -0.1])
def test_pairs_of_tiles_that_differ(n, wl, far, Hq, Hkv, D, sinks, scale):
    """Queries from `far` on, the second tile of a pair, see keys from 128 on and the sinks."""
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert far % 256 == 128 and far - wl <= 255 and far - wl >= 128 > far - 128 - wl
    gen = torch.Generator().manual_seed(n + sinks)
    q, k, v, do = ((torch.randn(n, h, D, generator=gen)).to(torch.bfloat16) for h in (Hq, Hkv, Hkv, Hq))
    r = packed_sinks(q, k, v, [(0, n)], (wl, 0), sinks, scale=scale, do=do)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for bad in (math.nan, math.inf):
        kb, vb = k.clone(), v.clone()
        if sinks < 100:  # rows behind the sinks, out of sight
            kb[sinks], kb[100] = bad, -bad
            vb[sinks], vb[100], vb[127] = bad, bad, -bad
        d = [x.cuda() for x in (q, kb, vb, do)]
        o, lse = fa.fwd_varlen(*d[:3], cu, window=(wl, 0), sinks=sinks, scale=scale)
        assert fa.fwd_status() == fa.FA_OK
        assert_within(o[far:], r["o"][far:], r["o_tol"][far:], "o")
        assert_within(lse[:, far:], r["lse"][:, far:], r["lse_tol"][:, far:], "lse")
        for det in (False, True):
            dq, dk, dv = fa.bwd_varlen(*d[:3], o, d[3], lse, cu, window=(wl, 0), sinks=sinks, scale=scale,
                                       deterministic=det)
            assert_within(dq[far:], r["dq"][far:], r["dq_tol"][far:], "dq")
            for name, x in (("dk", dk), ("dv", dv)):
                assert_within(x[far:], r[name][far:], r[name + "_tol"][far:], name)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sinks", [1, 32, 33])
@pytest.mark.parametrize("wr", [0, 70, -1])
def test_every_row_of_such_pairs(D, sinks, wr):
    """All results of sequences with such a pair, next to ones without."""
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lens = [385, 384, 257, 100, 900]
    bounds, at = [], 3
    for n in lens:
        bounds.append((at, at + n))
        at += n
    gen = torch.Generator().manual_seed(sinks)
    q, k, v, do = ((torch.randn(at, h, D, generator=gen)).to(torch.bfloat16) for h in (3, 1, 1, 3))
    cu = torch.tensor([3] + [hi for _, hi in bounds], dtype=torch.int32, device="cuda")
    d = [x.cuda() for x in (q, k, v, do)]
    for wl in (130, 200, 256):
        r = packed_sinks(q, k, v, bounds, (wl, wr), sinks, do=do)
        o, lse = fa.fwd_varlen(*d[:3], cu, window=(wl, wr), sinks=sinks)
        assert fa.fwd_status() == fa.FA_OK
        assert_within(o, r["o"], r["o_tol"], "o")
        assert_within(lse, r["lse"], r["lse_tol"], "lse")
        g = fa.bwd_varlen(*d[:3], o, d[3], lse, cu, window=(wl, wr), sinks=sinks)
        for name, x in zip(("dq", "dk", "dv"), g):
            assert_within(x, r[name], r[name + "_tol"], name)
