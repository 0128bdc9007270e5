"""The sinks' parts in the backward's workspace: rows counted by the library, a workspace of
exactly its size between guards, and results where parts of neighbours lie side by side."""
import random

import pytest
import torch

import __graft_entry__
import exact_attention_blackwell_tiled_gb300 as fa
from packed_reference import assert_within
from sink_reference import packed_sinks
from test_sinks import _slot

EDGES = [(0, 1), (0, 2), (0, 3), (0, 128), (1, 3), (1, 4), (2, 4), (3, 4), (61, 64), (62, 64), (63, 64),
         (125, 128), (126, 128), (127, 128), (128, 128), (500, 16)]


def _rows(B, T, wl, sinks):
    """Rows per head of each of the four arrays: of one head of 64 a row is 256 bytes, which
    sizes are rounded to."""
    size = fa.varlen_workspace_bytes(B, T, 1, 1, 64, True, False, window=(wl, 0), sinks=sinks)
    more = size - fa.varlen_workspace_bytes(B, T, 1, 1, 64, True, False)
    assert more % (4 * 256) == 0
    return more // (4 * 256)


def _lengths(rng, wl, sinks):
    return [rng.choice([1, 2, wl + 1, wl + 2, wl + 3, sinks, 127, 128, 129, 300]) for _ in range(rng.randrange(2, 24))]


@pytest.mark.parametrize("wl,sinks", EDGES)
def test_slots_lie_in_the_library_s_count(wl, sinks):
    __graft_entry__.build()
    rng = random.Random(wl * 1000 + sinks)
    for _ in range(200):
        lens, row0, top = _lengths(rng, wl, sinks), rng.randrange(0, 400), 0
        for n in lens:
            if n > wl + 1:
                top = max(top, _slot(wl, sinks, row0, -(-n // 128) - 1) + min(sinks, n))
            row0 += n
        if wl < row0 - 1:
            assert top <= _rows(len(lens), row0, wl, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("wl,sinks", EDGES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1)])
def test_between_guards(wl, sinks, D, Hq, Hkv):
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rng = random.Random(wl * 1000 + sinks + D)
    for first in (0, 129):
        lens = _lengths(rng, wl, sinks) + [wl + 2, wl + 2, max(wl + 2, 129)]
        bounds, at = [], first
        for n in lens:
            bounds.append((at, at + n))
            at += n
        gen = torch.Generator().manual_seed(at)
        q, k, v, do = (torch.randn(at, h, D, generator=gen).to(torch.bfloat16) for h in (Hq, Hkv, Hkv, Hq))
        r = packed_sinks(q, k, v, bounds, (wl, 0), sinks, do=do)
        d = [x.cuda() for x in (q, k, v, do)]
        cu = torch.tensor([first] + [hi for _, hi in bounds], dtype=torch.int32, device="cuda")
        o, lse = fa.fwd_varlen(*d[:3], cu, window=(wl, 0), sinks=sinks)
        for det in (False, True):
            size = fa.varlen_workspace_bytes(len(lens), at, Hq, Hkv, D, True, det, window=(wl, 0), sinks=sinks)
            room = torch.full((size + 8192,), 0xff, dtype=torch.uint8, device="cuda")
            g = fa.bwd_varlen(*d[:3], o, d[3], lse, cu, window=(wl, 0), sinks=sinks, deterministic=det,
                              workspace=room[4096:4096 + size])
            assert bool((room[:4096] == 0xff).all()) and bool((room[4096 + size:] == 0xff).all())
            for name, x in zip(("dq", "dk", "dv"), g):
                assert_within(x, r[name], r[name + "_tol"], f"{name}, deterministic={det}")
