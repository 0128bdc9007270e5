"""Attention of single tokens to the 4-bit cache under a window with sinks
(fa_cache4_attend_sink), and the calls around it in a run, against the plain forms."""
import ctypes
import math

import pytest
import torch

import __graft_entry__
import cache4_reference as ref
import exact_attention_blackwell_tiled_gb300 as fa
from packed_reference import assert_within
from sink_reference import packed_sinks
from test_cache4 import _cu, _filled, _i32, _kv
from test_norm_rope import plain

P = ctypes.c_void_p(256 * 1024)


def test_refusals():
    __graft_entry__.build()
    L = fa.lib()

    def call(sinks, ws=P):
        return L.fa_cache4_attend_sink(P, 512, 128, P, 4, 64, P, P, 2, 4, 2, 128, P, P, 2, 5, sinks, 0.1, None,
                                       None, 0, ws, 1 << 40, None)
    assert call(-1) == 1
    assert call(1, ws=None) == 4


@pytest.fixture(scope="module")
def gpu():
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def visible(m, wl, sinks):
    j = torch.arange(m)
    return j[(j >= m - 1 - wl) | (j < sinks)]


CASES = [
    # lengths, page, Hkv, group, window, sinks
    ([1, 0, 2, 17], 16, 1, 1, 0, 0),
    ([1, 0, 2, 17], 16, 2, 4, 0, 1),
    ([300, 31, 64], 32, 2, 5, 15, 4),
    ([300, 31, 64], 32, 2, 5, 16, 16),
    ([1000, 0, 64, 513], 64, 3, 8, 100, 17),
    ([2049, 777, 130], 128, 1, 12, 128, 33),
    ([4000], 64, 1, 40, 1000, 4),
    ([4000, 900], 16, 2, 16, 333, 0),
    ([250] * 100, 32, 4, 1, 47, 5),
    ([129] * 40, 16, 4, 2, 128, 4),               # a window that hides nothing of them
    ([40, 3000], 64, 8, 4, 2, 200),               # more sinks than the window holds
    ([5000, 4999, 4998], 64, 8, 4, 2047, 4),
]


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,page,Hkv,group,wl,sinks", CASES)
def test_attend(gpu, D, lens, page, Hkv, group, wl, sinks):
    cache, table, n, cu, k, v = _filled(lens, Hkv, D, page, fill=255)
    q = torch.randn(len(lens), Hkv * group, D, generator=torch.Generator().manual_seed(1)).to(
        torch.bfloat16)
    # entries that no visible token lies in may hold anything, and are not reported
    for b, m in enumerate(lens):
        keep = set((visible(m, wl, sinks) // page).tolist())
        for e in range(table.shape[1]):
            if e not in keep:
                table[b, e] = (-1, 2 ** 31 - 1)[e % 2]
    slots = max(lens) + 2
    w0 = torch.rand(len(lens), Hkv, slots, generator=torch.Generator().manual_seed(2))
    wd = w0.cuda()
    kw = dict(window_left=wl, sinks=sinks)
    o, lse = fa.cache4_attend(q.cuda(), cache, table, n, **kw)
    o2, lse2 = fa.cache4_attend(q.cuda(), cache, table, n, weights=wd, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    step = torch.full_like(wd, 7.0)
    fa.cache4_attend(q.cuda(), cache, table, n, weights_out=step, **kw)
    apart = torch.full_like(wd, 7.0)
    fa.cache4_attend(q.cuda(), cache, table, n, weights=w0.cuda(), weights_out=apart, **kw)
    live = (torch.arange(slots) < torch.tensor(lens)[:, None]).cuda()[:, None].expand_as(wd)
    assert torch.equal(apart[live], wd[live]) and bool((apart[~live] == 7).all())
    assert fa.cache4_status() == fa.FA_OK
    for b, m in enumerate(lens):
        j = visible(m, wl, sinks)
        r = ref.attend(q[b], k[cu[b]:cu[b + 1]][j], v[cu[b]:cu[b + 1]][j])
        if m == 0:
            assert bool((o[b] == 0).all()) and bool((lse[b] == -math.inf).all())
        else:
            assert_within(o[b], r["o"], r["o_tol"], f"o of {b}")
            assert_within(lse[b], r["lse"], r["lse_tol"], f"lse of {b}")
        p, tol = (torch.zeros(Hkv, m, dtype=torch.float64) for _ in range(2))
        p[:, j], tol[:, j] = r["p"], r["p_tol"]
        want = w0[b, :, :m].double() + p
        assert_within(wd[b, :, :m], want, tol + 2.0 ** -23 * want, f"weights of {b}")
        assert_within(step[b, :, :m], p, tol + 2.0 ** -23 * p, "step")
        assert torch.equal(wd[b, :, m:].cpu(), w0[b, :, m:])
        assert bool((step[b, :, m:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_a_window_that_hides_nothing_is_the_plain_call(gpu, D):
    lens = [900, 3, 250]
    cache, table, n, *_ = _filled(lens, 2, D, 16)
    q = torch.randn(3, 8, D, device="cuda").to(torch.bfloat16)
    a = fa.cache4_attend(q, cache, table, n)
    for kw in (dict(window_left=10 ** 12), dict(window_left=table.shape[1] * 16), dict(window_left=3, sinks=2000)):
        b = fa.cache4_attend(q, cache, table, n, **kw)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_a_bad_page_in_sight_is_reported(gpu):
    cache, table, n, cu, k, v = _filled([400], 1, 64, 16)
    q = torch.randn(1, 2, 64, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    table[0, 24] = -1                            # tokens 384 .. 399, in the window
    o, lse = fa.cache4_attend(q.cuda(), cache, table, n, window_left=100, sinks=20)
    assert fa.cache4_status() == 1
    j = visible(400, 100, 20)
    j = j[j < 384]
    r = ref.attend(q[0], k[j], v[j])
    assert_within(o[0], r["o"], r["o_tol"], "o")
    assert_within(lse[0], r["lse"], r["lse_tol"], "lse")
    # its tokens weigh nothing
    w = torch.full((1, 1, 400), 0.5, device="cuda")
    ws = torch.full((fa.cache4_attend_workspace_bytes(1, 2, 1, 64, 400),), 0xff, dtype=torch.uint8,
                    device="cuda")
    fa.cache4_attend(q.cuda(), cache, table, n, window_left=100, sinks=20, weights=w, workspace=ws)
    assert fa.cache4_status() == 1
    p, tol = (torch.zeros(1, 400, dtype=torch.float64) for _ in range(2))
    p[:, j], tol[:, j] = r["p"], r["p_tol"]
    assert_within(w[0], 0.5 + p, tol + 2.0 ** -23 * (0.5 + p), "weights")
    assert bool((w[0, 0, 384:] == 0.5).all()) and bool((w[0, 0, 20:299] == 0.5).all())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_prompts_and_steps(gpu, D):
    """The calls as a server makes them: tables, norms and rotation, attention of the prompts,
    append, then steps whose pages go back to the pool behind the window."""
    Hq, Hkv, page, wl, sinks, steps = 4, 2, 16, 50, 3, 40
    lens = [130, 1, 0, 77]
    B, T = len(lens), sum(lens)
    gen = torch.Generator().manual_seed(D)
    w = (1 + 0.2 * torch.randn(2, D, generator=gen)).to(torch.bfloat16)
    wd = w.cuda()
    cos, sin = fa.rope_table(512, D)
    width = 12
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, count = fa.page_pool(26)               # fewer than all tokens would take (30)
    cache = fa.cache4_empty(26, Hkv, D, page)
    held = _i32([0] * B)

    def projection(n):
        return torch.randn(n, Hq + 2 * Hkv, D, generator=gen).to(torch.bfloat16)

    def turned(x, pos):
        """q, k by the call, checked against the plain form, and v."""
        d = x.cuda()
        q, k, v = d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:]
        q, k = fa.norm_rope_fwd(q, k, wd[0], wd[1], cos, sin, pos)
        for i, (y, h) in enumerate(((q, slice(0, Hq)), (k, slice(Hq, Hq + Hkv)))):
            r = plain(x[:, h], w[i], pos.cpu().long(), D, False)
            assert_within(y, r["y"], r["y_tol"], "turned")
        return q, k, v

    # prompts
    new = _i32(lens)
    cu, pos, slots = fa.page_update(table, free, count, held, new, page, T, window_left=wl, sinks=sinks)
    q, k, v = turned(projection(T), pos)
    o, lse = fa.fwd_varlen(q, k, v, cu, window=(wl, 0), sinks=sinks)
    bounds = list(zip(cu.tolist(), cu.tolist()[1:]))
    r = packed_sinks(q.cpu(), k.cpu(), v.cpu(), bounds, (wl, 0), sinks)
    assert_within(o, r["o"], r["o_tol"], "prompt")
    assert_within(lse, r["lse"], r["lse_tol"], "prompt lse")
    fa.cache4_append_slots(cache, k, v, slots)
    held.copy_(new)
    seen = [(k[lo:hi].cpu(), v[lo:hi].cpu()) for lo, hi in bounds]
    # steps
    for i in range(steps):
        new = held + 1
        cu, pos, slots = fa.page_update(table, free, count, held, new, page, B, window_left=wl, sinks=sinks)
        assert pos.tolist() == held.tolist()
        q, k, v = turned(projection(B), pos)
        fa.cache4_append_slots(cache, k, v, slots)
        held.copy_(new)
        o, lse = fa.cache4_attend(q, cache, table, held, window_left=wl, sinks=sinks)
        for b in range(B):
            kk, vv = (torch.cat((x, y[b:b + 1].cpu())) for x, y in zip(seen[b], (k, v)))
            seen[b] = (kk, vv)
            j = visible(len(kk), wl, sinks)
            r = ref.attend(q[b].cpu(), kk[j], vv[j])
            assert_within(o[b], r["o"], r["o_tol"], f"step {i}, {b}")
            assert_within(lse[b], r["lse"], r["lse_tol"], f"step {i}, {b}")
    assert fa.cache4_status() == fa.FA_OK and fa.fwd_status() == fa.FA_OK
    # all sequences end: the pool is whole again
    fa.page_update(table, free, count, held, torch.zeros_like(held), page, 0, window_left=wl, sinks=sinks)
    assert count.item() == 26 and sorted(free.tolist()) == list(range(26))


@pytest.mark.gpu
def test_training_layer(gpu):
    """norm_rope and attention_varlen in one graph of torch's, against fp64: gradients of the
    projection and of the norms' weights."""
    Hq, Hkv, D, window, sinks = 4, 2, 64, (20, 0), 3
    lens = [90, 33]
    T = sum(lens)
    gen = torch.Generator().manual_seed(12)
    fused = torch.randn(T, Hq + 2 * Hkv, D, generator=gen).to(torch.bfloat16)
    w = (1 + 0.2 * torch.randn(2, D, generator=gen))
    do = torch.randn(T, Hq, D, generator=gen).to(torch.bfloat16)
    pos = torch.cat([torch.arange(n) for n in lens])
    cos, sin = fa.rope_table(128, D)
    x = fused.cuda().requires_grad_()
    wq, wk = (t.cuda().requires_grad_() for t in w)
    cu = _i32([0, 90, T])
    q, k = fa.norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], wq, wk, cos, sin, pos.int().cuda())
    o = fa.attention_varlen(q, k, x[:, Hq + Hkv:], cu, window=window, sinks=sinks, deterministic=True)
    o.backward(do.cuda())
    # the chain rule on the calls' own intermediate values, each within its bounds
    r = packed_sinks(q.detach().cpu(), k.detach().cpu(), fused[:, Hq + Hkv:], [(0, 90), (90, T)], window,
                     sinks, do=do)
    assert_within(o, r["o"], r["o_tol"], "o")
    assert_within(x.grad[:, Hq + Hkv:], r["dv"], r["dv_tol"], "dv")
    det = [t.detach() for t in (q, k, x[:, Hq + Hkv:])]
    oo, lse = fa.fwd_varlen(*det, cu, window=window, sinks=sinks)
    g = fa.bwd_varlen(*det, oo, do.cuda(), lse, cu, window=window, sinks=sinks, deterministic=True)
    for i, h in enumerate((slice(0, Hq), slice(Hq, Hq + Hkv))):
        p = plain(fused[:, h], w[i], pos, D, False, dy=g[i].cpu())
        assert_within(x.grad[:, h], p["dx"], p["dx_tol"], "dx")
        assert_within((wq, wk)[i].grad, p["dw"], p["dw_tol"], "dw")
