"""Packed attention under a window with sinks (fa_fwd_varlen_sink, fa_bwd_varlen_sink)
against the plain 64-bit form."""
import ctypes
import math

import pytest
import torch

import __graft_entry__
import exact_attention_blackwell_tiled_gb300 as fa
from packed_reference import assert_within
from sink_reference import packed_sinks, sink_mask

P256 = ctypes.c_void_p(256 * 1024)
P16 = ctypes.c_void_p(256 * 1024 + 16)


# ------------------------------------------------------------------ without a GPU

@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return fa.lib()


def test_refusals(L):
    def fwd(sinks, T=8, ws=P256, need=1 << 20):
        return L.fa_fwd_varlen_sink(P16, P16, P16, P16, P16, P16, 2, T, 2, 2, 64, None, None, None,
                                    4, 0, sinks, 0.1, ws, need, None)

    def bwd(sinks, T=8, need=None):
        need = L.fa_varlen_sink_workspace_bytes(2, 8, 2, 2, 64, 1, 0, 4, 4) if need is None else need
        return L.fa_bwd_varlen_sink(P16, P16, P16, P16, P16, P16, P16, P16, P16, P16, 2, T, 2, 2, 64,
                                    None, None, None, 4, 0, sinks, 0.1, P256, need, 0, None)
    assert fwd(-1) == 1 and bwd(-1) == 1
    assert fwd(129) == 2 and bwd(129) == 2
    assert fwd(4, T=0) == 0 and bwd(4, T=0) == 0
    assert fwd(4, ws=None) == 4
    plain = L.fa_varlen_workspace_bytes(2, 8, 2, 2, 64, 1, 0)
    assert bwd(4, need=plain) == 4
    assert L.fa_varlen_sink_workspace_bytes(2, 8, 2, 2, 64, 1, 0, 4, 129) == 0
    assert L.fa_varlen_sink_workspace_bytes(2, 8, 2, 2, 64, 1, 0, 4, -1) == 0
    # without sinks, or with a window that hides nothing, it is the plain call's
    for wl, sinks in ((4, 0), (-1, 4), (7, 4), (1 << 30, 4)):
        assert L.fa_varlen_sink_workspace_bytes(2, 8, 2, 2, 64, 1, 1, wl, sinks) == \
            L.fa_varlen_workspace_bytes(2, 8, 2, 2, 64, 1, 1)


def test_workspace_grows_with_what_it_holds(L):
    """Parts take rows for runs of queries, not rows per token: 16384 tokens of 16 heads of
    128 under 1024 with 4 sinks cost far below one accumulator more."""
    plain = L.fa_varlen_workspace_bytes(4, 16384, 16, 16, 128, 1, 0)
    more = L.fa_varlen_sink_workspace_bytes(4, 16384, 16, 16, 128, 1, 0, 1023, 4)
    assert 0 < more - plain < 16384 * 16 * 128 * 4 // 4
    # the narrowest window with the most sinks stays within a few of them
    worst = L.fa_varlen_sink_workspace_bytes(4, 16384, 16, 16, 128, 1, 0, 0, 128)
    assert worst - plain < 10 * 16384 * 16 * 128 * 4


def _slot(wl, sinks, row0, tile):
    return ((row0 // 128 + row0 // (wl + 2) + tile) * sinks if wl + 2 >= sinks
            else (row0 // 128 + tile) * sinks + row0)


@pytest.mark.parametrize("wl,sinks", [(0, 1), (0, 128), (1, 4), (2, 4), (3, 4), (63, 64), (61, 64),
                                      (100, 4), (127, 128), (126, 128), (500, 16)])
def test_parts_do_not_meet(L, wl, sinks):
    """The rows of the sinks' parts, per head, by their closed form: no two tiles of long
    sequences share one, and all lie inside the workspace's count."""
    import random
    rng = random.Random(wl * 1000 + sinks)
    for _ in range(60):
        used, row0 = set(), rng.randrange(0, 5)
        for _ in range(rng.randrange(1, 60)):
            n = rng.choice([0, 1, 2, wl + 1, wl + 2, wl + 3, 127, 128, 129, 300, 1000])
            if n > wl + 1:
                for tile in range(-(-n // 128)):
                    first = _slot(wl, sinks, row0, tile)
                    rows = range(first, first + min(sinks, n))
                    assert used.isdisjoint(rows)
                    used.update(rows)
            row0 += n
        T = row0
        bound = ((T // 128 + T // (wl + 2) + 2) * sinks if wl + 2 >= sinks
                 else (T // 128 + 2) * sinks + T)
        assert not used or max(used) < bound


def test_reference_gradients_by_differences():
    gen = torch.Generator().manual_seed(3)
    n, D, window, sinks = 7, 4, (2, 0), 2
    x = [torch.randn(n, 1, D, generator=gen, dtype=torch.float64) for _ in range(4)]
    q, k, v, do = x
    r = packed_sinks(q, k, v, [(0, n)], window, sinks, scale=0.7, do=do)
    mask = sink_mask(n, window, sinks)
    assert mask[6].tolist() == [True, True, False, False, True, True, True]

    def loss(q, k, v):
        s = (q[:, 0] @ k[:, 0].T * 0.7).masked_fill(~mask, -math.inf)
        return float(((torch.softmax(s, 1) @ v[:, 0]) * do[:, 0]).sum())
    for name, t in (("dq", 0), ("dk", 1), ("dv", 2)):
        for at in ((0, 0, 1), (3, 0, 0), (6, 0, 3)):
            args = [y.clone() for y in (q, k, v)]
            eps = 1e-6
            args[t][at] += eps
            up = loss(*args)
            args[t][at] -= 2 * eps
            diff = (up - loss(*args)) / (2 * eps)
            assert abs(diff - float(r[name][at])) < 1e-7


# ------------------------------------------------------------------ on the GPU

def _inputs(T, Hq, Hkv, D, seed, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(T, h, D, generator=gen) * spread).to(torch.bfloat16)
            for h in (Hq, Hkv, Hkv, Hq)]


def _bounds(lens, first=0):
    out, at = [], first
    for n in lens:
        out.append((at, at + n))
        at += n
    return out


def _cu(bounds):
    return torch.tensor([bounds[0][0]] + [hi for _, hi in bounds], dtype=torch.int32, device="cuda")


CASES = [
    # lengths, Hq, Hkv, D, window, sinks
    ([1, 0, 2, 130, 5], 2, 2, 64, (0, 0), 1),
    ([1, 0, 2, 130, 5], 2, 1, 128, (1, 0), 4),
    ([300], 2, 2, 128, (63, 0), 4),
    ([700, 129, 128, 127], 2, 2, 64, (100, 0), 16),
    ([513, 900], 4, 2, 128, (200, 0), 7),
    ([513, 900], 4, 2, 64, (200, 0), 33),
    ([640, 257], 2, 1, 128, (130, 3), 128),       # the widest sinks, a right side
    ([640, 257], 2, 1, 64, (130, -1), 65),        # no right side
    ([400, 90], 3, 3, 128, (10, 0), 64),          # more sinks than the window holds
    ([400, 90], 3, 3, 64, (2, 0), 100),
    ([1200], 8, 1, 128, (127, 0), 4),
    ([1200, 1200], 1, 1, 64, (255, 0), 17),
    ([40] * 30 + [500], 4, 4, 64, (37, 0), 3),
    ([40] * 30 + [500], 4, 4, 128, (38, 0), 3),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Hq,Hkv,D,window,sinks", CASES)
def test_forward_and_backward(lens, Hq, Hkv, D, window, sinks):
    __graft_entry__.build()
    bounds = _bounds(lens)
    T = bounds[-1][1]
    q, k, v, do = _inputs(T, Hq, Hkv, D, 17 + T)
    r = packed_sinks(q, k, v, bounds, window, sinks, do=do)
    cu = _cu(bounds)
    d = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.fwd_varlen(*d[:3], cu, window=window, sinks=sinks)
    assert fa.fwd_status() == fa.FA_OK
    assert_within(o, r["o"], r["o_tol"], "o")
    assert_within(lse, r["lse"], r["lse_tol"], "lse")
    for det in (False, True):
        ws = torch.full((fa.varlen_workspace_bytes(len(lens), T, Hq, Hkv, D, True, det, window=window,
                                                   sinks=sinks),), 0xff, dtype=torch.uint8, device="cuda")
        g = fa.bwd_varlen(*d[:3], o, d[3], lse, cu, window=window, sinks=sinks, deterministic=det,
                          workspace=ws)
        assert fa.bwd_status(ws) == fa.FA_OK
        for name, x in zip(("dq", "dk", "dv"), g):
            assert_within(x, r[name], r[name + "_tol"], f"{name}, deterministic={det}")
        if det:
            for _ in range(3):
                again = fa.bwd_varlen(*d[:3], o, d[3], lse, cu, window=window, sinks=sinks,
                                      deterministic=True)
                assert all(torch.equal(x, y) for x, y in zip(g, again))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("det", [False, True])
def test_large_scores_and_strides(D, det):
    """Slices of a fused projection, scores far apart, a negative scale too; tokens in front
    of the first and behind the last sequence stay as they were and may be NaN."""
    __graft_entry__.build()
    Hq, Hkv, window, sinks = 4, 2, (70, 0), 5
    bounds = _bounds([333, 0, 150], first=9)
    T = bounds[-1][1] + 11
    gen = torch.Generator().manual_seed(5)
    fused = (torch.randn(T, Hq + 2 * Hkv, D, generator=gen) * 3).to(torch.bfloat16)
    do = torch.randn(T, Hq, D, generator=gen).to(torch.bfloat16)
    for rows in (slice(0, 9), slice(T - 11, T)):
        fused[rows] = math.nan
    dev = fused.cuda()
    parts = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    cu = _cu(bounds)
    for scale in (None, -0.05, 0.0):
        r = packed_sinks(*(x.cpu() for x in parts), bounds, window, sinks, scale=scale, do=do)
        o = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((Hq, T), 7.0, device="cuda")
        fa.fwd_varlen(*parts, cu, window=window, sinks=sinks, scale=scale, out=o, lse=lse)
        assert_within(o, r["o"], r["o_tol"], "o")
        assert_within(lse, r["lse"], r["lse_tol"], "lse")
        grads = [torch.full((T, h, D), 7.0, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv)]
        fa.bwd_varlen(*parts, o, do.cuda(), lse, cu, window=window, sinks=sinks, scale=scale,
                      deterministic=det, dq=grads[0], dk=grads[1], dv=grads[2])
        for name, x in zip(("dq", "dk", "dv"), grads):
            assert_within(x, r[name], r[name + "_tol"], name)
        for x in (o, *grads):
            assert bool((x[:9] == 7).all()) and bool((x[-11:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sinks", [4, 40])
@pytest.mark.parametrize("det", [False, True])
def test_nan_and_infinity_out_of_sight(D, sinks, det):
    """Keys behind the sinks, in their tile, reach no query whose tiles of the window begin
    further on: neither through a weight of zero nor through a masked score."""
    __graft_entry__.build()
    n, window = 700, (100, 0)
    q, k, v, do = _inputs(n, 2, 1, D, 23)
    r = packed_sinks(q, k, v, [(0, n)], window, sinks, do=do)
    far = 384                                  # queries from here on see keys from 284 on
    for bad in (math.nan, math.inf):
        kb, vb = k.clone(), v.clone()
        kb[sinks], kb[100] = bad, -bad
        vb[sinks + 1], vb[127] = bad, -bad
        d = [x.cuda() for x in (q, kb, vb, do)]
        cu = _cu([(0, n)])
        o, lse = fa.fwd_varlen(*d[:3], cu, window=window, sinks=sinks)
        assert_within(o[far:], r["o"][far:], r["o_tol"][far:], "o")
        assert_within(lse[:, far:], r["lse"][:, far:], r["lse_tol"][:, far:], "lse")
        dq, dk, dv = fa.bwd_varlen(*d[:3], o, d[3], lse, cu, window=window, sinks=sinks, deterministic=det)
        assert_within(dq[far:], r["dq"][far:], r["dq_tol"][far:], "dq")
        for name, x in (("dk", dk), ("dv", dv)):
            assert_within(x[far:], r[name][far:], r[name + "_tol"][far:], name)


@pytest.mark.gpu
def test_a_window_that_hides_nothing_is_the_plain_call():
    __graft_entry__.build()
    q, k, v, do = (x.cuda() for x in _inputs(500, 4, 2, 128, 1))
    cu = _cu(_bounds([200, 300]))
    for window in ((499, 0), (-1, 0), (2 ** 31 - 1, 0)):
        a = fa.fwd_varlen(q, k, v, cu, window=window, sinks=4)
        b = fa.fwd_varlen(q, k, v, cu, window=window)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        ga, gb = (fa.bwd_varlen(q, k, v, *b[:1], do, b[1], cu, window=window, deterministic=True,
                                sinks=s) for s in (4, 0))
        assert all(torch.equal(x, y) for x, y in zip(ga, gb))


@pytest.mark.gpu
def test_autograd_and_capture():
    """attention_varlen's gradients are the calls'; a captured step replays on new lengths."""
    __graft_entry__.build()
    window, sinks, T, Hq, Hkv, D = (50, 0), 4, 600, 4, 2, 64
    x = _inputs(T, Hq, Hkv, D, 2)
    q, k, v = (t.cuda().requires_grad_() for t in x[:3])
    do = x[3].cuda()
    cu = _cu(_bounds([250, 350]))
    o = fa.attention_varlen(q, k, v, cu, window=window, sinks=sinks, deterministic=True)
    o.backward(do)
    oo, lse = fa.fwd_varlen(q.detach(), k.detach(), v.detach(), cu, window=window, sinks=sinks)
    g = fa.bwd_varlen(q.detach(), k.detach(), v.detach(), oo, do, lse, cu, window=window,
                      sinks=sinks, deterministic=True)
    assert torch.equal(o, oo)
    assert all(torch.equal(a.grad, b) for a, b in zip((q, k, v), g))

    d = [t.cuda() for t in x[:3]]

    def step():
        oo, lse = fa.fwd_varlen(*d, cu, window=window, sinks=sinks)
        return (oo, *fa.bwd_varlen(*d, oo, do, lse, cu, window=window, sinks=sinks, deterministic=True))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for lens in ([250, 350], [1, 599], [600, 0]):
        cu.copy_(_cu(_bounds(lens)))
        d[0].copy_(torch.randn(T, Hq, D, generator=torch.Generator().manual_seed(lens[0])))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


@pytest.mark.gpu
def test_two_streams():
    __graft_entry__.build()
    window, sinks = (300, 0), 20
    sets = [[t.cuda() for t in _inputs(2000, 4, 2, 128, s)] for s in (1, 2)]
    cu = _cu(_bounds([1500, 500]))

    def step(q, k, v, do):
        o, lse = fa.fwd_varlen(q, k, v, cu, window=window, sinks=sinks)
        return (o, *fa.bwd_varlen(q, k, v, o, do, lse, cu, window=window, sinks=sinks, deterministic=True))
    want = [step(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[] for _ in sets]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(*sets[i]))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for g in runs:
            assert all(torch.equal(a, b) for a, b in zip(w, g))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("det", [False, True])
def test_long_sequences_in_many_shares(D, det):
    """A sequence whose sinks' parts come from many blocks, next to short ones; sampled rows
    and the sinks' gradients against the plain form."""
    __graft_entry__.build()
    Hq, Hkv, window, sinks = 4, 2, (300, 0), 6
    bounds = _bounds([50, 5000, 1, 700])
    T = bounds[-1][1]
    q, k, v, do = (x.cuda() for x in _inputs(T, Hq, Hkv, D, 77))
    cu = _cu(bounds)
    o, lse = fa.fwd_varlen(q, k, v, cu, window=window, sinks=sinks)
    g = fa.bwd_varlen(q, k, v, o, do, lse, cu, window=window, sinks=sinks, deterministic=det)
    # the long sequence by itself, in fp64 on the GPU, and the bounds of its sinks' rows
    lo, hi = bounds[1]
    n = hi - lo
    i = torch.arange(n, device="cuda")
    mask = (i[None] <= i[:, None]) & ((i[None] >= i[:, None] - window[0]) | (i[None] < sinks))
    scale, u = 1 / math.sqrt(D), 2.0 ** -8
    dk, dv = (torch.zeros(n, Hkv, D, dtype=torch.float64, device="cuda") for _ in range(2))
    dk_tol, dv_tol = torch.zeros_like(dk), torch.zeros_like(dv)
    for h in range(Hq):
        qh, doh = q[lo:hi, h].double(), do[lo:hi, h].double()
        kh, vh = k[lo:hi, h // 2].double(), v[lo:hi, h // 2].double()
        s = (qh @ kh.T * scale).masked_fill(~mask, -math.inf)
        z = torch.logsumexp(s, 1, keepdim=True)
        p = (s - z).exp()
        out = p @ vh
        e_s = (D + 8) * 2.0 ** -23 * scale * (qh.abs() @ kh.abs().T).masked_fill(~mask, 0).amax(1, keepdim=True)
        o_tol = u * out.abs() + (u + 2 * e_s + n * 2.0 ** -23) * (p @ vh.abs())
        assert bool(((o[lo:hi, h].double() - out).abs() <= o_tol).all())
        dp = doh @ vh.T
        ds = p * (dp - (doh * out).sum(1, keepdim=True))
        e_dp = (D + 2) * 2.0 ** -23 * (doh.abs() @ vh.abs().T)
        e_delta = (doh.abs() * o_tol).sum(1, keepdim=True) + (D + 2) * 2.0 ** -23 * (doh * out).abs().sum(1, keepdim=True)
        e_ds = (u + 2 * e_s + n * 2.0 ** -23) * ds.abs() + p * (e_delta + e_dp)
        dq = ds @ kh * scale
        dq_tol = u * dq.abs() + scale * (e_ds @ kh.abs())
        assert bool(((g[0][lo:hi, h].double() - dq).abs() <= dq_tol).all())
        dv[:, h // 2] += p.T @ doh
        dv_tol[:, h // 2] += (p * (u + 2 * e_s + n * 2.0 ** -23)).T @ doh.abs()
        dk[:, h // 2] += ds.T @ qh * scale
        dk_tol[:, h // 2] += scale * (e_ds.T @ qh.abs())
    for x, ref, tol in ((g[1], dk, dk_tol), (g[2], dv, dv_tol)):
        assert bool(((x[lo:hi].double() - ref).abs() <= tol + u * ref.abs()).all())


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Hq,Hkv,D,window,sinks", [
    ([700, 300], 7, 1, 64, (100, 0), 4),              # an odd group
    ([40] * 30 + [500], 8, 2, 64, (37, 0), 3),        # many short sequences, an even one
    ([40] * 30 + [500], 8, 2, 128, (37, 0), 40),
    ([90] * 16, 4, 2, 128, (20, 0), 2),               # the most sequences that a block plans
    ([90] * 17, 4, 2, 128, (20, 0), 2),
    ([200] * 10, 4, 1, 64, (50, 0), 2),
    ([200] * 11, 4, 1, 64, (50, 0), 2),
    ([500, 300], 4, 2, 128, (-1, 7), 0),              # windows without sinks, open to the left
    ([500, 300], 4, 2, 64, (30, -1), 0),              # and to the right
    ([500, 300], 4, 4, 64, (30, 9), 0),
])
def test_units_of_every_kind(lens, Hq, Hkv, D, window, sinks):
    """Two tiles of a head or two heads of a tile, planned by a launch or by each block."""
    test_forward_and_backward(lens, Hq, Hkv, D, window, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [3, 40])
@pytest.mark.parametrize("group", [1, 2])
def test_boundaries_out_of_order(B, group):
    """Recorded, and nothing is written, whoever plans the call."""
    __graft_entry__.build()
    T, D, window, sinks = 40 * B, 64, (20, 0), 3
    q, k, v, do = (x.cuda() for x in _inputs(T, 2 * group, 2, D, B))
    for bad in (T + 1, -1, 41):
        cu = _cu(_bounds([40] * B))
        cu[B if bad > T else 1 if bad < 0 else 2] = bad if bad != 41 else 39
        o = torch.full_like(q, 7.0)
        lse = torch.full((2 * group, T), 7.0, device="cuda")
        fa.fwd_varlen(q, k, v, cu, window=window, sinks=sinks, out=o, lse=lse)
        assert fa.fwd_status() == 1
        assert bool((o == 7).all()) and bool((lse == 7).all())
        for det in (False, True):
            ws = torch.empty(fa.varlen_workspace_bytes(B, T, 2 * group, 2, D, True, det, window=window,
                                                       sinks=sinks), dtype=torch.uint8, device="cuda")
            g = [torch.full_like(x, 7.0) for x in (q, k, v)]
            fa.bwd_varlen(q, k, v, o, do, lse, cu, window=window, sinks=sinks, deterministic=det,
                          workspace=ws, dq=g[0], dk=g[1], dv=g[2])
            assert fa.bwd_status(ws) == 1
            assert all(bool((x == 7).all()) for x in g)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [2, 30])
@pytest.mark.parametrize("Hq", [2, 4])
def test_nothing_but_empty_sequences(B, Hq):
    """Rows of no sequence are left as they were, in every result."""
    __graft_entry__.build()
    T, D, window, sinks = 3000, 128, (20, 0), 3  # (the window hides keys in T rows)
    q, k, v, do = (x.cuda() for x in _inputs(T, Hq, 2, D, 4))
    for at in (0, 7, T):
        cu = torch.full((B + 1,), at, dtype=torch.int32, device="cuda")
        o, lse = torch.full_like(q, 7.0), torch.full((Hq, T), 7.0, device="cuda")
        fa.fwd_varlen(q, k, v, cu, window=window, sinks=sinks, out=o, lse=lse)
        assert fa.fwd_status() == fa.FA_OK and bool((o == 7).all()) and bool((lse == 7).all())
        for det in (False, True):
            g = [torch.full_like(x, 7.0) for x in (q, k, v)]
            fa.bwd_varlen(q, k, v, o, do, lse, cu, window=window, sinks=sinks, deterministic=det,
                          dq=g[0], dk=g[1], dv=g[2])
            assert all(bool((x == 7).all()) for x in g)


@pytest.mark.gpu
def test_a_captured_call_follows_its_boundaries():
    """One graph, replayed for other boundaries, planned by its blocks and by a launch."""
    __graft_entry__.build()
    Hq, Hkv, D, window, sinks, T = 4, 2, 64, (40, 0), 5, 600
    q, k, v, do = (x.cuda() for x in _inputs(T, Hq, Hkv, D, 8))
    for B in (4, 24):
        cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        o, lse = torch.zeros_like(q), torch.zeros(Hq, T, device="cuda")
        g = [torch.zeros_like(x) for x in (q, k, v)]

        def step():
            fa.fwd_varlen(q, k, v, cu, window=window, sinks=sinks, out=o, lse=lse)
            fa.bwd_varlen(q, k, v, o, do, lse, cu, window=window, sinks=sinks, deterministic=True,
                          dq=g[0], dk=g[1], dv=g[2])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        gen = torch.Generator().manual_seed(B)
        for _ in range(4):
            cuts = torch.randint(0, T + 1, (B + 1,), generator=gen).sort().values.to(torch.int32)
            cu.copy_(cuts.cuda())
            for x in (o, lse, *g):
                x.fill_(3.0)
            graph.replay()
            got = [x.clone() for x in (o, lse, *g)]
            for x in (o, lse, *g):
                x.fill_(3.0)
            step()
            assert all(torch.equal(x, y) for x, y in zip(got, (o, lse, *g)))
            bounds = list(zip(cuts[:-1].tolist(), cuts[1:].tolist()))
            r = packed_sinks(q.cpu(), k.cpu(), v.cpu(), bounds, window, sinks, do=do.cpu())
            assert_within(o, r["o"], r["o_tol"], "o")
            for name, x in zip(("dq", "dk", "dv"), g):
                assert_within(x, r[name], r[name + "_tol"], name)
        del graph
    assert fa.fwd_status() == fa.FA_OK
