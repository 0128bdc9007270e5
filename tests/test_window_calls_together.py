"""The window, norm and page calls where others go on around them: streams and their pools,
threads, sequences whose neighbours hold NaN, lengths cut by the weights, the largest sides."""
import math
import threading

import pytest
import torch

import __graft_entry__
import cache4_reference as ref
import exact_attention_blackwell_tiled_gb300 as fa
from packed_reference import assert_within
from test_cache4 import _filled
from test_cache4_sinks import visible
from test_streams import _check_pool, _i32

pytestmark = pytest.mark.gpu

D, HQ, HKV, LENS = 128, 8, 2, [300, 37, 1200]
T = sum(LENS)
WINDOW = dict(window=(100, 0), sinks=4)


@pytest.fixture(scope="module", autouse=True)
def _built():
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _rows(seed=6):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(T, h, D, generator=gen).to(torch.bfloat16).cuda() for h in (HQ, HKV, HKV, HQ)]


def _turning():
    gen = torch.Generator().manual_seed(3)
    w = torch.rand(2, D, generator=gen).cuda()
    cos, sin = fa.rope_table(2000, D)
    return w[0], w[1], cos, sin, torch.randint(0, 2000, (T,), generator=gen).int().cuda()


class _Tables:
    """A step's page update that begins from the same tables in every call."""

    def __init__(self):
        self.saved = torch.full((3, 40), -1, dtype=torch.int32, device="cuda")
        self.table = self.saved.clone()
        self.stack, self.height = fa.page_pool(120)
        self.free, self.count = self.stack.clone(), self.height.clone()
        self.lens, self.new = _i32([0] * 3), _i32(LENS)

    def __call__(self, stream, **kw):
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            self.table.copy_(self.saved)
            self.free.copy_(self.stack)
            self.count.copy_(self.height)
        return fa.page_update(self.table, self.free, self.count, self.lens, self.new, 64, T, window_left=100,
                              sinks=4, stream=stream, **kw)


def test_calls_allocate_on_their_stream():
    q, k, v, do = _rows()
    cu = _i32([0, 300, 337, T])
    _check_pool(lambda s, **kw: fa.fwd_varlen(q, k, v, cu, stream=s, **WINDOW, **kw), names=("out", "lse"),
                workspace=True)
    o, lse = fa.fwd_varlen(q, k, v, cu, **WINDOW)
    _check_pool(lambda s, **kw: fa.bwd_varlen(q, k, v, o, do, lse, cu, deterministic=True, stream=s, **WINDOW, **kw),
                names=("dq", "dk", "dv"), workspace=True)
    t = _turning()
    _check_pool(lambda s, **kw: fa.norm_rope_fwd(q, k, *t, stream=s, **kw), names=("q_out", "k_out"),
                workspace=False)
    _check_pool(lambda s, **kw: fa.norm_rope_bwd(q, k, *t, do, v, stream=s, **kw),
                names=("dq", "dk", "dq_weight", "dk_weight"), workspace=True)
    _check_pool(_Tables(), names=("cu_seqlens", "positions", "slots"), workspace=False)
    _check_pool(lambda s, **kw: fa.rope_table(700, 64, stream=s), names=(), workspace=False)
    assert fa.fwd_status() == fa.FA_OK and fa.cache4_status() == fa.FA_OK


def test_threads_with_streams_of_their_own():
    q, k, v, do = _rows()
    t = _turning()
    cu = _i32([0, 300, 337, T])

    def calls(tables, cache, stream=None):
        kw = dict(stream=stream)
        cu_, pos, slots = tables(stream)
        a, b = fa.norm_rope_fwd(q, k, *t, **kw)
        o, lse = fa.fwd_varlen(a, b, v, cu, **WINDOW, **kw)
        g = fa.bwd_varlen(a, b, v, o, do, lse, cu, deterministic=True, **WINDOW, **kw)
        h = fa.norm_rope_bwd(q, k, *t, g[0], g[1], **kw)
        fa.cache4_append_slots(cache, b, v, slots, **kw)
        s = fa.cache4_attend(a[:3], cache, tables.table, tables.new, window_left=100, sinks=4, **kw)
        return (cu_, pos, slots, a, b, o, lse, *g, *h, *s)

    def own():
        return _Tables(), fa.cache4_empty(120, HKV, D, 64)

    want = calls(*own())
    torch.cuda.synchronize()
    failed = []

    def run(i):
        try:
            side = torch.cuda.Stream()
            mine = own()
            torch.cuda.synchronize()
            for _ in range(12):
                if i % 2:
                    got = calls(*mine, side)
                else:
                    with torch.cuda.stream(side):
                        got = calls(*mine)
                side.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(want, got)):
                    failed.append((i, [torch.equal(a, b) for a, b in zip(want, got)]))
        except Exception as e:  # reported by the main thread
            failed.append((i, repr(e)))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not failed
    assert fa.fwd_status() == fa.FA_OK and fa.cache4_status() == fa.FA_OK


@pytest.mark.parametrize("lens", [[33, 1, 129, 7, 200], [128, 64, 256, 63, 65], [3, 500, 17, 255, 1],
                                  [300, 385, 640, 20, 513]], ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("scale", [None, -0.2])
@pytest.mark.parametrize("window,sinks", [((20, 0), 4), ((150, 3), 40), ((5, -1), 128), ((0, 0), 1)])
@pytest.mark.parametrize("dim,Hq", [(64, 2), (64, 6), (128, 4)])
def test_foreign_rows(dim, Hq, window, sinks, scale, lens):
    """Infinities and NaN in the sequences between and in rows of none change no bit."""
    first, tail = 2, 40
    cu = torch.tensor([first, *lens]).cumsum(0)
    n = int(cu[-1]) + tail
    gen = torch.Generator().manual_seed(n)
    t = [torch.randn(n, h, dim, generator=gen).to(torch.bfloat16).cuda() for h in (Hq, 2, 2, Hq)]
    cud = cu.to(torch.int32).cuda()

    def run(fill):
        q, k, v, do = (x.clone() for x in t)
        for x in (q, k, v, do):
            for b in (1, 3):
                x[cu[b]:cu[b + 1]] = fill
            x[:first] = fill
            x[cu[-1]:] = fill
        kw = dict(scale=scale, window=window, sinks=sinks)
        o, lse = fa.fwd_varlen(q, k, v, cud, **kw)
        return o, lse.T, *fa.bwd_varlen(q, k, v, o, do, lse, cud, deterministic=True, **kw)

    clean = run(0.5)
    for fill in (math.nan, math.inf, -math.inf):
        for a, b in zip(clean, run(fill)):
            for s in (0, 2, 4):
                x, y = a[cu[s]:cu[s + 1]], b[cu[s]:cu[s + 1]]
                assert torch.equal(x, y) and bool(torch.isfinite(y.float()).all())
    assert fa.fwd_status() == fa.FA_OK


@pytest.mark.parametrize("dim", [64, 128])
def test_length_cut_by_the_weights(dim):
    """The window of a sequence that is cut is its last token's that is left."""
    lens, slots, wl, sinks = [400, 90], 250, 60, 5
    cache, table, n, cu, k, v = _filled(lens, 2, dim, 16, fill=255)
    q = torch.randn(2, 8, dim, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    w = torch.zeros(2, 2, slots, device="cuda")
    o, lse = fa.cache4_attend(q.cuda(), cache, table, n, weights=w, window_left=wl, sinks=sinks)
    assert fa.cache4_status() == 1
    for b, m in enumerate((250, 90)):
        j = visible(m, wl, sinks)
        r = ref.attend(q[b], k[cu[b]:cu[b + 1]][j], v[cu[b]:cu[b + 1]][j])
        assert_within(o[b], r["o"], r["o_tol"], f"o of {b}")
        assert_within(lse[b], r["lse"], r["lse_tol"], f"lse of {b}")
        p, tol = (torch.zeros(2, m, dtype=torch.float64) for _ in range(2))
        p[:, j], tol[:, j] = r["p"], r["p_tol"]
        assert_within(w[b, :, :m], p, tol + 2.0 ** -23 * p, "weights")


def test_the_largest_sides():
    """Windows and sinks up to 2^31 - 1 hide nothing."""
    big = 2 ** 31 - 1
    q, k, v, do = (x[:300] for x in _rows())
    cu = _i32([0, 200, 300])
    want = fa.fwd_varlen(q, k, v, cu, causal=True)
    for window in ((big, 0), (big, big), (299, big)):
        a = fa.fwd_varlen(q, k, v, cu, window=window, sinks=128)
        b = fa.fwd_varlen(q, k, v, cu, window=(-1, window[1]))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(fa.fwd_varlen(q, k, v, cu, window=(big, 0), sinks=1)[0], want[0])
    cache, table, n, *_ = _filled([900, 3], 2, 64, 16)
    q1 = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    want = fa.cache4_attend(q1, cache, table, n)
    for kw in (dict(window_left=big), dict(window_left=0, sinks=big), dict(window_left=big, sinks=big)):
        got = fa.cache4_attend(q1, cache, table, n, **kw)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    lens = _i32([100, 0])
    for kw in (dict(window_left=big, sinks=0), dict(window_left=0, sinks=big), dict()):
        t = torch.full((2, 20), -1, dtype=torch.int32, device="cuda")
        free, count = fa.page_pool(40)
        got = fa.page_update(t, free, count, torch.zeros_like(lens), lens, 16, 100, **kw)
        assert bool((got[2] >= 0).all()) and count.item() == 33
    assert fa.cache4_status() == fa.FA_OK


def test_two_graphs_in_turn():
    """Graphs of two calls with workspaces of their own, replayed in turn and side by side."""
    cu = _i32([0, 300, 337, T])
    sets, want, graphs = [_rows(s) for s in (1, 2)], [], []

    def step(q, k, v, do):
        o, lse = fa.fwd_varlen(q, k, v, cu, **WINDOW)
        return (o, *fa.bwd_varlen(q, k, v, o, do, lse, cu, deterministic=True, **WINDOW))
    for s in sets:
        want.append(step(*s))
    torch.cuda.synchronize()
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(*s)
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in sets]
    for beside in (False, True):
        for _ in range(5):
            for (g, _), st in zip(graphs, streams):
                if beside:
                    with torch.cuda.stream(st):
                        g.replay()
                else:
                    g.replay()
        torch.cuda.synchronize()
        for (_, out), w in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))
