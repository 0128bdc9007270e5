"""Attention over packed sequences (fa_fwd_varlen, fa_bwd_varlen) against the plain
64-bit form, sequence by sequence."""
import ctypes
import math

import pytest
import torch

import __graft_entry__
import exact_attention_blackwell_tiled_gb300 as fa
from packed_reference import assert_within, mask_of, one_head, packed

P256 = ctypes.c_void_p(256 * 1024)
P16 = ctypes.c_void_p(256 * 1024 + 16)
P17 = ctypes.c_void_p(256 * 1024 + 17)


# ------------------------------------------------------------------ without a GPU

@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return fa.lib()


def _fwd(L, q=P16, k=P16, v=P16, o=P16, lse=P16, cu=P16, B=2, T=8, Hq=2, Hkv=2, D=64, qs=None,
         ws=P256, wsb=None, scale=0.1):
    wsb = L.fa_varlen_workspace_bytes(2, 8, 2, 2, 64, 0, 0) if wsb is None else wsb
    return L.fa_fwd_varlen(q, k, v, o, lse, cu, B, T, Hq, Hkv, D,
                           None if qs is None else ctypes.byref(fa.PackedStride(*qs)), None, None,
                           -1, 0, scale, ws, wsb, None)


def test_forward_refusals(L):
    assert _fwd(L, B=0) == 1
    assert _fwd(L, T=-1) == 1
    assert _fwd(L, Hq=3, Hkv=2) == 1
    assert _fwd(L, D=96) == 2
    assert _fwd(L, scale=math.inf) == 1
    assert _fwd(L, q=None) == 1
    assert _fwd(L, cu=None) == 1
    assert _fwd(L, o=P17) == 3
    assert _fwd(L, lse=P17) == 3
    assert _fwd(L, qs=(132, 64)) == 3     # rows 264 bytes apart
    assert _fwd(L, qs=(128, 56)) == 1     # heads overlap
    assert _fwd(L, qs=(0, 64)) == 1       # a broadcast input
    assert _fwd(L, ws=None) == 4
    assert _fwd(L, ws=P16) == 4
    assert _fwd(L, wsb=L.fa_varlen_workspace_bytes(2, 8, 2, 2, 64, 0, 0) - 1) == 4
    assert _fwd(L, T=0, q=None, cu=None, ws=None) == 0
    assert _fwd(L, T=1 << 30, Hq=2) == 1  # rows over all heads pass 32 bits
    assert _fwd(L, B=(1 << 18) + 1) == 1  # more sequences than a plan is made for


def test_backward_refusals(L):
    need = L.fa_varlen_workspace_bytes(2, 8, 2, 2, 64, 1, 1)

    def bwd(do=P16, dq=P16, ws=P256, wsb=need, T=8, D=64):
        return L.fa_bwd_varlen(P16, P16, P16, P16, do, P16, dq, P16, P16, P16, 2, T, 2, 2, D, None,
                               None, None, -1, 0, 0.1, ws, wsb, 1, None)
    assert bwd(do=None) == 1
    assert bwd(dq=P17) == 3
    assert bwd(D=80) == 2
    assert bwd(wsb=need - 1) == 4
    assert bwd(T=0, do=None) == 0


def test_workspace_bytes(L):
    assert L.fa_varlen_workspace_bytes(0, 8, 2, 2, 64, 0, 0) == 0
    assert L.fa_varlen_workspace_bytes(1, 8, 3, 2, 64, 0, 0) == 0
    # forward: 1000 / 256 + 4 items of 32 bytes, 3 maps of 128 bytes per sequence, the header
    assert L.fa_varlen_workspace_bytes(4, 1000, 8, 2, 128, 0, 0) == 256 + 256 + 4 * 3 * 128
    # backward: fp32 [Hq, T, D] accumulators, one, or four in the deterministic mode
    one = L.fa_varlen_workspace_bytes(4, 1000, 8, 2, 128, 1, 0)
    det = L.fa_varlen_workspace_bytes(4, 1000, 8, 2, 128, 1, 1)
    acc = 8 * 1000 * 128 * 4
    # ... and, few units of grouped heads, a part of dK and of dV per query head
    assert 3 * acc < one < 3.1 * acc and 6 * acc < det < 6.1 * acc
    same = L.fa_varlen_workspace_bytes(4, 1000, 8, 8, 128, 1, 0)
    assert acc < same < 1.1 * acc
    many = L.fa_varlen_workspace_bytes(4, 100000, 8, 4, 128, 1, 0)
    assert 100 * acc < many < 110 * acc


def test_binding_refusals():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(TypeError):
        fa.fwd_varlen(x, x, x, cu)
    with pytest.raises(ValueError):
        fa._var_window(True, (-1, 0))
    with pytest.raises(TypeError):
        fa.fwd_varlen(4, x, x, cu)


def test_reference_gradient():
    """The reference's gradient formulas against torch's own differentiation and
    against central differences of its forward."""
    gen = torch.Generator().manual_seed(3)
    n, D = 7, 64
    q, k, v, do = (torch.randn(n, D, generator=gen, dtype=torch.float64) for _ in range(4))
    for window in ((-1, 0), (2, 1)):
        mask = mask_of(n, False, window)
        r = one_head(q, k, v, 0.125, mask, do)
        leaves = [x.clone().requires_grad_() for x in (q, k, v)]
        s = (leaves[0] @ leaves[1].T * 0.125).masked_fill(~mask, -math.inf)
        (torch.softmax(s, 1) @ leaves[2]).backward(do)
        for leaf, name in zip(leaves, ("dq", "dk", "dv")):
            assert torch.allclose(leaf.grad, r[name], rtol=1e-12, atol=1e-13)
        d = torch.randn(n, D, generator=gen, dtype=torch.float64)
        h = 1e-5
        loss = [(one_head(q + e * d, k, v, 0.125, mask)["o"] * do).sum() for e in (h, -h)]
        # differences err by h^2 times a third derivative of order 1, and by 2^-53 / h
        assert abs((loss[0] - loss[1]) / (2 * h) - (r["dq"] * d).sum()) < 1e-7


# ------------------------------------------------------------------ on a GPU

@pytest.fixture(scope="module")
def gpu():
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _cu(lens, first=0):
    c = [first]
    for x in lens:
        c.append(c[-1] + x)
    return c


def _inputs(T, Hq, Hkv, D, seed):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(T, h, D, generator=gen).to(torch.bfloat16) for h in (Hq, Hkv, Hkv, Hq)]


LENS = [[1], [0, 1, 2, 0, 3], [64, 65], [128], [127, 129, 0, 128, 1], [300, 1, 257, 255],
        [513, 640, 77]]


@pytest.mark.gpu
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mask", ["causal", "none", "window"])
def test_parity(gpu, lens, D, mask):
    kw = {"causal": dict(causal=True), "none": {}, "window": dict(window=(70, 5))}[mask]
    rkw = {"causal": dict(causal=True), "none": dict(causal=False),
           "window": dict(window=(70, 5))}[mask]
    Hq, Hkv = (4, 2) if len(lens) % 2 else (3, 3)
    cu = _cu(lens)
    T = cu[-1]
    q, k, v, do = _inputs(T, Hq, Hkv, D, 7 + T)
    ref = packed(q, k, v, list(zip(cu, cu[1:])), do=do, **rkw)
    qd, kd, vd, dod = (x.cuda() for x in (q, k, v, do))
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, lse = fa.fwd_varlen(qd, kd, vd, cud, **kw)
    assert fa.fwd_status() == fa.FA_OK
    assert fa.last_launch_count() == 2
    assert_within(o, ref["o"], ref["o_tol"], "o")
    assert_within(lse, ref["lse"], ref["lse_tol"], "lse")
    for det in (False, True):
        grads = fa.bwd_varlen(qd, kd, vd, o, dod, lse, cud, deterministic=det, **kw)
        for g, n in zip(grads, ("dq", "dk", "dv")):
            assert_within(g, ref[n], ref[n + "_tol"], f"{n} det={det}")
        if det:
            again = fa.bwd_varlen(qd, kd, vd, o, dod, lse, cud, deterministic=True, **kw)
            for a, b in zip(grads, again):
                assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_foreign_rows_do_not_reach_a_sequence(gpu, D):
    """NaN and infinities in one sequence, before the first and behind the last row
    change no bit of the other sequences; rows of no sequence are not written."""
    lens, first, tail = [70, 131, 40, 300], 5, 60
    cu = _cu(lens, first)
    T = cu[-1] + tail
    q, k, v, do = (x.cuda() for x in _inputs(T, 4, 2, D, 3))
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")

    def run(dirty):
        t = [x.clone() for x in (q, k, v, do)]
        if dirty:
            for x in t:
                x[:first] = float("inf")
                x[cu[1]:cu[2]] = float("nan")
                x[cu[-1]:] = float("nan")
        out = [torch.full_like(x, 7.0) for x in (t[0], t[0], t[1], t[2])]
        lse = torch.full((4, T), 7.0, device="cuda")
        fa.fwd_varlen(t[0], t[1], t[2], cud, causal=True, out=out[0], lse=lse)
        fa.bwd_varlen(t[0], t[1], t[2], out[0], t[3], lse, cud, causal=True, deterministic=True,
                      dq=out[1], dk=out[2], dv=out[3])
        return out, lse

    clean, lse0 = run(False)
    dirty, lse1 = run(True)
    live = torch.ones(T, dtype=torch.bool, device="cuda")
    live[cu[1]:cu[2]] = False
    for a, b in zip(clean, dirty):
        assert torch.equal(a[live], b[live])
        assert bool((b[:first] == 7).all()) and bool((b[cu[-1]:] == 7).all())
    assert torch.equal(lse0[:, live], lse1[:, live])
    assert bool((lse1[:, :first] == 7).all()) and bool((lse1[:, cu[-1]:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_strided_inputs(gpu, D):
    """q, k, v as slices of one fused projection, and with heads outermost, give the
    bits of contiguous inputs."""
    T, Hq, Hkv = 333, 4, 2
    cud = torch.tensor([0, 130, 333], dtype=torch.int32, device="cuda")
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=torch.Generator().manual_seed(1)).to(
        torch.bfloat16).cuda()
    sl = [qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]]
    do = torch.randn(T, Hq, D, device="cuda").to(torch.bfloat16)

    def run(q, k, v):
        o, lse = fa.fwd_varlen(q, k, v, cud, causal=True)
        return (o, lse, *fa.bwd_varlen(q, k, v, o, do, lse, cud, causal=True, deterministic=True))

    base = run(*(x.contiguous() for x in sl))
    outer = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in sl]
    for got in (run(*sl), run(*outer)):
        for a, b in zip(base, got):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_equals_the_dense_call(gpu):
    """Sequences of one length: the packed call against the dense one."""
    B, S, H, D = 3, 300, 2, 128
    q, k, v, do = (x.cuda() for x in _inputs(B * S, H, H, D, 9))
    cud = torch.arange(B + 1, dtype=torch.int32, device="cuda") * S
    o, lse = fa.fwd_varlen(q, k, v, cud, causal=True)
    dense = [x.view(B, S, H, D).transpose(1, 2).contiguous() for x in (q, k, v)]
    o2, lse2 = fa.fwd(*dense, causal=True)
    assert torch.equal(o.view(B, S, H, D).transpose(1, 2), o2)
    assert torch.equal(lse.view(H, B, S).transpose(0, 1), lse2)


@pytest.mark.gpu
def test_autograd(gpu):
    lens = [90, 0, 211]
    cu = _cu(lens)
    T = cu[-1] + 9
    q, k, v, do = _inputs(T, 4, 2, 64, 21)
    ref = packed(q, k, v, list(zip(cu, cu[1:])), do=do)
    leaves = [x.cuda().requires_grad_() for x in (q, k, v)]
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o = fa.attention_varlen(*leaves, cud, causal=True, deterministic=True)
    o.backward(do.cuda())
    assert_within(o, ref["o"], ref["o_tol"], "o")
    for x, n in zip(leaves, ("dq", "dk", "dv")):
        assert_within(x.grad, ref[n], ref[n + "_tol"], n)
        assert bool((x.grad[cu[-1]:] == 0).all())


@pytest.mark.gpu
def test_captured_training_step(gpu):
    """Forward and backward captured into one graph, replayed on new values and
    boundaries.  (No eager graph of the leaves lives at the capture.)"""
    cu = [0, 70, 70, 300]
    q, k, v, do = (x.cuda() for x in _inputs(cu[-1], 4, 2, 64, 31))
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]

    def step(leaves):
        o = fa.attention_varlen(*leaves, cud, causal=True, deterministic=True)
        grads = torch.autograd.grad(o, leaves, do)
        return [o.detach(), *grads]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(leaves)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(leaves)
    for shift, cut in ((1, [0, 70, 70, 300]), (7, [0, 256, 257, 299])):
        with torch.no_grad():
            for x, y in zip(leaves, (q, k, v)):
                x.copy_(y.roll(shift, 0))
        cud.copy_(torch.tensor(cut, dtype=torch.int32))
        g.replay()
        want = step([x.detach().clone().requires_grad_() for x in leaves])
        for a, b in zip(out, want):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_binding_refusals_of_device_tensors(gpu):
    q, k, v, do = (x.cuda() for x in _inputs(6, 4, 2, 64, 3))
    cu = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    o, lse = fa.fwd_varlen(q, k, v, cu)

    def refuses(error, fn, *a, **kw):
        with pytest.raises(error):
            fn(*a, **kw)

    refuses(TypeError, fa.fwd_varlen, q.half(), k, v, cu)
    refuses(TypeError, fa.fwd_varlen, q, k.cpu(), v, cu)
    refuses(ValueError, fa.fwd_varlen, q[None], k, v, cu)
    refuses(ValueError, fa.fwd_varlen, q, k[:5], v[:5], cu)
    refuses(ValueError, fa.fwd_varlen, q, k, v[:, :1], cu)
    refuses(TypeError, fa.fwd_varlen, q, k, v, cu.long())
    refuses(TypeError, fa.fwd_varlen, q, k, v, cu.cpu())
    refuses(fa.FAError, fa.fwd_varlen, q, k, v, cu[:1])  # no sequence
    refuses(fa.FAError, fa.fwd_varlen, q[:, :3], k, v, cu)
    refuses(fa.FAError, fa.fwd_varlen, q[:, :1].expand(6, 4, 64), k, v, cu)  # heads 0 apart
    refuses(ValueError, fa.fwd_varlen, q, k, v, cu, out=torch.empty_like(q)[:5])
    refuses(ValueError, fa.fwd_varlen, q, k, v, cu, lse=lse.T.contiguous())
    refuses(ValueError, fa.fwd_varlen, q, k, v, cu, causal=True, window=(-1, 0))
    refuses(ValueError, fa.bwd_varlen, q, k, v, o[:5], do, lse, cu)
    refuses(ValueError, fa.bwd_varlen, q, k, v, o, do.float(), lse, cu)
    refuses(ValueError, fa.bwd_varlen, q, k, v, o, do, lse, cu, dk=torch.empty_like(q))
    refuses(fa.FAError, fa.bwd_varlen, q, k, v, o, do, lse, cu,
            workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert fa.fwd_status() == fa.FA_OK


@pytest.mark.gpu
def test_bad_boundaries_are_reported(gpu):
    """Boundaries out of order or range: no output, and a status."""
    T, H, D = 200, 2, 64
    q, k, v, do = (x.cuda() for x in _inputs(T, H, H, D, 2))
    good = torch.tensor([0, 60, 200], dtype=torch.int32, device="cuda")
    o, lse = fa.fwd_varlen(q, k, v, good)
    for bad in ([0, 150, 100], [0, 50, 201], [-4, 50, 200]):
        cud = torch.tensor(bad, dtype=torch.int32, device="cuda")
        out = torch.full_like(q, 3.0)
        fa.fwd_varlen(q, k, v, cud, out=out)
        assert fa.fwd_status() == 1
        assert bool((out == 3).all())
        ws = torch.empty(fa.varlen_workspace_bytes(2, T, H, H, D, True), dtype=torch.uint8,
                         device="cuda")
        dq = torch.full_like(q, 3.0)
        fa.bwd_varlen(q, k, v, o, do, lse, cud, dq=dq, workspace=ws)
        assert fa.bwd_status(ws) == 1
        assert bool((dq == 3).all())
    assert fa.fwd_status() == fa.FA_OK


@pytest.mark.gpu
def test_captured_and_on_another_stream(gpu):
    """Two captured graphs with workspaces of their own replay on new inputs and new
    boundaries; a call on another stream gives the same bits."""
    T, H, D, B = 400, 2, 128, 3
    q, k, v, do = (x.cuda() for x in _inputs(T, H, H, D, 4))
    cuts = [[0, 100, 100, 400], [0, 1, 258, 390], [0, 399, 400, 400]]
    cud = torch.tensor(cuts[0], dtype=torch.int32, device="cuda")

    def both(ws_f, ws_b, out):
        fa.fwd_varlen(q, k, v, cud, causal=True, out=out[0], lse=out[1], workspace=ws_f)
        fa.bwd_varlen(q, k, v, out[0], do, out[1], cud, causal=True, deterministic=True,
                      workspace=ws_b, dq=out[2], dk=out[3], dv=out[4])

    def buffers():
        return ([torch.empty(fa.varlen_workspace_bytes(B, T, H, H, D, b, b), dtype=torch.uint8,
                             device="cuda") for b in (False, True)],
                [torch.zeros_like(q), torch.zeros(H, T, device="cuda"),
                 *(torch.zeros_like(x) for x in (q, k, v))])

    sets = [buffers() for _ in range(2)]
    both(*sets[0][0], sets[0][1])
    torch.cuda.synchronize()
    graphs = []
    for ws, out in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            both(*ws, out)
        graphs.append(g)
    side = torch.cuda.Stream()
    for i, cut in enumerate(cuts):
        q.copy_(torch.randn_like(q.float()).to(q.dtype))
        cud.copy_(torch.tensor(cut, dtype=torch.int32))
        want = buffers()
        both(*want[0], want[1])
        for g in graphs:
            g.replay()
        other = buffers()[1]
        side.wait_stream(torch.cuda.current_stream())
        fa.fwd_varlen(q, k, v, cud, causal=True, out=other[0], lse=other[1], stream=side)
        fa.bwd_varlen(q, k, v, other[0], do, other[1], cud, causal=True, deterministic=True,
                      dq=other[2], dk=other[3], dv=other[4], stream=side)
        torch.cuda.synchronize()
        for out in (sets[0][1], sets[1][1], other):
            for a, b in zip(out, want[1]):
                assert torch.equal(a[:, :cut[-1]] if a.dim() == 2 else a[:cut[-1]],
                                   b[:, :cut[-1]] if b.dim() == 2 else b[:cut[-1]]), i


@pytest.mark.gpu
@pytest.mark.parametrize("count", [400, 4500])
def test_many_sequences_and_grouped_heads(gpu, count):
    """More sequences than SMs, or than the plan keeps lengths of, one kv head for
    eight query heads, sampled."""
    gen = torch.Generator().manual_seed(8)
    lens = torch.randint(0, 40 if count < 1000 else 5, (count,), generator=gen).tolist() + [1500]
    cu = _cu(lens)
    q, k, v, do = _inputs(cu[-1], 8, 1, 128, 12)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    qd, kd, vd, dod = (x.cuda() for x in (q, k, v, do))
    o, lse = fa.fwd_varlen(qd, kd, vd, cud, causal=True)
    grads = fa.bwd_varlen(qd, kd, vd, o, dod, lse, cud, causal=True)
    assert fa.fwd_status() == fa.FA_OK
    picked = [(cu[i], cu[i + 1]) for i in (0, 7, 100, 399)]
    ref = packed(q, k, v, picked, do=do)
    for got, n in zip((o, lse, *grads), ("o", "lse", "dq", "dk", "dv")):
        assert_within(got, ref[n], ref[n + "_tol"], n)
    # every row's weights sum to one: with v = 1, o is 1 up to the rounding of the
    # weights (2^-8) and of o (2^-8)
    o1, _ = fa.fwd_varlen(qd, kd, torch.ones_like(vd), cud, causal=True)
    assert float((o1.float() - 1).abs().max()) <= 2.0 ** -7
