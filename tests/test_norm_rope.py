"""Norms of queries and keys with the rotation by position (fa_norm_rope_fwd / _bwd,
fa_rope_table) against the plain 64-bit form.

Bounds (u = 2^-8, half a bf16 step; every fp32 operation errs by 2^-24 of its result):
  y   u |y| + 2^-20 (|n_a| + |n_b|): r is off by some 8 half steps (a sum of D squares in
      chains of 8 and a tree, the root), then four products and a sum, and the tables' own
      2^-25 of at most 1
  dx  u |dx| + 2^-18 r ((|dy_a| + |dy_b|) |w| + |xh| mean |h xh|): the same, and the mean of
      D products in chains of 16 and a tree
  dw  (64 + chain) 2^-24 sum |g xh|, chain: the rows that one lane adds up; the tree over
      lanes, warps and blocks has fewer than 64 steps
"""
import ctypes
import math

import pytest
import torch

import __graft_entry__
import exact_attention_blackwell_tiled_gb300 as fa
from packed_reference import assert_within

U = 2.0 ** -8
P = ctypes.c_void_p(256 * 1024)
P8 = ctypes.c_void_p(256 * 1024 + 8)
P2 = ctypes.c_void_p(256 * 1024 + 2)


def pairs_of(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def angles(positions, rot, base=10000.0):
    rate = base ** (-2 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    return positions.double()[:, None] * rate


def rotate(x, ang, rot, interleaved, sign=1):
    a, b = pairs_of(rot, interleaved)
    c, s = ang.cos()[:, None], sign * ang.sin()[:, None]
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def partner_sum(x, rot, interleaved):
    """|x_a| + |x_b| for both of each pair."""
    a, b = pairs_of(rot, interleaved)
    y = x.abs()
    y[..., a] = y[..., b] = x[..., a].abs() + x[..., b].abs()
    return y


def plain(x, w, positions, rot, interleaved, eps=1e-6, dy=None, chain=8):
    """fp64 y (dx, dw) of bf16 x [T, H, D] with bounds; rows of no sequence are NaN."""
    D = x.shape[-1]
    live = positions >= 0
    x, w = x.double(), w.double()
    ang = angles(positions.clamp(min=0), rot)
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    u = x * r
    n = u * w
    y = rotate(n, ang, rot, interleaved)
    out = {"y": y, "y_tol": U * y.abs() + 2.0 ** -20 * partner_sum(n, rot, interleaved)}
    if dy is not None:
        dy = dy.double()
        g = rotate(dy, ang, rot, interleaved, -1)
        h = g * w
        out["dx"] = r * (h - u * (h * u).mean(-1, keepdim=True))
        out["dx_tol"] = U * out["dx"].abs() + 2.0 ** -18 * r * (
            partner_sum(dy, rot, interleaved) * w.abs() + u.abs() * (h * u).abs().mean(-1, keepdim=True))
        gu = (g * u)[live]
        out["dw"] = gu.sum((0, 1))
        out["dw_tol"] = (64 + chain) * 2.0 ** -24 * gu.abs().sum((0, 1)) + 1e-30
    for name in ("y", "dx"):
        if name in out:
            out[name][~live] = math.nan
            out[name + "_tol"][~live] = math.nan
    return out


# ------------------------------------------------------------------ without a GPU

@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return fa.lib()


def test_refusals(L):
    def fwd(q=P, out=P, w=P, cos=P, pos=P, T=4, Hq=2, Hkv=1, D=64, rows=8, rot=64, eps=1e-6, s=None):
        st = None if s is None else ctypes.byref(fa.PackedStride(*s))
        return L.fa_norm_rope_fwd(q, P, out, P, w, P, 0, cos, P, pos, T, Hq, Hkv, D, rows, rot, 0, eps,
                                  st, None, st, None, 0, None)
    assert fwd(q=None) == 1 and fwd(out=None) == 1 and fwd(w=None) == 1
    assert fwd(cos=None) == 1 and fwd(pos=None) == 1
    assert fwd(T=-1) == 1 and fwd(Hq=0) == 1 and fwd(Hkv=0) == 1 and fwd(rows=0) == 1
    assert fwd(D=96) == 2
    for rot in (0, 8, 24, 80, 128):
        assert fwd(rot=rot) == 1
    assert fwd(eps=-1e-6) == 1 and fwd(eps=math.nan) == 1
    assert fwd(q=P8) == 3 and fwd(cos=P8) == 3 and fwd(pos=P2) == 3
    assert fwd(s=(132, 64)) == 3
    assert fwd(s=(-128, 64)) == 1
    assert fwd(s=(128, 56)) == 1            # the results' heads would overlap
    assert fwd(T=0, q=None, pos=None) == 0
    assert fwd(T=(1 << 30) + 1) == 1 and fwd(Hq=(1 << 20) + 1) == 1

    def bwd(dw=P, dy=P, ws=P, T=4):
        return L.fa_norm_rope_bwd(P, P, dy, P, P, P, dw, P, P, P, 0, P, P, P, T, 2, 1, 64, 8, 64, 0,
                                  1e-6, None, None, None, None, None, None, 0, ws, 1 << 20, None)
    assert bwd(dw=None) == 1 and bwd(dy=None) == 1
    assert bwd(ws=None) == 4 and bwd(ws=P8) == 4
    assert bwd(dw=P2) == 3

    def table(c=P, n=4, rot=32, base=1e4):
        return L.fa_rope_table(c, P, n, rot, base, None)
    assert table(c=None) == 1 and table(n=0) == 1 and table(rot=20) == 1 and table(rot=144) == 1
    assert table(base=0.0) == 1 and table(base=math.inf) == 1 and table(c=P8) == 3
    assert L.fa_norm_rope_workspace_bytes(4, 2, 1, 80) == 0


def test_binding_refusals():
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fa.norm_rope_fwd(x, x, None, None, None, None, None)


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_gradients_by_differences(interleaved):
    gen = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(3, 2, 64, generator=gen, dtype=torch.float64) for _ in range(2))
    w = torch.randn(64, generator=gen, dtype=torch.float64)
    pos = torch.tensor([0, 5, 77])
    r = plain(x, w, pos, 32, interleaved, dy=dy)

    def loss(x, w):
        return float((plain(x, w, pos, 32, interleaved)["y"] * dy).sum())
    eps = 1e-6
    for at in ((0, 0, 0), (1, 1, 17), (2, 0, 40)):
        d = torch.zeros_like(x)
        d[at] = eps
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * eps) - float(r["dx"][at])) < 1e-6
    for at in (0, 20, 63):
        d = torch.zeros_like(w)
        d[at] = eps
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * eps) - float(r["dw"][at])) < 1e-6


# ------------------------------------------------------------------ on the GPU

@pytest.fixture(scope="module")
def gpu():
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _rows(T, H, D, gen, spread=1.0):
    scale = torch.rand(H, D, generator=gen) * 2 + 0.1
    return (torch.randn(T, H, D, generator=gen) * scale * spread).to(torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("rot,base", [(16, 10000.0), (64, 500000.0), (128, 10000.0)])
def test_table(gpu, rot, base):
    n = 131072
    cos, sin = fa.rope_table(n, rot, base)
    ang = angles(torch.arange(n), rot, base).cuda()
    # half a step of fp32 below 1, and fp64's own error of the angle
    tol = 2.0 ** -25 + n * 2.0 ** -50
    assert float((cos.double() - ang.cos()).abs().max()) <= tol
    assert float((sin.double() - ang.sin()).abs().max()) <= tol


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", [(1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (5, 8, 1, 128, 64),
                                            (67, 14, 2, 64, 32), (130, 9, 3, 128, 16),
                                            (257, 4, 4, 64, 48), (64, 32, 8, 128, 112),
                                            (2000, 16, 16, 128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("wtype", [torch.bfloat16, torch.float32])
def test_forward_and_backward(gpu, T, Hq, Hkv, D, rot, interleaved, wtype):
    gen = torch.Generator().manual_seed(T + D)
    fused = torch.cat([_rows(T, h, D, gen) for h in (Hq, Hkv, Hkv)], 1)
    w = (1 + 0.3 * torch.randn(2, D, generator=gen)).to(wtype)
    pos = torch.randint(0, 4000, (T,), generator=gen)
    pos[::7] = 0
    dy = [_rows(T, h, D, gen) for h in (Hq, Hkv)]
    cos, sin = fa.rope_table(4000, rot)
    d = fused.cuda()
    x = (d[:, :Hq], d[:, Hq:Hq + Hkv])
    wd = w.cuda()
    args = (*x, wd[0], wd[1], cos, sin, pos.int().cuda())
    y = fa.norm_rope_fwd(*args, interleaved=interleaved)
    g = fa.norm_rope_bwd(*args, *(t.cuda() for t in dy), interleaved=interleaved)
    assert fa.fwd_status() == fa.FA_OK
    again = fa.norm_rope_bwd(*args, *(t.cuda() for t in dy), interleaved=interleaved)
    assert all(torch.equal(a, b) for a, b in zip(g, again))
    for i in range(2):
        r = plain(x[i].cpu(), w[i], pos, rot, interleaved, dy=dy[i])
        assert_within(y[i], r["y"], r["y_tol"], f"y {i}")
        assert_within(g[i], r["dx"], r["dx_tol"], f"dx {i}")
        assert_within(g[2 + i], r["dw"], r["dw_tol"], f"dw {i}")


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [1e-18, 1e-3, 1e15])
def test_magnitudes(gpu, spread):
    """Rows near the ends of the range (their squares stay in fp32's), and rows of zeros."""
    T, D, rot = 33, 128, 128
    gen = torch.Generator().manual_seed(4)
    q, k = _rows(T, 2, D, gen, spread), _rows(T, 1, D, gen, spread)
    q[3] = 0
    w = torch.ones(D)
    pos = torch.arange(T)
    dy = [_rows(T, h, D, gen) for h in (2, 1)]
    cos, sin = fa.rope_table(T, rot)
    args = (q.cuda(), k.cuda(), w.cuda(), w.cuda(), cos, sin, pos.int().cuda())
    y = fa.norm_rope_fwd(*args)
    g = fa.norm_rope_bwd(*args, *(t.cuda() for t in dy))
    for i, x in enumerate((q, k)):
        r = plain(x, w, pos, rot, False, dy=dy[i])
        assert_within(y[i], r["y"], r["y_tol"], "y")
        assert_within(g[i], r["dx"], r["dx_tol"] + 2.0 ** -133, "dx")  # (below bf16's normal range)
        assert_within(g[2 + i], r["dw"], r["dw_tol"], "dw")


@pytest.mark.gpu
def test_tokens_of_no_sequence(gpu):
    """Negative positions: rows left as they were, or zeros; NaN in them reaches nothing.  A
    position past the tables counts as one and is reported."""
    T, D, rot = 20, 64, 64
    gen = torch.Generator().manual_seed(6)
    q, k = _rows(T, 9, D, gen), _rows(T, 2, D, gen)
    pos = torch.arange(T)
    pos[[0, 7, 19]] = -1
    pos[8] = -2 ** 31
    dead = pos < 0
    q[dead], k[dead] = math.nan, math.inf
    dy = [_rows(T, h, D, gen) for h in (9, 2)]
    for t in dy:
        t[dead] = math.nan
    w = (1 + torch.rand(D, generator=gen)).cuda()
    cos, sin = fa.rope_table(T, rot)
    args = (q.cuda(), k.cuda(), w, w, cos, sin, pos.int().cuda())
    for zero in (False, True):
        y = [torch.full((T, h, D), 7.0, dtype=torch.bfloat16, device="cuda") for h in (9, 2)]
        g = [torch.full((T, h, D), 7.0, dtype=torch.bfloat16, device="cuda") for h in (9, 2)]
        fa.norm_rope_fwd(*args, q_out=y[0], k_out=y[1], zero_skipped=zero)
        _, _, *dw = fa.norm_rope_bwd(*args, *(t.cuda() for t in dy), dq=g[0], dk=g[1], zero_skipped=zero)
        for i, x in enumerate((q, k)):
            r = plain(x, w.cpu(), pos, rot, False, dy=dy[i])
            assert_within(y[i], r["y"], r["y_tol"], "y")
            assert_within(g[i], r["dx"], r["dx_tol"], "dx")
            assert_within(dw[i], r["dw"], r["dw_tol"], "dw")
            for t in (y[i], g[i]):
                assert bool((t[dead.cuda()] == (0 if zero else 7)).all())
    assert fa.fwd_status() == fa.FA_OK
    late = pos.clone()
    late[3] = T
    y = torch.full((T, 9, D), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.norm_rope_fwd(*args[:6], late.int().cuda(), q_out=y)
    assert bool((y[3] == 7).all())
    assert fa.fwd_status() == 1 and fa.fwd_status() == fa.FA_OK


@pytest.mark.gpu
def test_in_place_and_slices(gpu):
    """The results over the inputs; the gradients into slices of one, or over dy."""
    T, Hq, Hkv, D, rot = 50, 5, 2, 128, 96
    gen = torch.Generator().manual_seed(8)
    fused = torch.cat([_rows(T, h, D, gen) for h in (Hq, Hkv, Hkv)], 1).cuda()
    w = torch.rand(2, D, generator=gen).cuda()
    pos = torch.randint(0, 99, (T,), generator=gen).int().cuda()
    cos, sin = fa.rope_table(99, rot)
    dy = [_rows(T, h, D, gen).cuda() for h in (Hq, Hkv)]
    parts = (fused[:, :Hq], fused[:, Hq:Hq + Hkv])
    y = fa.norm_rope_fwd(*parts, w[0], w[1], cos, sin, pos)
    g = fa.norm_rope_bwd(*parts, w[0], w[1], cos, sin, pos, *dy)
    grad = torch.full_like(fused, 7.0)
    g2 = fa.norm_rope_bwd(*parts, w[0], w[1], cos, sin, pos, *dy, dq=grad[:, :Hq],
                          dk=grad[:, Hq:Hq + Hkv])
    assert all(torch.equal(a, b) for a, b in zip(g, g2))
    assert bool((grad[:, Hq + Hkv:] == 7).all())
    over = [t.clone() for t in dy]
    g3 = fa.norm_rope_bwd(*parts, w[0], w[1], cos, sin, pos, *over, dq=over[0], dk=over[1])
    assert all(torch.equal(a, b) for a, b in zip(g, g3))
    rest = fused[:, Hq + Hkv:].clone()
    z = fa.norm_rope_fwd(*parts, w[0], w[1], cos, sin, pos, q_out=parts[0], k_out=parts[1])
    assert z[0].data_ptr() == fused.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip(y, z))
    assert torch.equal(fused[:, Hq + Hkv:], rest)


@pytest.mark.gpu
def test_heads_of_one_row(gpu):
    """A broadcast input: every token reads one row."""
    D = 64
    row = torch.randn(1, 2, D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    x = row.expand(9, 2, D)
    w = torch.ones(D, device="cuda")
    cos, sin = fa.rope_table(9, D)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    a = fa.norm_rope_fwd(x, x, w, w, cos, sin, pos)
    b = fa.norm_rope_fwd(x.contiguous(), x.contiguous(), w, w, cos, sin, pos)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_autograd(gpu):
    T, Hq, Hkv, D = 40, 4, 2, 64
    gen = torch.Generator().manual_seed(3)
    q, k = (_rows(T, h, D, gen).cuda().requires_grad_() for h in (Hq, Hkv))
    w = [(1 + torch.rand(D, generator=gen)).to(torch.bfloat16).cuda().requires_grad_() for _ in range(2)]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    pos[5] = -1
    cos, sin = fa.rope_table(T, D)
    dy = [_rows(T, h, D, gen).cuda() for h in (Hq, Hkv)]
    y = fa.norm_rope(q, k, *w, cos, sin, pos)
    torch.autograd.backward(y, dy)
    det = [t.detach() for t in (q, k, *w)]
    g = fa.norm_rope_bwd(*det, cos, sin, pos, *dy, zero_skipped=True)
    for a, b in zip((q, k, *w), g):
        assert torch.equal(a.grad, b.to(a.dtype))
    assert bool((y[0][5] == 0).all()) and bool((q.grad[5] == 0).all())
    z = fa.norm_rope(q, k, *w, cos, sin, pos)
    first = torch.autograd.grad(z[0].float().sum(), q, create_graph=True)[0]
    with pytest.raises(RuntimeError):
        first.float().sum().backward()


@pytest.mark.gpu
def test_no_tokens(gpu):
    D = 128
    x = torch.zeros(0, 2, D, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(D, device="cuda")
    cos, sin = fa.rope_table(4, D)
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    y = fa.norm_rope_fwd(x, x, w, w, cos, sin, pos)
    assert y[0].shape == x.shape
    g = fa.norm_rope_bwd(x, x, w, w, cos, sin, pos, x, x)
    assert bool((g[2] == 0).all()) and bool((g[3] == 0).all())


@pytest.mark.gpu
def test_capture_and_streams(gpu):
    T, H, D = 300, 8, 128
    gen = torch.Generator().manual_seed(5)
    cos, sin = fa.rope_table(1000, D)
    w = torch.rand(2, D, generator=gen).cuda()
    sets = [([_rows(T, H, D, gen).cuda() for _ in range(4)],
             torch.randint(0, 1000, (T,), generator=gen).int().cuda()) for _ in range(3)]

    def step(x, pos):
        y = fa.norm_rope_fwd(x[0], x[1], w[0], w[1], cos, sin, pos)
        return (*y, *fa.norm_rope_bwd(x[0], x[1], w[0], w[1], cos, sin, pos, x[2], x[3]))
    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[] for _ in sets]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(step(*sets[i]))
    torch.cuda.synchronize()
    for a, runs in zip(want, got):
        assert all(torch.equal(x, y) for b in runs for x, y in zip(a, b))
    x = [t.clone() for t in sets[0][0]]
    pos = sets[0][1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, pos)
    for i, (xs, p) in enumerate(sets):
        for a, b in zip(x, xs):
            a.copy_(b)
        pos.copy_(p)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


@pytest.mark.gpu
def test_offsets_past_32_bits(gpu):
    """Rows 2^26 elements apart: the last ones lie behind 2^32 elements."""
    T, D, step = 70, 64, 1 << 26
    try:
        far = torch.zeros(T * step, dtype=torch.bfloat16, device="cuda")
    except torch.cuda.OutOfMemoryError:
        pytest.skip("not enough memory")
    gen = torch.Generator().manual_seed(1)
    q, k = _rows(T, 2, D, gen).cuda(), _rows(T, 1, D, gen).cuda()
    qf, kf = far.as_strided((T, 2, D), (step, D, 1)), far.as_strided((T, 1, D), (step, D, 1), 4 * D)
    qf.copy_(q)
    kf.copy_(k)
    w = torch.ones(D, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    cos, sin = fa.rope_table(T, D)
    want = fa.norm_rope_fwd(q, k, w, w, cos, sin, pos)
    got = fa.norm_rope_fwd(qf, kf, w, w, cos, sin, pos, q_out=qf, k_out=kf)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    del far, qf, kf, got
    torch.cuda.empty_cache()


def test_table_refuses_host_memory():
    with pytest.raises(TypeError):
        fa.rope_table(4, 64, device="cpu")
