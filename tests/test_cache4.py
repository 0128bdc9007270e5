"""The paged 4-bit cache: append, read, attend and evict against the plain forms."""
import ctypes
import math

import pytest
import torch

import __graft_entry__
import cache4_reference as ref
import exact_attention_blackwell_tiled_gb300 as fa
from packed_reference import assert_within, packed

P = ctypes.c_void_p(256 * 1024)
P4 = ctypes.c_void_p(256 * 1024 + 4)
P2 = ctypes.c_void_p(256 * 1024 + 2)


# ------------------------------------------------------------------ without a GPU

@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return fa.lib()


def test_page_bytes(L):
    # 16 slots: codes D/2 and parameters D/8 bytes, of key and value
    assert L.fa_cache4_page_bytes(1, 128, 16) == 16 * 2 * (64 + 16)
    assert L.fa_cache4_page_bytes(8, 64, 128) == 8 * 128 * 2 * (32 + 8)
    for bad in ((0, 128, 64), (1, 96, 64), (1, 128, 48), (1, 128, 8), (1, 128, 256)):
        assert L.fa_cache4_page_bytes(*bad) == 0


def test_append_refusals(L):
    def call(cache=P, pages=4, page=64, k=P, v=P, ks=None, B=2, T=5, Hkv=2, D=128, cu=P, lens=P,
             table=P, width=2):
        return L.fa_cache4_append(cache, pages, page, k, v,
                                  None if ks is None else ctypes.byref(fa.PackedStride(*ks)), None,
                                  B, T, Hkv, D, cu, lens, table, width, None)
    assert call(cache=None) == 1
    assert call(k=None) == 1
    assert call(pages=0) == 1
    assert call(width=0) == 1
    assert call(T=-1) == 1
    assert call(cu=None) == 1              # one token per sequence needs T == B
    assert call(D=80) == 2
    assert call(page=20) == 2
    assert call(cache=P4) == 3
    assert call(lens=P2) == 3
    assert call(ks=(260, 128)) == 3
    assert call(ks=(-256, 128)) == 1
    assert call(width=1 << 25) == 1        # slots pass 2^30
    assert call(T=0, cache=None) == 0


def test_read_refusals(L):
    def call(k=P, S=4, first=None, count=P, D=64, page=16):
        return L.fa_cache4_read(P, 4, page, k, P, 2, 2, S, D, first, count, P, 2, None)
    assert call(k=None) == 1
    assert call(S=-1) == 1
    assert call(count=None) == 1
    assert call(D=32) == 2
    assert call(k=P4) == 3
    assert call(first=P2) == 3
    assert call(S=0, k=None) == 0


def test_attend_refusals(L):
    def call(q=P, qb=512, qh=128, o=P, B=2, Hq=4, Hkv=2, D=128, page=64, lens=P, scale=0.1,
             w_in=None, w_out=None, slots=0, ws=P, wsb=1 << 40):
        return L.fa_cache4_attend(q, qb, qh, P, 4, page, o, P, B, Hq, Hkv, D, lens, P,
                                  2 if B < 9 else 1 << 20, scale, w_in, w_out, slots, ws, wsb, None)
    assert call(q=None) == 1
    assert call(o=None) == 1
    assert call(Hq=3) == 1
    assert call(scale=math.nan) == 1
    assert call(qb=-8) == 1
    assert call(w_out=P, slots=0) == 1
    assert call(w_in=P) == 1               # weights to add to, but nowhere to put them
    assert call(D=256) == 2
    assert call(Hq=258, Hkv=2) == 2        # 129 query heads per kv head
    assert call(qh=100) == 3
    assert call(q=P4) == 3
    assert call(w_out=P2, slots=4) == 3
    assert call(ws=None) == 4
    assert call(ws=P4) == 4
    assert call(B=1 << 20, Hq=1 << 10, Hkv=1 << 10, page=128) == 1  # a list past 2^40 blocks


def test_evict_refusals(L):
    def call(w=P, cap=64, budget=8, recent=2, ow=1, page=16, src=P, D=64):
        return L.fa_cache4_evict(P, 4, page, w, cap, P, P, 4, 2, 2, D, budget, recent, P, ow, src,
                                 P, P, None)
    assert call(w=None) == 1
    assert call(budget=0) == 1
    assert call(recent=9) == 1
    assert call(recent=-1) == 1
    assert call(budget=17) == 1            # more than the new pages hold
    assert call(cap=0) == 1
    assert call(D=100) == 2
    assert call(src=P2) == 3


def test_binding_refusals():
    c = torch.zeros(2, 1, 16 * 80, dtype=torch.uint8)
    with pytest.raises(TypeError):
        fa.cache4_read(c, None, None, None, 1, 64)                  # host memory
    with pytest.raises(TypeError):
        fa.cache4_append(c, torch.zeros(1, 1, 64, dtype=torch.bfloat16), None, None, None)


def test_reference_quantiser_is_the_formula():
    """fp32 steps against the same steps in 64 bits, on random vectors, ties and groups
    of one value."""
    gen = torch.Generator().manual_seed(0)
    x = (torch.randn(64, 128, generator=gen) * torch.rand(64, 1, generator=gen) * 9).to(torch.bfloat16)
    x[0] = 1.5
    x[1, :32] = torch.arange(32).bfloat16() / 2  # steps of a half: ties
    z, mn, c = ref.quantise(x)
    g = x.double().unflatten(-1, (-1, 32))
    c64 = ((g.amax(-1) - g.amin(-1)) / 15).float().bfloat16().double()
    assert torch.equal(c.double(), c64)
    z64 = ((g - g.amin(-1, keepdim=True)) / c64.clamp_min(1e-300)[..., None]).round().clamp(0, 15)
    z64[c64 == 0] = 0
    assert torch.equal(z.double(), z64)
    err = (ref.stored(x)[0] - x.double()).abs().unflatten(-1, (-1, 32)).amax(-1)
    assert bool((err <= c64 * (0.5 + 15 * U_SCALE)).all())


U_SCALE = 2.0 ** -8  # the scale's own rounding, relative: moves code 15 by 15 of it


# ------------------------------------------------------------------ on a GPU

@pytest.fixture(scope="module")
def gpu():
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _cu(lens):
    c = [0]
    for x in lens:
        c.append(c[-1] + x)
    return c


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _table(lens, page, seed=0, spare=1, first=0):
    width = max(1, max(-(-x // page) for x in lens)) + spare
    n = width * len(lens)
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(seed)) + first
    return perm.to(torch.int32).view(len(lens), width).cuda(), n


def _kv(T, Hkv, D, seed):
    gen = torch.Generator().manual_seed(seed)
    off = torch.randn(Hkv, D, generator=gen) * 2
    return ((torch.randn(T, Hkv, D, generator=gen) + off).to(torch.bfloat16),
            torch.randn(T, Hkv, D, generator=gen).to(torch.bfloat16))


def _filled(lens, Hkv, D, page, seed=5, fill=0):
    """A cache with lens tokens appended: (cache, table, lens, cu, k, v)."""
    cu = _cu(lens)
    k, v = _kv(cu[-1], Hkv, D, seed)
    table, n = _table(lens, page, seed)
    cache = fa.cache4_empty(n, Hkv, D, page)
    cache.fill_(fill)
    if cu[-1]:
        fa.cache4_append(cache, k.cuda(), v.cuda(), table, _i32([0] * len(lens)), _i32(cu))
    return cache, table, _i32(lens), cu, k, v


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_and_read(gpu, D, page):
    """Ragged prompts, then a token each, read back whole and in part: the formula's
    values to the bit."""
    Hkv, lens = 3, [1, 0, 37, 130, 16]
    cu = _cu(lens)
    k, v = _kv(cu[-1] + 5, Hkv, D, page)
    k[2], v[3] = 1.5, 0.0                              # groups of one value
    k[5:20] = (torch.arange(15 * Hkv * D).view(15, Hkv, D) * 7 % 31).bfloat16() / 4  # ties
    v[5:20] = (torch.arange(15 * Hkv * D).view(15, Hkv, D) * 11 % 48).bfloat16()
    k[4] = torch.linspace(-1e30, 1e30, D).bfloat16()   # wide and tiny ranges
    v[4] = (torch.linspace(0, 1, D) * 1e-38).bfloat16()
    table, n = _table([x + 1 for x in lens], page)
    cache = fa.cache4_empty(n, Hkv, D, page)
    qkv = torch.cat((k, v), 1).cuda()                  # slices of one fused projection
    kd, vd = qkv[:, :Hkv], qkv[:, Hkv:]
    zero = _i32([0] * 5)
    fa.cache4_append(cache, kd[:cu[-1]], vd[:cu[-1]], table, zero, _i32(cu))
    fa.cache4_append(cache, kd[cu[-1]:], vd[cu[-1]:], table, _i32(lens))
    assert fa.cache4_status() == fa.FA_OK
    S = max(lens) + 3
    got = fa.cache4_read(cache, table, None, _i32([x + 1 for x in lens]), S, D)
    for x, y in ((k, got[0]), (v, got[1])):
        z, mn, c = ref.quantise(x)
        val = (mn[..., None] + c[..., None] * z).flatten(-2).to(torch.bfloat16)
        want = torch.zeros(5, Hkv, S, D, dtype=torch.bfloat16)
        for b, m in enumerate(lens):
            want[b, :, :m] = val[cu[b]:cu[b + 1]].transpose(0, 1)
            want[b, :, m] = val[cu[-1] + b]
        assert torch.equal(y.cpu(), want)
    first, count = [0, 1, 20, 100, 16], [1, 0, 9, 31, 1]
    part = fa.cache4_read(cache, table, _i32(first), _i32(count), 40, D)
    for y, whole in zip(part, got):
        for b in range(5):
            n_ = count[b]
            assert torch.equal(y[b, :, :n_], whole[b, :, first[b]:first[b] + n_])
            assert bool((y[b, :, n_:] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,page,Hkv,group", [
    ([1], 16, 1, 1), ([0, 5, 16, 17], 16, 2, 4), ([300, 31], 32, 2, 5), ([1000, 0, 64], 64, 3, 8),
    ([2049, 777], 128, 1, 12), ([129] * 40, 16, 4, 2), ([4000], 64, 1, 40), ([900, 0, 33], 16, 2, 16),
    ([250] * 100, 32, 4, 1)])
def test_attend(gpu, D, lens, page, Hkv, group):
    cache, table, n, cu, k, v = _filled(lens, Hkv, D, page, fill=255)
    q = torch.randn(len(lens), Hkv * group, D, generator=torch.Generator().manual_seed(1)).to(
        torch.bfloat16)
    slots = max(lens) + 2
    w0 = torch.rand(len(lens), Hkv, slots, generator=torch.Generator().manual_seed(2))
    wd = w0.cuda()
    o, lse = fa.cache4_attend(q.cuda(), cache, table, n)
    assert fa.last_launch_count() in (1, 2)
    o2, lse2 = fa.cache4_attend(q.cuda(), cache, table, n, weights=wd)
    assert fa.cache4_status() == fa.FA_OK
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    step = torch.full_like(wd, 7.0)
    fa.cache4_attend(q.cuda(), cache, table, n, weights_out=step)
    for b, m in enumerate(lens):
        r = ref.attend(q[b], k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]])
        if m == 0:
            assert bool((o[b] == 0).all()) and bool((lse[b] == -math.inf).all())
        else:
            assert_within(o[b], r["o"], r["o_tol"], f"o of {b}")
            assert_within(lse[b], r["lse"], r["lse_tol"], f"lse of {b}")
            want = w0[b, :, :m].double() + r["p"]
            assert_within(wd[b, :, :m], want, r["p_tol"] + 2.0 ** -23 * want, f"weights of {b}")
            assert_within(step[b, :, :m], r["p"], r["p_tol"] + 2.0 ** -23 * r["p"], "step")
        assert torch.equal(wd[b, :, m:].cpu(), w0[b, :, m:])  # behind the last: as it was
        assert bool((step[b, :, m:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
def test_attend_scales_and_late_maxima(gpu, scale):
    """Scores that keep growing along the cache, and scales of every sign."""
    D, Hkv, n = 128, 1, 700
    cache, table, lens, cu, k, v = _filled([n], Hkv, D, 16)
    k = (k.float() * torch.linspace(0.1, 3, n)[:, None, None]).to(torch.bfloat16)
    fa.cache4_append(cache, k.cuda(), v.cuda(), table, _i32([0]), _i32(cu))
    q = k[n - 1, 0][None, None].expand(1, 4, D).contiguous()  # points at the last key
    o, lse = fa.cache4_attend(q.cuda(), cache, table, lens, scale=scale)
    r = ref.attend(q[0], k, v, scale)
    assert_within(lse[0], r["lse"], r["lse_tol"], "lse")
    assert_within(o[0], r["o"], r["o_tol"], "o")


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shift", [29, -20])
def test_attend_is_the_same_at_other_magnitudes(gpu, D, shift):
    """Powers of two on q, k and v change no code and no rounding: the scores are
    the same, and O is O times the power, to the bit."""
    up, Hkv = 2.0 ** shift, 2
    cache, table, lens, cu, k, v = _filled([130, 1501, 0, 17], Hkv, D, 32)
    q = torch.randn(4, 6, D, device="cuda").to(torch.bfloat16)
    w = torch.zeros(2, 4, Hkv, 1501, device="cuda")
    o, lse = fa.cache4_attend(q, cache, table, lens, weights=w[0])
    fa.cache4_append(cache, (k / up).cuda(), (v * up).cuda(), table, torch.zeros_like(lens), _i32(cu))
    o2, lse2 = fa.cache4_attend(q * up, cache, table, lens, weights=w[1])
    assert torch.equal(o * up, o2) and torch.equal(lse, lse2) and torch.equal(w[0], w[1])
    assert fa.cache4_status() == fa.FA_OK


@pytest.mark.gpu
def test_binding_refusals_of_device_tensors(gpu):
    D, Hkv = 64, 2
    cache, table, lens, *_ = _filled([40, 7], Hkv, D, 16)
    q = torch.randn(2, 4, D, device="cuda").to(torch.bfloat16)
    k = torch.randn(2, Hkv, D, device="cuda").to(torch.bfloat16)
    w = torch.zeros(2, Hkv, 48, device="cuda")
    out = table + table.numel()
    good = dict(q=q, cache=cache, page_table=table, cache_lens=lens, weights=w)
    fa.cache4_attend(**good)

    def attend(error, **kw):
        with pytest.raises(error):
            fa.cache4_attend(**{**good, **kw})

    attend(TypeError, q=q.float())
    attend(TypeError, q=q.cpu())
    attend(ValueError, q=q[0])
    attend(ValueError, q=q.transpose(1, 2).contiguous().transpose(1, 2))
    attend(TypeError, cache=cache.cpu())
    attend(TypeError, cache=cache.view(torch.int8))
    attend(ValueError, cache=cache[:, :, :-1])
    attend(ValueError, cache=cache[:, :, :-80].contiguous())
    attend(TypeError, page_table=table.long())
    attend(TypeError, page_table=table.cpu())
    attend(ValueError, page_table=table[:1])
    attend(TypeError, cache_lens=lens.long())
    attend(TypeError, cache_lens=[40, 7])
    attend(ValueError, cache_lens=lens[:1])
    attend(TypeError, weights=w.double())
    attend(ValueError, weights=w[:, :1].contiguous())
    attend(ValueError, weights_out=torch.zeros(2, Hkv, 47, device="cuda"))
    attend(ValueError, out=torch.empty(2, 4, D, device="cuda"))
    attend(ValueError, lse=torch.empty(4, 2, device="cuda"))
    attend(ValueError, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    attend(fa.FAError, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    attend(fa.FAError, scale=math.inf)
    attend(TypeError, scale="1")
    attend(fa.FAError, q=q[:, :3])  # three query heads to two kv heads
    with pytest.raises(ValueError):
        fa.cache4_append(cache, k, k[:, :1], table, lens)
    with pytest.raises(ValueError):
        fa.cache4_append(cache, k[:, :1], k[:, :1], table, lens)
    with pytest.raises(fa.FAError):  # one token per sequence without boundaries
        fa.cache4_append(cache, k[:1], k[:1], table, lens)
    with pytest.raises(ValueError):
        fa.cache4_append(cache, k, k, table, lens, _i32([0, 2]))
    with pytest.raises(fa.FAError):
        fa.cache4_read(cache, table, None, lens, -1, D)
    with pytest.raises(ValueError):
        fa.cache4_read(cache, table, lens[:1], lens, 8, D)
    with pytest.raises(ValueError):
        fa.cache4_read(cache, table, None, lens, 8, 96)
    for budget, recent in ((0, 0), (8, 9), (8, -1), (table.shape[1] * 16 + 1, 0)):
        with pytest.raises(ValueError):
            fa.cache4_evict(cache, table, lens, w, out, D, budget, recent)
    with pytest.raises(TypeError):
        fa.cache4_evict(cache, table, lens, w, out, D, 8.0)
    with pytest.raises(OverflowError):
        fa.cache4_evict(cache, table, lens, w, out, D, 1 << 40)
    assert fa.cache4_status() == fa.FA_OK


@pytest.mark.gpu
def test_calls_on_two_streams_at_once(gpu):
    D, Hkv = 128, 2
    sets = []
    for n in (300, 2000, 700):  # one block per row, shares, both
        cache, table, lens, *_ = _filled([n, 3 * n], Hkv, D, 64, seed=n)
        q = torch.randn(2, 8, D, device="cuda").to(torch.bfloat16)
        sets.append((q, cache, table, lens))
    want = [fa.cache4_attend(*x) for x in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for st in streams:
            got.append([fa.cache4_attend(*x, stream=st) for x in sets])
    torch.cuda.synchronize()
    for run in got:
        for (o, lse), (o2, lse2) in zip(want, run):
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
def test_attend_one_row_of_any_stride(gpu):
    """The stride of a dimension of one element means nothing."""
    D = 64
    cache, table, lens, *_ = _filled([40], 1, D, 16)
    q = torch.randn(2 * D, device="cuda").to(torch.bfloat16)
    a = fa.cache4_attend(q[:D].view(1, 1, D), cache, table, lens)
    b = fa.cache4_attend(q.as_strided((1, 1, D), (3, 5, 1)), cache, table, lens)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_attend_repeats_to_the_bit_and_takes_strides(gpu):
    D, Hkv, group = 64, 2, 3
    cache, table, n, *_ = _filled([500, 1200, 3], Hkv, D, 32)
    wide = torch.randn(3, 2 * Hkv * group, D, device="cuda").to(torch.bfloat16)
    q = wide[:, ::2]
    w = torch.zeros(3, Hkv, 1200, device="cuda")
    a = fa.cache4_attend(q, cache, table, n, weights_out=w)
    for _ in range(3):
        w2 = torch.zeros_like(w)
        b = fa.cache4_attend(q.contiguous(), cache, table, n, weights_out=w2)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(w, w2)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,budget,recent", [
    ([50, 7, 300], 40, 10), ([33], 32, 0), ([100, 64, 65], 64, 64), ([2500, 1, 0], 999, 17),
    ([40], 1, 0), ([40], 1, 1), ([5000], 17, 5), ([17000, 16384], 4099, 100)])
def test_evict(gpu, D, lens, budget, recent):
    Hkv, page = 2, (16 if max(lens) < 6000 else 128)
    cache, table, n, cu, k, v = _filled(lens, Hkv, D, page)
    gen = torch.Generator().manual_seed(budget)
    slots = max(lens) + 3
    w = (torch.rand(len(lens), Hkv, slots, generator=gen) * 8).round() / 8  # nine values: ties
    w[:, 0] = torch.rand(len(lens), slots, generator=gen)
    w[0, 1, : lens[0] // 2] = 0.0
    kept = [min(x, budget) for x in lens]
    extra, m = _table([budget] * len(lens), page, 3, spare=0, first=cache.shape[0])
    big = torch.cat((cache, torch.full((m, *cache.shape[1:]), 255, dtype=torch.uint8,
                                       device="cuda")))
    before = big.clone()
    src, w_out, n_out = fa.cache4_evict(big, table, n, w.cuda(), extra, D, budget, recent)
    assert fa.cache4_status() == fa.FA_OK
    assert torch.equal(big[: cache.shape[0]], before[: cache.shape[0]])  # the old pages stay
    assert n_out.tolist() == kept
    old = fa.cache4_read(big, table, None, n, max(lens) or 1, D)
    new = fa.cache4_read(big, extra, None, n_out, budget, D)
    for b, x in enumerate(lens):
        for h in range(Hkv):
            want = ref.evict(w[b, h], x, budget, recent)
            assert src[b, h].tolist() == want + [-1] * (budget - len(want))
            assert torch.equal(w_out[b, h, : len(want)].cpu(), w[b, h, want])
            assert bool((w_out[b, h, len(want):] == 0).all())
            for a, c in zip(old, new):
                assert torch.equal(c[b, h, : len(want)], a[b, h, want])
    # the lengths updated in place
    src2, w2, n2 = fa.cache4_evict(big, table, n, w.cuda(), extra, D, budget, recent, lens_out=n)
    assert n2 is n and n.tolist() == kept
    assert torch.equal(src2, src) and torch.equal(w2, w_out)


@pytest.mark.gpu
def test_bad_tables_and_lengths_are_reported(gpu):
    """Ids outside the pool, lengths outside the table: no access there, a status."""
    D, Hkv, page = 128, 2, 16
    cache, table, n, cu, k, v = _filled([40, 20], Hkv, D, page)
    q = torch.randn(2, 4, D, device="cuda").to(torch.bfloat16)
    good = fa.cache4_attend(q, cache, table, n)
    assert fa.cache4_status() == fa.FA_OK
    bad = table.clone()
    bad[0, 1] = cache.shape[0]
    bad[1, 1] = -1
    o, lse = fa.cache4_attend(q, cache, bad, n)
    assert fa.cache4_status() == 1 and fa.cache4_status() == fa.FA_OK
    left = [torch.cat((x[:16], x[32:40])) for x in (k, v)]  # slots 16..31 are left out
    r = ref.attend(q[0].cpu(), *left)
    assert_within(o[0], r["o"], r["o_tol"], "o without the bad page")
    before = cache.clone()
    fa.cache4_append(cache, k[:2].cuda(), v[:2].cuda(), bad, _i32([16, 16]))
    assert fa.cache4_status() == 1 and torch.equal(cache, before)
    vals = fa.cache4_read(cache, bad, None, n, 40, D)
    assert fa.cache4_status() == 1 and bool((vals[0][0, :, 16:32] == 0).all())
    fa.cache4_append(cache, k[:2].cuda(), v[:2].cuda(), table, _i32([-1, 10000]))
    assert fa.cache4_status() == 1 and torch.equal(cache, before)
    fa.cache4_attend(q, cache, table, _i32([1 << 30, -5]))
    assert fa.cache4_status() == 1
    out_table, m = _table([16, 16], page, 1, spare=0, first=cache.shape[0] - 2)  # past the pool
    w = torch.rand(2, Hkv, 64, device="cuda")
    fa.cache4_evict(cache, table, n, w, out_table + 2, D, 16, 4)
    assert fa.cache4_status() == 1 and torch.equal(cache, before)
    again = fa.cache4_attend(q, cache, table, n)
    assert fa.cache4_status() == fa.FA_OK
    assert torch.equal(good[0], again[0])


@pytest.mark.gpu
def test_captured_steps(gpu):
    """A captured append + attend step replays as the cache grows; a second graph with
    its own workspace runs beside it; a call on another stream gives the same bits."""
    D, Hkv, group, page, B = 128, 2, 4, 16, 3
    lens = [14, 0, 100]
    cache, _, _, cu, k, v = _filled(lens, Hkv, D, page)
    table, n_pages = _table([200] * B, page, 9)
    cache = fa.cache4_empty(n_pages, Hkv, D, page)
    fa.cache4_append(cache, k.cuda(), v.cuda(), table, _i32([0] * B), _i32(cu))
    n = _i32(lens)
    one = _i32([1] * B)
    kn, vn = (torch.zeros(B, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(B, Hkv * group, D, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(B, Hkv, 200, device="cuda")
    bufs = [[torch.empty(fa.cache4_attend_workspace_bytes(B, Hkv * group, Hkv, D, 200),
                         dtype=torch.uint8, device="cuda"),
             torch.zeros_like(q), torch.zeros(B, Hkv * group, device="cuda")] for _ in range(2)]

    def step(buf, **kw):
        fa.cache4_attend(q, cache, table, n, out=buf[1], lse=buf[2], workspace=buf[0], **kw)

    step(bufs[0])
    fa.cache4_append(cache, kn, vn, table, n)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        fa.cache4_append(cache, kn, vn, table, n)
        n.add_(one)
        step(bufs[0], weights=w)
    with torch.cuda.graph(g2):
        step(bufs[1])
    side = torch.cuda.Stream()
    ks = [[k[cu[b]:cu[b + 1]]] for b in range(B)]
    vs = [[v[cu[b]:cu[b + 1]]] for b in range(B)]
    total = [torch.zeros(Hkv, 200, dtype=torch.float64) for _ in range(B)]
    tol = [torch.zeros(Hkv, 200, dtype=torch.float64) for _ in range(B)]
    for i in range(5):
        a, c = _kv(B, Hkv, D, 100 + i)
        kn.copy_(a)
        vn.copy_(c)
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(i)).bfloat16())
        g1.replay()
        g2.replay()
        side.wait_stream(torch.cuda.current_stream())
        other = fa.cache4_attend(q, cache, table, n, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(bufs[0][1], bufs[1][1]) and torch.equal(bufs[0][1], other[0])
        for b in range(B):
            ks[b].append(a[b:b + 1])
            vs[b].append(c[b:b + 1])
            r = ref.attend(q[b].cpu(), torch.cat(ks[b]), torch.cat(vs[b]))
            assert_within(bufs[0][1][b], r["o"], r["o_tol"], f"step {i} sequence {b}")
            m = r["p"].shape[1]
            total[b][:, :m] += r["p"]
            tol[b][:, :m] += r["p_tol"] + 2.0 ** -23 * total[b][:, :m]
            assert_within(w[b], total[b], tol[b], f"weights {i} {b}")
    assert fa.cache4_status() == fa.FA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_steps_eviction_steps(gpu, D):
    """The calls as a program makes them: packed prompts, their store, steps with
    weights, an eviction to fresh pages, more steps."""
    Hkv, group, page, budget, recent = 2, 4, 16, 48, 16
    lens = [130, 60, 20]
    B, cu = len(lens), _cu(lens)
    gen = torch.Generator().manual_seed(77)
    k, v = _kv(cu[-1], Hkv, D, 70)
    q = torch.randn(cu[-1], Hkv * group, D, generator=gen).to(torch.bfloat16)
    o, lse = fa.fwd_varlen(q.cuda(), k.cuda(), v.cuda(), _i32(cu), causal=True)
    r = packed(q, k, v, list(zip(cu, cu[1:])))
    assert_within(o, r["o"], r["o_tol"], "prompt")
    table, n_pages = _table([max(lens) + 8] * B, page, 1)
    fresh, n_fresh = _table([budget + 8] * B, page, 2, first=n_pages)
    cache = fa.cache4_empty(n_pages + n_fresh, Hkv, D, page)
    n = _i32([0] * B)
    fa.cache4_append(cache, k.cuda(), v.cuda(), table, n, _i32(cu))
    n += _i32(lens)
    slots = max(lens) + 8
    w = torch.zeros(B, Hkv, slots, device="cuda")
    # per (sequence, kv head): the keys and values held, as the program's own record
    held = [[(k[cu[b]:cu[b + 1], h], v[cu[b]:cu[b + 1], h]) for h in range(Hkv)] for b in range(B)]

    def steps(first, count, table, n, w):
        for i in range(first, first + count):
            a, c = _kv(B, Hkv, D, 200 + i)
            qs = torch.randn(B, Hkv * group, D, generator=gen).to(torch.bfloat16)
            fa.cache4_append(cache, a.cuda(), c.cuda(), table, n)
            n += 1
            o, lse = fa.cache4_attend(qs.cuda(), cache, table, n, weights=w)
            for b in range(B):
                for h in range(Hkv):
                    kk, vv = held[b][h]
                    kk, vv = torch.cat((kk, a[b:b + 1, h])), torch.cat((vv, c[b:b + 1, h]))
                    held[b][h] = (kk, vv)
                    heads = slice(h * group, (h + 1) * group)
                    r = ref.attend(qs[b, heads], kk[:, None], vv[:, None])
                    assert_within(o[b, heads], r["o"], r["o_tol"], f"step {i}, {b}, {h}")
                    assert_within(lse[b, heads], r["lse"], r["lse_tol"], f"lse {i}, {b}, {h}")

    steps(0, 4, table, n, w)
    src, w2, n2 = fa.cache4_evict(cache, table, n, w, fresh, D, budget, recent)
    for b in range(B):
        for h in range(Hkv):
            want = ref.evict(w[b, h].cpu(), lens[b] + 4, budget, recent)
            assert src[b, h, :len(want)].tolist() == want
            held[b][h] = tuple(x[want] for x in held[b][h])
    w3 = torch.zeros(B, Hkv, budget + 8, device="cuda")
    w3[:, :, :budget] = w2
    steps(4, 4, fresh, n2, w3)
    assert fa.cache4_status() == fa.FA_OK
    assert n2.tolist() == [min(x + 4, budget) + 4 for x in lens]
