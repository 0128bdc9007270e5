"""The 4-bit cache at the edges of its tables: pages out of range, idle sequences."""
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


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _filled(lens, Hkv, D, page, pages, seed=3):
    """A pool of `pages` pages of other bytes with the sequences in the first ones."""
    gen = torch.Generator().manual_seed(seed)
    T, width = sum(lens), max(-(-n // page) for n in lens)
    k, v = (torch.randn(T, Hkv, D, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    cache = fa.cache4_empty(pages, Hkv, D, page)
    cache.fill_(0x5a)
    table = torch.arange(len(lens) * width, dtype=torch.int32, device="cuda").view(len(lens), width)
    cu = torch.tensor([0, *lens]).cumsum(0).to(torch.int32).cuda()
    fa.cache4_append(cache, k, v, table, _i32([0] * len(lens)), cu)
    return cache, table


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("budget", [24, 100])  # fewer than the tokens, or all of them
def test_evict_of_a_token_whose_page_is_out_of_range(D, budget):
    """It is reported and becomes a token of zeros; nothing of the new page's old bytes is
    left in a live slot, and nothing behind the last slot is written."""
    lens, page, Hkv, recent = [40, 33], 16, 2, 8
    cache, table = _filled(lens, Hkv, D, page, 30)
    n = _i32(lens)
    bad = table.clone()
    bad[0, 1], bad[1, 2] = 30, -1
    w = torch.rand(2, Hkv, 40, generator=torch.Generator().manual_seed(budget)).cuda()
    width = -(-budget // page)
    fresh = (16 + torch.arange(2 * width, dtype=torch.int32, device="cuda")).view(2, width)
    before = cache.clone()
    src, _, kept = fa.cache4_evict(cache, bad, n, w, fresh, D, budget, recent)
    assert fa.cache4_status() == 1
    assert kept.tolist() == [min(x, budget) for x in lens]
    old = fa.cache4_read(before, bad, None, n, 40, D)  # zeros where the page is out of range
    assert fa.cache4_status() == 1
    new = fa.cache4_read(cache, fresh, None, kept, budget, D)
    assert fa.cache4_status() == fa.FA_OK
    for b in range(2):
        m = int(kept[b])
        for h in range(Hkv):
            at = src[b, h, :m].long()
            assert bool((at // page == (1 if b == 0 else 2)).any())  # (some of them are kept)
            for x, y in zip(old, new):
                assert torch.equal(y[b, h, :m], x[b, h, at])
    # slots behind the last kept one: as they were
    full = _i32([width * page] * 2)
    was, now = (fa.cache4_read(c, fresh, None, full, width * page, D) for c in (before, cache))
    for b in range(2):
        for x, y in zip(was, now):
            assert torch.equal(x[b, :, int(kept[b]):], y[b, :, int(kept[b]):])


@pytest.mark.parametrize("D", [64, 128])
def test_read_looks_only_at_pages_with_rows(D):
    """No row of a sequence asked for: its pages, released, are not looked at, wherever
    `first` lies in a block; rows asked for of the last page alone do not report the others."""
    cache, table = _filled([40, 33], 2, D, 16, 6)
    gone = table.clone()
    gone[0] = -1
    k, v = fa.cache4_read(cache, gone, _i32([37, 20]), _i32([0, 9]), 20, D)
    assert fa.cache4_status() == fa.FA_OK
    whole = fa.cache4_read(cache, table, None, _i32([40, 33]), 40, D)
    for x, y in zip((k, v), whole):
        assert bool((x[0] == 0).all()) and bool((x[1, :, 9:] == 0).all())
        assert torch.equal(x[1, :, :9], y[1, :, 20:29])
    gone[0, 2] = table[0, 2]
    k, v = fa.cache4_read(cache, gone, _i32([35, 0]), _i32([5, 0]), 20, D)
    assert fa.cache4_status() == fa.FA_OK
    assert torch.equal(k[0, :, :5], whole[0][0, :, 35:]) and torch.equal(v[0, :, :5], whole[1][0, :, 35:])
    fa.cache4_read(cache, gone, _i32([31, 0]), _i32([5, 0]), 20, D)
    assert fa.cache4_status() == 1  # slot 31 lies on a page that is gone


@pytest.mark.parametrize("first", [None, 3])
def test_read_reports_a_negative_count(first):
    """A length out of range, as the other calls report it; the rows are zeros."""
    cache, table = _filled([40, 33], 2, 64, 16, 6)
    at = None if first is None else _i32([first] * 2)
    k, v = fa.cache4_read(cache, table, at, _i32([8, -2]), 8, 64)
    assert fa.cache4_status() == 1
    assert bool((k[1] == 0).all()) and bool((v[1] == 0).all()) and bool((k[0] != 0).any())


@pytest.mark.parametrize("D", [64, 128])
def test_pages_past_32_bit_offsets(D):
    """A pool of more than 2^32 bytes: the first and the last pages, and the eviction from
    the one end to the other."""
    Hkv, page, lens = 4, 128, [300, 140]
    per_page = fa.cache4_empty(1, Hkv, D, page).numel()
    pages = (1 << 32) // per_page + 40
    gen = torch.Generator().manual_seed(D)
    k, v = (torch.randn(440, Hkv, D, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(2, 2 * Hkv, D, generator=gen).to(torch.bfloat16).cuda()
    n, cu = _i32(lens), _i32([0, 300, 440])
    low = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    high = pages - 6 + low
    cache = fa.cache4_empty(pages, Hkv, D, page)
    got = []
    for table in (low, high):
        fa.cache4_append(cache, k, v, table, _i32([0, 0]), cu)
        w = torch.zeros(2, Hkv, 300, device="cuda")
        out = fa.cache4_attend(q, cache, table, n, weights=w)
        got.append((*out, w, *fa.cache4_read(cache, table, None, n, 300, D)))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert bool((got[0][3] != 0).any())
    src, _, kept = fa.cache4_evict(cache, high, n, got[0][2], low + 6, D, 100, 10)
    new = fa.cache4_read(cache, low + 6, None, kept, 100, D)
    for x, y in zip(got[0][3:], new):
        assert torch.equal(y, x.gather(2, src.long()[..., None].expand(-1, -1, -1, D)))
    assert fa.cache4_status() == fa.FA_OK
