"""Page tables brought up to date on the device (fa_page_update), and appends by slot
(fa_cache4_append_slots), against their definitions in plain Python."""
import ctypes
import random

import pytest
import torch

import __graft_entry__
import cache4_reference as ref
import exact_attention_blackwell_tiled_gb300 as fa

P = ctypes.c_void_p(256 * 1024)
P4 = ctypes.c_void_p(256 * 1024 + 4)
P2 = ctypes.c_void_p(256 * 1024 + 2)


def simulate(table, stack, height, lens, new, page, wl, sinks, T):
    """The definition, entry by entry.  Returns what the call leaves and returns, and whether
    it records something."""
    table, stack = [list(r) for r in table], list(stack)
    pages, bad = len(stack), False
    wanted = []
    for b, (had, has) in enumerate(zip(lens, new)):
        n0, n1 = -(-had // page), -(-has // page)
        for e in range(max(n0, n1)):
            hidden = wl >= 0 and (e + 1) * page <= has - 1 - wl and e * page >= sinks
            if e >= n0:
                if not hidden:
                    wanted.append((b, e))
            elif (hidden or e >= n1) and 0 <= table[b][e] < pages:
                stack[height] = table[b][e]
                height += 1
                table[b][e] = -1
    for b, e in wanted:
        height -= 1
        table[b][e] = stack[height] if height >= 0 else -1
        bad |= height < 0
    cu, pos, slots = [0], [], []
    for b, (had, has) in enumerate(zip(lens, new)):
        for i in range(had, has):
            p = table[b][i // page]
            pos.append(i)
            slots.append(p * page + i % page if p >= 0 else -1)
        cu.append(len(pos))
    bad |= len(pos) > T
    pad = [-1] * max(0, T - len(pos))
    return (table, stack, max(height, 0), [min(x, T) for x in cu], (pos + pad)[:T], (slots + pad)[:T],
            bad)


# ------------------------------------------------------------------ without a GPU

@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return fa.lib()


def test_refusals(L):
    def call(table=P, width=4, stack=P, count=P, pages=9, lens=P, new=P, B=2, page=16, sinks=0, T=3,
             cu=P, pos=P, slots=P):
        return L.fa_page_update(table, width, stack, count, pages, lens, new, B, page, -1, sinks, T, cu,
                                pos, slots, None)
    for name in ("table", "stack", "count", "lens", "new", "cu", "pos", "slots"):
        assert call(**{name: None}) == 1
    assert call(B=0) == 1 and call(B=65537) == 1 and call(pages=0) == 1 and call(width=0) == 1
    assert call(T=-1) == 1 and call(sinks=-1) == 1
    assert call(page=24) == 2
    assert call(B=65536, width=1 << 14) == 1
    assert call(table=P2) == 3 and call(pos=P2) == 3 and call(slots=P4) == 3

    def slot(cache=P, k=P, slots=P, T=3, D=64, s=None):
        return L.fa_cache4_append_slots(cache, 4, 16, k, P, None if s is None else
                                        ctypes.byref(fa.PackedStride(*s)), None, T, 2, D, slots, None)
    assert slot(cache=None) == 1 and slot(slots=None) == 1 and slot(T=-1) == 1
    assert slot(D=80) == 2
    assert slot(k=P4) == 3 and slot(slots=P4) == 3 and slot(s=(130, 64)) == 3
    assert slot(T=0, slots=None) == 0


def test_simulation_on_a_small_case():
    # 16-token pages, window 20, one sink: at 70 tokens entries 1 and 2 are hidden
    out = simulate([[5, 6, 7, -1, -1, -1], [1, -1, -1, -1, -1, -1]], [0, 2, 3, 4, -1, -1, -1, -1], 4,
                   [48, 9], [70, 0], 16, 20, 1, 24)
    assert out[0] == [[5, -1, -1, 1, 7, -1], [-1] * 6]
    assert out[1][:7] == [0, 2, 3, 4, 6, 7, 1] and out[2] == 5
    assert out[3] == [0, 22, 22] and out[4][:2] == [48, 49] and out[4][-2:] == [-1, -1]
    assert out[5][0] == 16 and out[5][21] == 7 * 16 + 5 and not out[6]


# ------------------------------------------------------------------ on the GPU

@pytest.fixture(scope="module")
def gpu():
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _state(rng, B, page, most, wl, sinks, lens, extra):
    """Tables as earlier calls left them, and a pool with `extra` pages beyond them."""
    width = most // page + 1
    held = [[e * page < n and not (wl >= 0 and (e + 1) * page <= n - 1 - wl and e * page >= sinks)
             for e in range(width)] for n in lens]
    used = sum(map(sum, held))
    pages = used + extra
    order = list(range(pages))
    rng.shuffle(order)
    table = [[order.pop() if h else rng.choice([-1, -7, pages, 2 ** 31 - 1]) if e * page >= n else -1
              for e, h in enumerate(row)] for row, n in zip(held, lens)]
    return table, order + [-1] * used, len(order)


def _check(table, stack, height, lens, new, page, wl, sinks, T, stream=None):
    want = simulate(table, stack, height, lens, new, page, wl, sinks, T)
    d = [_i32(table), _i32(stack), _i32([height])]
    got = fa.page_update(*d, _i32(lens), _i32(new), page, T, window_left=wl, sinks=sinks)
    bad = fa.cache4_status()
    assert d[0].tolist() == want[0]
    assert d[1].tolist() == want[1]
    assert d[2].tolist() == [want[2]]
    assert got[0].tolist() == want[3] and got[1].tolist() == want[4] and got[2].tolist() == want[5]
    assert bad == (1 if want[6] else 0)
    return want


@pytest.mark.gpu
@pytest.mark.parametrize("B,most,grow", [(1, 1, 1), (1, 5000, 1), (1, 200, 4097), (3, 40, 33), (32, 300, 1),
                                         (33, 100, 7), (64, 2000, 1), (65, 300, 40), (200, 60, 90),
                                         (1024, 100, 1), (1500, 30, 20)])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_against_the_definition(gpu, B, most, grow, page):
    rng = random.Random(B * 1000 + most + page)
    for wl, sinks in ((-1, 0), (0, 0), (33, 4), (500, 1), (100, 200)):
        lens = [rng.choice([0, rng.randrange(most + 1), most]) for _ in range(B)]
        new = [rng.choice([n + rng.randrange(grow + 1), n + 1, n + 1, n, rng.randrange(n + 1), 0])
               for n in lens]
        T = sum(max(0, b - a) for a, b in zip(lens, new))
        state = _state(rng, B, page, most + grow + 1, wl, sinks, lens,
                       sum(max(0, -(-b // page) - -(-a // page)) for a, b in zip(lens, new)) + 1)
        _check(*state, lens, new, page, wl, sinks, T + rng.choice([0, 0, 5]))


@pytest.mark.gpu
def test_pool_too_small_and_rows_too_few(gpu):
    rng = random.Random(4)
    lens, new = [30, 0, 64], [100, 50, 64]
    state = _state(rng, 3, 16, 120, -1, 0, lens, 4)
    out = _check(*state, lens, new, 16, -1, 0, 120)
    assert out[6] and out[2] == 0
    state = _state(rng, 3, 16, 120, -1, 0, lens, 50)
    assert _check(*state, lens, new, 16, -1, 0, 77)[6]
    # pages that come back serve the call's own new tokens
    state = _state(rng, 2, 16, 80, -1, 0, [64, 0], 0)
    out = _check(*state, [64, 0], [0, 64], 16, -1, 0, 64)
    assert not out[6] and out[2] == 0


@pytest.mark.gpu
def test_lengths_and_counts_out_of_range(gpu):
    """Cut and recorded; nothing out of bounds is touched."""
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    free, count = fa.page_pool(20)
    guard = table.clone()
    cu, pos, slots = fa.page_update(table, free, count, _i32([-5, 0, 0]), _i32([3, 65, 2 ** 31 - 1]), 16, 140)
    assert fa.cache4_status() == 1
    assert cu.tolist() == [0, 3, 67, 131] and count.item() == 20 - 1 - 4 - 4
    assert pos[:3].tolist() == [0, 1, 2] and pos[67:131].tolist() == list(range(64))
    assert pos[131:].tolist() == [-1] * 9 and bool((slots[:131] >= 0).all())
    table.copy_(guard)
    for given, left in ((-4, 0), (25, 19)):
        free, count = fa.page_pool(20)
        count.fill_(given)
        fa.page_update(table, free, count, _i32([0, 0, 0]), _i32([1, 0, 0]), 16, 1)
        assert fa.cache4_status() == 1 and count.item() == left
        assert table[0, 0].item() == (-1 if given < 0 else 19)
        table.copy_(guard)
    # a page named twice comes back once too often: the stack ends at its last element
    table[:, 0] = 3
    free, count = fa.page_pool(5)
    count.fill_(4)
    fa.page_update(table, free, count, _i32([1, 1, 1]), _i32([0, 0, 0]), 16, 0)
    assert fa.cache4_status() == 1 and count.item() == 5 and free.tolist() == [0, 1, 2, 3, 3]


@pytest.mark.gpu
@pytest.mark.parametrize("B,width", [(1, 9001), (3, 2501), (40, 2050), (70, 1283), (64, 2049)])
def test_long_tables_under_a_window(gpu, B, width):
    """Many pages behind a window at once, in rows that begin at any 4 bytes, with holes; then
    the next step, which finds them gone."""
    rng = random.Random(B)
    lens, table, used = [], [], 0
    for b in range(B):
        n = rng.choice([width * 16 - 3, width * 16 // 2, rng.randrange(1, width * 16 - 2), 5])
        row = [-1] * width
        for e in range(-(-n // 16)):
            if rng.random() < 0.9:
                row[e], used = used, used + 1
        lens.append(n)
        table.append(row)
    stack = list(range(used, used + 9 * B))
    new = [n + rng.randrange(0, 3) for n in lens]
    _check(table, stack + [0] * used, len(stack), lens, new, 16, 1000, 20, 3 * B)
    new = [rng.choice([0, n, n // 3]) for n in lens]  # shorter ones give back both ends
    _check(table, stack + [0] * used, len(stack), lens, new, 16, 777, 0, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [8192, 8193, 50000])
def test_many_new_tokens(gpu, T):
    """Prompts of many tokens, more than the one launch writes, some of them empty."""
    rng = random.Random(T)
    new, left = [], T
    while left:
        n = min(left, rng.choice([0, 1, 3, 200, 3000]))
        new.append(n)
        left -= n
    B, width = len(new), 3000 // 16 + 1
    pages = sum(-(-n // 16) for n in new)
    _check([[-1] * width for _ in new], list(range(pages)), pages, [0] * B, new, 16, -1, 0, T)
    _check([[-1] * width for _ in new], list(range(pages)), pages, [0] * B, new, 16, 100, 5, T + 1500)


@pytest.mark.gpu
def test_more_sequences_than_a_stretch(gpu):
    """A thousand tokens of more sequences than one block of the second launch keeps."""
    B = 30000
    table = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    free, count = fa.page_pool(B)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = (torch.arange(B, device="cuda") % 3 == 1).int()
    T = 10000
    cu, pos, slots = fa.page_update(table, free, count, lens, new, 16, T)
    assert fa.cache4_status() == fa.FA_OK and int(cu[-1]) == T == int(new.sum())
    at = torch.arange(T, device="cuda")
    assert torch.equal(slots, (B - 1 - at) * 16) and bool((pos == 0).all())


@pytest.mark.gpu
def test_many_sequences(gpu):
    """The most there can be, in closed form: a page and a token each."""
    B = 65536
    table = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    free, count = fa.page_pool(B)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    cu, pos, slots = fa.page_update(table, free, count, lens, lens + 1, 16, B)
    at = torch.arange(B, device="cuda")
    assert torch.equal(table[:, 0].long(), B - 1 - at) and count.item() == 0
    assert torch.equal(slots, (B - 1 - at) * 16) and torch.equal(cu[:-1].long(), at)
    assert bool((pos == 0).all()) and fa.cache4_status() == fa.FA_OK
    fa.page_update(table, free, count, lens + 1, lens, 16, 0)
    assert torch.equal(free.long(), B - 1 - at) and count.item() == B and bool((table == -1).all())


@pytest.mark.gpu
@pytest.mark.parametrize("B", [10, 70])
def test_a_captured_step_replays(gpu, B):
    """Many steps of one graph against the simulation: windows, ends and starts."""
    rng = random.Random(9)
    page, wl, sinks, width, pages = 16, 40, 3, 12, 5 * B
    T = 6 * B
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, count = fa.page_pool(pages)
    lens, new = _i32([0] * B), _i32([0] * B)

    def step():
        out = fa.page_update(table, free, count, lens, new, page, T, window_left=wl, sinks=sinks)
        lens.copy_(new)
        return out
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    state = (table.tolist(), free.tolist(), count.item())
    old = [0] * B
    for i in range(60):
        nxt = [0 if rng.random() < 0.05 else min(n + rng.choice([1, 1, 1, 6]), width * page) for n in old]
        want = simulate(*state, old, nxt, page, wl, sinks, T)
        new.copy_(_i32(nxt))
        graph.replay()
        assert out[0].tolist() == want[3] and out[1].tolist() == want[4] and out[2].tolist() == want[5]
        state, old = want[:3], nxt
        assert table.tolist() == want[0] and count.item() == want[2]
    assert fa.cache4_status() == fa.FA_OK
    held = [p for row in state[0] for p in row if p >= 0]
    assert sorted(held + state[1][:state[2]]) == list(range(pages))  # no page lost, none twice


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_append_by_slot(gpu, D):
    """The same cache as by table; tokens without a slot are nowhere; a slot past the last
    page is recorded."""
    Hkv, page, lens = 3, 32, [37, 0, 70]
    T = sum(lens)
    gen = torch.Generator().manual_seed(D)
    fused = torch.randn(T + 4, 2 * Hkv, D, generator=gen).to(torch.bfloat16).cuda()
    k, v = fused[:, :Hkv], fused[:, Hkv:]
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    free, count = fa.page_pool(9)
    cu, pos, slots = fa.page_update(table, free, count, _i32([0] * 3), _i32(lens), page, T + 4)
    a, b = (fa.cache4_empty(9, Hkv, D, page) for _ in range(2))
    fa.cache4_append(a, k, v, table, _i32([0] * 3), cu)
    fa.cache4_append_slots(b, k, v, slots)
    assert fa.cache4_status() == fa.FA_OK and torch.equal(a, b)
    got = fa.cache4_read(b, table, None, _i32(lens), 70, D)
    z, mn, c = ref.quantise(k[:37].cpu())
    val = (mn[..., None] + c[..., None] * z).flatten(-2).to(torch.bfloat16)
    assert torch.equal(got[0][0, :, :37].cpu(), val.transpose(0, 1))
    slots[5] = 9 * page
    slots[6] = 2 ** 62
    before = b.clone()
    fa.cache4_append_slots(b, k, v, slots)
    assert fa.cache4_status() == 1 and torch.equal(b, before)


@pytest.mark.gpu
def test_binding_refusals(gpu):
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    free, count = fa.page_pool(6)
    lens = _i32([0, 0])
    good = dict(page_table=table, free_pages=free, free_count=count, lens=lens, new_lens=lens, page_size=16, T=0)
    fa.page_update(**good)

    def call(error, **kw):
        with pytest.raises(error):
            fa.page_update(**{**good, **kw})
    call(TypeError, page_table=table.cpu())
    call(TypeError, page_table=table.long())
    call(TypeError, free_pages=free.cpu())
    call(ValueError, free_count=free)
    call(ValueError, new_lens=lens[:1])
    call(TypeError, lens=[0, 0])
    call(fa.FAError, T=-1)
    call(fa.FAError, page_size=8)
    call(fa.FAError, sinks=-1)
    call(ValueError, slots=torch.zeros(0, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        fa.cache4_append_slots(fa.cache4_empty(2, 1, 64, 16), *(torch.zeros(
            2, 1, 64, dtype=torch.bfloat16, device="cuda"),) * 2, lens)
