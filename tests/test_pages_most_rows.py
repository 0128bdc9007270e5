"""As many rows of new tokens as fa_page_update takes, 2^31 - 1."""
import pytest
import torch

import __graft_entry__
import exact_attention_blackwell_tiled_gb300 as fa

MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def gpu():
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 40 * 2 ** 30:
        pytest.skip("less than 40 GB free")
    yield
    torch.cuda.empty_cache()


def _sample(n):
    gen = torch.Generator().manual_seed(1)
    at = torch.randint(0, n, (100000,), generator=gen)
    return torch.cat((at, torch.arange(3000), torch.arange(n - 3000, n))).cuda()


@pytest.mark.gpu
def test_every_row_a_token(gpu):
    page, width = 128, 2 ** 23
    lens = [2 ** 30, 2 ** 30 - 1]
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    free, count = fa.page_pool(2 * width)
    new = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu, pos, slots = fa.page_update(table, free, count, torch.zeros_like(new), new, page, MOST)
    assert fa.cache4_status() == fa.FA_OK
    assert cu.tolist() == [0, 2 ** 30, MOST] and count.item() == 0
    at = _sample(MOST)
    b = (at >= 2 ** 30).long()
    i = at - b * 2 ** 30
    assert torch.equal(pos[at].long(), i)
    # pages come from the top of the stack, in the order of (sequence, entry)
    assert torch.equal(slots[at], (2 * width - 1 - b * width - i // page) * page + i % page)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [MOST, MOST - 1022, MOST - 1023])
def test_rows_without_a_token(gpu, T):
    table = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    free, count = fa.page_pool(4)
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu, pos, slots = fa.page_update(table, free, count, lens, lens + 40, 16, T)
    assert fa.cache4_status() == fa.FA_OK and cu.tolist() == [0, 40]
    at = _sample(T)
    live = at < 40
    assert torch.equal(pos[at].long(), torch.where(live, at, -1))
    assert torch.equal(slots[at], torch.where(live, (3 - at // 16) * 16 + at % 16, -1))
