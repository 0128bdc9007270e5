"""torch.use_deterministic_algorithms fills new memory with NaN (the largest number, for
integers): results that a call allocates show it in the rows that the call leaves as they are."""
import pytest
import torch

import __graft_entry__
import exact_attention_blackwell_tiled_gb300 as fa


@pytest.fixture
def deterministic():
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    was = torch.are_deterministic_algorithms_enabled(), torch.utils.deterministic.fill_uninitialized_memory
    torch.use_deterministic_algorithms(True)
    torch.utils.deterministic.fill_uninitialized_memory = True
    try:
        yield
    finally:
        torch.use_deterministic_algorithms(was[0])
        torch.utils.deterministic.fill_uninitialized_memory = was[1]


def _rows(T, H, D, seed):
    return torch.randn(T, H, D, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(None, 0), ((20, 0), 0), ((20, 0), 3)])
def test_rows_of_no_sequence(deterministic, window, sinks):
    T, Hq, Hkv, D = 90, 4, 2, 64
    q, k, v, do = (_rows(T, h, D, i) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    cu = torch.tensor([7, 40, 80], dtype=torch.int32, device="cuda")
    o, lse = fa.fwd_varlen(q, k, v, cu, window=window, sinks=sinks)
    g = fa.bwd_varlen(q, k, v, o, do, lse, cu, window=window, sinks=sinks)
    for x in (o, lse.T, *g):
        assert bool(torch.isnan(x[:7]).all()) and bool(torch.isnan(x[80:]).all())
        assert bool(torch.isfinite(x[7:80]).all())


@pytest.mark.gpu
def test_tokens_of_no_sequence(deterministic):
    T, D = 9, 64
    q, k = _rows(T, 3, D, 1), _rows(T, 1, D, 2)
    w = torch.ones(D, device="cuda")
    cos, sin = fa.rope_table(16, D)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    pos[4] = -1
    out = fa.norm_rope_fwd(q, k, w, w, cos, sin, pos)
    out += fa.norm_rope_bwd(q, k, w, w, cos, sin, pos, q, k)[:2]
    for x in out:
        assert bool(torch.isnan(x[4]).all()) and bool(torch.isfinite(x[[0, 3, 5, 8]]).all())


@pytest.mark.gpu
def test_not_without_the_fill(deterministic):
    """The switch that torch has for it is the one that counts."""
    torch.utils.deterministic.fill_uninitialized_memory = False
    q = _rows(64, 2, 64, 3)
    cu = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    a = fa.fwd_varlen(q, q, q, cu)
    torch.utils.deterministic.fill_uninitialized_memory = True
    b = fa.fwd_varlen(q, q, q, cu)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
