"""Packed calls of more sequences than the plan keeps the lengths of (4096): those
around that number and behind it, forward and both backward modes."""
import pytest
import torch

import __graft_entry__
import exact_attention_blackwell_tiled_gb300 as fa
from packed_reference import assert_within, packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "none"])
@pytest.mark.parametrize("D", [64, 128])
def test_sequences_past_the_kept_lengths(D, causal):
    gen = torch.Generator().manual_seed(81)
    lens = torch.randint(0, 5, (4500,), generator=gen).tolist()
    # a few long ones, so that items of one sequence stand between those of others
    lens[4094], lens[4095], lens[4096], lens[4097], lens[4400] = 130, 257, 300, 1, 129
    lens += [700, 0, 3]
    cu = torch.tensor([0, *lens]).cumsum(0)
    T = int(cu[-1])
    q, k, v, do = (torch.randn(T, h, D, generator=gen).to(torch.bfloat16) for h in (4, 2, 2, 4))
    picked = [*range(4090, 4101), 4399, 4400, 4401, 4499, 4500, 4501, 4502]
    ref = packed(q, k, v, [(int(cu[i]), int(cu[i + 1])) for i in picked], causal=causal, do=do)
    qd, kd, vd, dod = (x.cuda() for x in (q, k, v, do))
    cud = cu.to(torch.int32).cuda()
    o, lse = fa.fwd_varlen(qd, kd, vd, cud, causal=causal)
    assert fa.fwd_status() == fa.FA_OK
    assert_within(o, ref["o"], ref["o_tol"], "o")
    assert_within(lse, ref["lse"], ref["lse_tol"], "lse")
    for det in (False, True):
        grads = fa.bwd_varlen(qd, kd, vd, o, dod, lse, cud, causal=causal, deterministic=det)
        for g, n in zip(grads, ("dq", "dk", "dv")):
            assert_within(g, ref[n], ref[n + "_tol"], f"{n} det={det}")
        if det:
            again = fa.bwd_varlen(qd, kd, vd, o, dod, lse, cud, causal=causal, deterministic=True)
            for a, b in zip(grads, again):
                assert torch.equal(a, b)


def test_tensors_past_32_bit_offsets():
    """More than 2^31 elements of q, o and their gradients: the last sequences against the
    reference on their rows alone."""
    Hq, Hkv, D, n, tail = 128, 2, 128, 128, [77, 300]
    lens = [n] * 1050 + tail
    cu = torch.tensor([0, *lens]).cumsum(0)
    T = int(cu[-1])
    assert T * Hq * D > 2 ** 31
    torch.manual_seed(5)
    q, do = (torch.randn(T, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.randn(T, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cud = cu.to(torch.int32).cuda()
    o, lse = fa.fwd_varlen(q, k, v, cud, causal=True)
    lo = T - sum(tail)
    heads = [0, 1, 63, 64, 127]  # of both kv heads
    rows = [x[lo:].cpu() for x in (q, k, v, do)]
    bounds = [(0, tail[0]), (tail[0], sum(tail))]

    def check(got, name, ref):
        assert_within(got, ref[name], ref[name + "_tol"], name)

    refs = []
    for h in heads:
        g = h // (Hq // Hkv)
        r = packed(rows[0][:, h:h + 1], rows[1][:, g:g + 1], rows[2][:, g:g + 1], bounds,
                   do=rows[3][:, h:h + 1])
        refs.append(r)
        check(o[lo:, h:h + 1], "o", r)
        check(lse[h:h + 1, lo:], "lse", r)
    for det in (False, True):
        dq, dk, dv = fa.bwd_varlen(q, k, v, o, do, lse, cud, causal=True, deterministic=det)
        for h, r in zip(heads, refs):
            check(dq[lo:, h:h + 1], "dq", r)
        del dq, dk, dv
    assert fa.fwd_status() == fa.FA_OK
