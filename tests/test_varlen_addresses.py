"""Packed calls whose tensors lie all over the address space, from call to call
somewhere else: strided and contiguous inputs, offsets, scales of every sign, windows.
(Tensor maps that one kernel wrote for the next one to load by once ended such a run in
an illegal access.)"""
import math
import random

import pytest
import torch

import __graft_entry__
import exact_attention_blackwell_tiled_gb300 as fa
from packed_reference import assert_within, packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def scattered():
    """Some 300 MB in pieces of 0.9 MB, half of them given back, so that small tensors
    land between the others, in segments far apart."""
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    held = [torch.empty(900 << 10, dtype=torch.uint8, device="cuda") for _ in range(330)]
    random.Random(4).shuffle(held)
    del held[165:]
    yield held


@pytest.mark.parametrize("seed", range(40))
def test_cases(scattered, seed):
    rng = random.Random(seed)
    D, Hkv = rng.choice([64, 128]), rng.choice([1, 2])
    Hq = Hkv * rng.choice([1, 2, 3])
    scale = rng.choice([None, None, -0.1, 0.0, 0.5])
    window = rng.choice([(-1, 0), (-1, -1), (rng.choice([0, 63, 200]), rng.choice([-1, 0, 5, 128]))])
    lens = [rng.choice([0, 1, rng.randint(1, 64), rng.randint(1, 500)]) for _ in range(rng.randint(1, 9))]
    first = rng.choice([0, 3])
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    T = max(1, cu[-1] + rng.randint(0, 5))
    gen = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=gen).to(torch.bfloat16)
    do = torch.randn(T, Hq, D, generator=gen).to(torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    # (the bounds are proportional to the scale's magnitude: give the reference |scale|
    # and the sign with q)
    size = 1 / math.sqrt(D) if scale is None else abs(scale)
    sign = -1 if scale is not None and scale < 0 else 1
    ref = packed(q * sign, k, v, list(zip(cu, cu[1:])), window=window, scale=size, do=do)
    if sign < 0:
        ref["dq"] = -ref["dq"]  # q * sign is the leaf there
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    big, dod = qkv.cuda(), do.cuda()
    parts = [big[:, :Hq], big[:, Hq:Hq + Hkv], big[:, Hq + Hkv:]]
    leaves = [x.detach().clone().requires_grad_() for x in parts]
    o = fa.attention_varlen(*leaves, cud, scale=scale, window=window, deterministic=seed % 2 == 0)
    o.backward(dod)
    o2, lse = fa.fwd_varlen(*parts, cud, scale=scale, window=window)
    assert fa.fwd_status() == fa.FA_OK
    assert torch.equal(o.detach()[first:cu[-1]], o2[first:cu[-1]])
    assert_within(o, ref["o"], ref["o_tol"], "o")
    assert_within(lse, ref["lse"], ref["lse_tol"], "lse")
    for x, n in zip(leaves, ("dq", "dk", "dv")):
        assert_within(x.grad, ref[n], ref[n + "_tol"], n)
