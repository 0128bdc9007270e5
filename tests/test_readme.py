"""README's decoding loop, run as it stands: every step's attention covers what the
cache holds, the newest token included, before and after evictions."""
import os
import re

import pytest
import torch

import __graft_entry__
import cache4_reference as ref
import exact_attention_blackwell_tiled_gb300 as fa
from packed_reference import assert_within

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def _loop():
    with open(README, encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    return next(b for b in blocks if "cache4_evict" in b)


def test_blocks_compile():
    compile(_loop(), README, "exec")


@pytest.mark.gpu
def test_decoding_loop():
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    D, Hkv, group, every, budget, recent, count = 128, 2, 4, 5, 48, 16, 18
    cu = [0, 130, 160, 220]
    B = len(cu) - 1
    gen = torch.Generator().manual_seed(41)

    def rand(*shape):
        return torch.randn(*shape, generator=gen).to(torch.bfloat16)

    k, v = rand(cu[-1], Hkv, D), rand(cu[-1], Hkv, D)
    held = [[(k[cu[b]:cu[b + 1], h], v[cu[b]:cu[b + 1], h]) for h in range(Hkv)] for b in range(B)]
    ns = {}

    def steps():
        for i in range(count):
            q1, k1, v1 = rand(B, Hkv * group, D), rand(B, Hkv, D), rand(B, Hkv, D)
            before = ns.get("src")
            yield q1.cuda(), k1.cuda(), v1.cuda()
            evicted = ns.get("src") is not before
            assert evicted == ((i + 1) % every == 0)
            for b in range(B):
                for h in range(Hkv):
                    kk, vv = (torch.cat((x, y[b:b + 1, h])) for x, y in zip(held[b][h], (k1, v1)))
                    heads = slice(h * group, (h + 1) * group)
                    r = ref.attend(q1[b, heads], kk[:, None], vv[:, None])
                    assert_within(ns["o"][b, heads], r["o"], r["o_tol"], f"step {i}, {b}, {h}")
                    assert_within(ns["lse"][b, heads], r["lse"], r["lse_tol"], f"lse {i}, {b}, {h}")
                    if evicted:
                        at = ns["src"][b, h, :min(budget, len(kk))].long().cpu()
                        kk, vv = kk[at], vv[at]
                    held[b][h] = (kk, vv)

    width = -(-(max(130, budget) + every) // 64)
    tables = torch.arange(2 * B * width, dtype=torch.int32, device="cuda").view(2, B, width)
    ns.update(fa=fa, torch=torch, pages=tables.numel(), Hkv=Hkv, D=D, B=B, k=k.cuda(), v=v.cuda(),
              table=tables[0], spare=tables[1], slots=130 + every, steps=steps(), every=every,
              budget=budget, recent=recent,
              cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    exec(compile(_loop(), README, "exec"), ns)
    # (30 tokens and 18 steps never pass the budget of 48)
    assert ns["lens"].tolist() == [budget + count % every, 30 + count, budget + count % every]
