"""README's serving loop under a window with sinks, run as it stands: prompts, steps, the end
of all sequences."""
import os
import re

import pytest
import torch

import __graft_entry__
import cache4_reference as ref
import exact_attention_blackwell_tiled_gb300 as fa
from packed_reference import assert_within
from sink_reference import packed_sinks

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def _loop():
    with open(README, encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    return next(b for b in blocks if "page_update" in b)


def test_block_compiles():
    compile(_loop(), README, "exec")


@pytest.mark.gpu
def test_serving_loop():
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    D, Hq, Hkv, window, sinks, count = 64, 6, 2, 90, 5, 70
    lens = [300, 17, 129]
    B = len(lens)
    gen = torch.Generator().manual_seed(7)
    ns = {}

    def projection(n):
        return torch.randn(n, Hq + 2 * Hkv, D, generator=gen).to(torch.bfloat16).cuda()

    def batches():
        new = torch.tensor(lens, dtype=torch.int32, device="cuda")
        yield sum(lens), new, projection(sum(lens))
        bounds = list(zip(ns["cu"].tolist(), ns["cu"].tolist()[1:]))
        q, k, v = (ns[x].cpu() for x in "qkv")
        r = packed_sinks(q, k, v, bounds, (window, 0), sinks)
        assert_within(ns["o"], r["o"], r["o_tol"], "prompt")
        held = [(k[lo:hi], v[lo:hi]) for lo, hi in bounds]
        for i in range(count):
            new = new + 1
            yield B, new, projection(B)
            for b in range(B):
                kk, vv = (torch.cat((x, ns[y][b:b + 1].cpu())) for x, y in zip(held[b], "kv"))
                held[b] = kk, vv
                j = torch.arange(len(kk))
                j = j[(j >= len(kk) - 1 - window) | (j < sinks)]
                r = ref.attend(ns["q"][b].cpu(), kk[j], vv[j])
                assert_within(ns["o"][b], r["o"], r["o_tol"], f"step {i}, {b}")
                assert_within(ns["lse"][b], r["lse"], r["lse_tol"], f"step {i}, {b}")
        yield 0, torch.zeros_like(new), projection(0)

    pages = 10   # 370, 87 and 199 tokens would take 6 + 2 + 4 = 12
    w = torch.ones(2, D, device="cuda")
    cos, sin = fa.rope_table(400, D)
    ns.update(fa=fa, torch=torch, pages=pages, Hq=Hq, Hkv=Hkv, D=D, B=B, window=window, sinks=sinks,
              batches=batches(), table=torch.full((B, 6), -1, dtype=torch.int32, device="cuda"),
              q_weight=w[0], k_weight=w[1], cos=cos, sin=sin)
    exec(compile(_loop(), README, "exec"), ns)
    assert sorted(ns["free"].tolist()) == list(range(pages))
