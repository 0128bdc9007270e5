"""README's serving loop where sequences end one by one, and where the prompts have as many
tokens as there are sequences."""
import pytest
import torch

import __graft_entry__
import cache4_reference as ref
import exact_attention_blackwell_tiled_gb300 as fa
from packed_reference import assert_within
from sink_reference import packed_sinks
from test_readme_serving import README, _loop


@pytest.mark.gpu
@pytest.mark.parametrize("padded", [False, True])  # a row for every sequence in every step
@pytest.mark.parametrize("lens,ends,count", [
    ([300, 17, 129], [40, 20, 60], 60),      # the second one ends first, then the first
    ([300, 17, 129], [60, 60, 1], 60),       # the last one after a single token
    ([2, 0], [30, 30], 30),                  # prompts of two tokens in all, for two sequences
    ([1, 1, 1, 1], [5, 100, 7, 9], 100),     # one is left on its own
])
def test_sequences_that_end(lens, ends, count, padded):
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    D, Hq, Hkv, window, sinks = 64, 6, 2, 90, 5
    B = len(lens)
    gen = torch.Generator().manual_seed(sum(lens))
    ns = {}

    def projection(n):
        return torch.randn(n, Hq + 2 * Hkv, D, generator=gen).to(torch.bfloat16).cuda()

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def batches():
        yield sum(lens), i32(lens), projection(sum(lens))
        bounds = list(zip(ns["cu"].tolist(), ns["cu"].tolist()[1:]))
        q, k, v = (ns[x].cpu() for x in "qkv")
        r = packed_sinks(q, k, v, bounds, (window, 0), sinks)
        assert_within(ns["o"], r["o"], r["o_tol"], "prompt")
        assert_within(ns["lse"], r["lse"], r["lse_tol"], "prompt lse")
        held = [(k[lo:hi], v[lo:hi]) for lo, hi in bounds]
        for i in range(count):
            going = [b for b in range(B) if i < ends[b]]
            new = [len(held[b][0]) + 1 if b in going else 0 for b in range(B)]
            T = B if padded else len(going)
            yield T, i32(new), projection(T)
            assert ns["o"].shape[0] == T
            for row, b in enumerate(going):
                held[b] = tuple(torch.cat((x, ns[y][row:row + 1].cpu())) for x, y in zip(held[b], "kv"))
                kk, vv = held[b]
                j = torch.arange(len(kk))
                j = j[(j >= len(kk) - 1 - window) | (j < sinks)]
                r = ref.attend(ns["q"][row].cpu(), kk[j], vv[j])
                assert_within(ns["o"][row], r["o"], r["o_tol"], f"step {i}, {b}")
                assert_within(ns["lse"][row], r["lse"], r["lse_tol"], f"step {i}, {b}")
        yield 0, i32([0] * B), projection(0)

    pages, w = 12, torch.ones(2, D, device="cuda")
    cos, sin = fa.rope_table(400, D)
    ns.update(fa=fa, torch=torch, pages=pages, Hq=Hq, Hkv=Hkv, D=D, B=B, window=window, sinks=sinks,
              batches=batches(), table=torch.full((B, 6), -1, dtype=torch.int32, device="cuda"),
              q_weight=w[0], k_weight=w[1], cos=cos, sin=sin)
    exec(compile(_loop(), README, "exec"), ns)
    assert sorted(ns["free"].tolist()) == list(range(pages))
