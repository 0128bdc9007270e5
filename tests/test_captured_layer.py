"""A training step of norms, rotation and attention under a window with sinks, captured into a
CUDA graph with its backward pass and replayed on other inputs, positions and boundaries."""
import pytest
import torch

import __graft_entry__
import exact_attention_blackwell_tiled_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [2, 40])
def test_captured_training_step(D, B):
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    T, Hq, Hkv = 600, 4, 2
    gen = torch.Generator().manual_seed(D)
    cos, sin = fa.rope_table(T, D)

    def inputs():
        x = torch.randn(T, Hq + 2 * Hkv, D, generator=gen).to(torch.bfloat16)
        w = 1 + torch.rand(2, D, generator=gen)
        cuts = torch.randint(0, T + 1, (B + 1,), generator=gen).sort().values.to(torch.int32)
        pos = torch.full((T,), -1, dtype=torch.int32)
        for lo, hi in zip(cuts[:-1].tolist(), cuts[1:].tolist()):
            pos[lo:hi] = torch.arange(hi - lo)
        do = torch.randn(T, Hq, D, generator=gen).to(torch.bfloat16)
        return [t.cuda() for t in (x, w, cuts, pos, do)]

    def step(x, w, cuts, pos, do):
        q, k = fa.norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], w[0], w[1], cos, sin, pos)
        o = fa.attention_varlen(q, k, x[:, Hq + Hkv:], cuts, window=(50, 0), sinks=4, deterministic=True)
        dx, dw = torch.autograd.grad(o, (x, w), do)
        return o.detach(), dx, dw

    held = inputs()
    x, w = (t.requires_grad_() for t in held[:2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*held)
    for _ in range(4):
        new = inputs()
        with torch.no_grad():
            for a, b in zip(held, new):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step(*(t.requires_grad_() for t in new[:2]), *new[2:])
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert fa.fwd_status() == fa.FA_OK
