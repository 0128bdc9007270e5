"""The gradients come from a kernel without a derivative: differentiating them again
raises, instead of taking them for constants."""
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


def _refuses(attend, *shapes):
    gen = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(*s, generator=gen).to(torch.bfloat16).cuda().requires_grad_() for s in shapes)
    o = attend(q, k, v)
    dq, = torch.autograd.grad(o.float().pow(2).sum(), q, create_graph=True)
    # a penalty on the gradient beside the loss itself: its share would be left out
    loss = o.float().sum() + dq.float().pow(2).sum()
    with pytest.raises(RuntimeError):
        loss.backward()


def test_attention_varlen():
    cu = torch.tensor([0, 30, 70], dtype=torch.int32, device="cuda")
    _refuses(lambda q, k, v: fa.attention_varlen(q, k, v, cu, causal=True), (70, 4, 64), (70, 2, 64),
             (70, 2, 64))


def test_attention():
    _refuses(lambda q, k, v: fa.attention(q, k, v, causal=True), (1, 4, 70, 64), (1, 2, 70, 64),
             (1, 2, 70, 64))
