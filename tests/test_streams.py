"""Calls with stream=: what a call allocates comes from that stream's pool, so that
nothing queued on the caller's stream still uses it, and calls on two streams do not
share a workspace."""
import gc

import pytest
import torch

import __graft_entry__
import exact_attention_blackwell_tiled_gb300 as fa

pytestmark = pytest.mark.gpu

D, HQ, HKV, LENS = 128, 8, 2, [300, 37, 1200]


@pytest.fixture(scope="module", autouse=True)
def _built():
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _packed():
    gen = torch.Generator().manual_seed(6)
    T = sum(LENS)
    q, k, v, do = (torch.randn(T, h, D, generator=gen).to(torch.bfloat16).cuda()
                   for h in (HQ, HKV, HKV, HQ))
    return q, k, v, do, _i32([0, 300, 337, T])


def _cache():
    q, k, v, _, cu = _packed()
    table = torch.arange(3 * 20, dtype=torch.int32, device="cuda").view(3, 20)
    cache = fa.cache4_empty(120, HKV, D, 64)
    fa.cache4_append(cache, k, v, table, _i32([0] * 3), cu)
    return cache, table, _i32(LENS), q[:3].contiguous()


def _segments(stream):
    return [(s["address"], s["address"] + s["total_size"]) for s in torch.cuda.memory_snapshot()
            if s["stream"] == stream.cuda_stream]


def _fresh_stream():
    """A stream whose pool holds nothing."""
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(64):
        side = torch.cuda.Stream()
        if not _segments(side):
            return side
    pytest.skip("every stream's pool is in use")


def _check_pool(call, **given):
    """call(stream, **outputs) twice on a stream of its own: with every output given, what
    is left to allocate (a workspace, where given names none) comes from its pool; with
    none, the outputs do."""
    side = _fresh_stream()
    outputs = call(None)
    torch.cuda.synchronize()
    call(side, **dict(zip(given["names"], outputs)))
    if given["workspace"]:
        assert _segments(side), "the workspace is not the stream's"
    new = call(side)
    mine = _segments(side)
    for t in new:
        assert any(lo <= t.data_ptr() < hi for lo, hi in mine), "an output is not the stream's"
    torch.cuda.synchronize()
    for a, b in zip(outputs, new):
        assert torch.equal(a, b)


def test_packed_calls_allocate_on_their_stream():
    q, k, v, do, cu = _packed()
    _check_pool(lambda s, **kw: fa.fwd_varlen(q, k, v, cu, causal=True, stream=s, **kw),
                names=("out", "lse"), workspace=True)
    o, lse = fa.fwd_varlen(q, k, v, cu, causal=True)
    _check_pool(lambda s, **kw: fa.bwd_varlen(q, k, v, o, do, lse, cu, causal=True,
                                              deterministic=True, stream=s, **kw),
                names=("dq", "dk", "dv"), workspace=True)


def test_cache_calls_allocate_on_their_stream():
    cache, table, n, q = _cache()
    _check_pool(lambda s, **kw: fa.cache4_attend(q, cache, table, n, stream=s, **kw),
                names=("out", "lse"), workspace=True)
    _check_pool(lambda s, **kw: fa.cache4_read(cache, table, None, n, 64, D, stream=s, **kw),
                names=("k", "v"), workspace=False)
    w = torch.rand(3, HKV, 1200, device="cuda")
    _check_pool(lambda s, **kw: fa.cache4_evict(cache, table, n, w, table + 60, D, 100, 10,
                                                stream=s, **kw),
                names=("src", "weights_out", "lens_out"), workspace=False)
    assert fa.cache4_status() == fa.FA_OK


def _dense():
    gen = torch.Generator().manual_seed(9)
    return [torch.randn(2, h, 700, D, generator=gen).to(torch.bfloat16).cuda()
            for h in (HQ, HKV, HKV, HQ)]


def test_dense_calls_allocate_on_their_stream():
    q, k, v, do = _dense()
    o, lse = fa.fwd(q, k, v, causal=True)
    _check_pool(lambda s, **kw: fa.fwd(q, k, v, causal=True, stream=s, **kw), names=("out", "lse"),
                workspace=False)
    _check_pool(lambda s, **kw: fa.fwd(q, k, v, n_splits=3, stream=s, **kw), names=("out", "lse"),
                workspace=True)
    _check_pool(lambda s, **kw: fa.bwd(q, k, v, o, do, lse, causal=True, deterministic=True,
                                       stream=s, **kw),
                names=("dq", "dk", "dv"), workspace=True)
    parts = torch.randn(3, 500, D, device="cuda"), torch.randn(3, 500, device="cuda")
    _check_pool(lambda s, **kw: fa.lse_merge(*parts, stream=s, **kw), names=("out", "lse"),
                workspace=False)
    x = torch.linspace(-3, 3, 1000, device="cuda")
    _check_pool(lambda s: (fa.exp2_test(x, 0, stream=s),), names=(), workspace=True)


def test_dense_calls_in_turn_on_two_streams():
    q, k, v, do = _dense()
    o, lse = fa.fwd(q, k, v, causal=True)

    def calls(stream):
        return (*fa.fwd(q, k, v, causal=True, stream=stream), *fa.fwd(q, k, v, n_splits=3, stream=stream),
                *fa.bwd(q, k, v, o, do, lse, causal=True, deterministic=True, stream=stream))

    want = calls(None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(10):
        got += [calls(None), calls(side)]
    torch.cuda.synchronize()
    for run in got:
        for a, b in zip(want, run):
            assert torch.equal(a, b)


def test_wait_test_on_another_stream():
    """The status is set, written and read on the stream of the call."""
    side = torch.cuda.Stream()
    flag = torch.ones(1, dtype=torch.int32, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    assert fa.wait_test(0, flag, stream=side) == fa.FA_OK


def test_calls_in_turn_on_two_streams():
    """No synchronisation between a call on the current stream and the next on another:
    each call frees its workspace as soon as it is launched."""
    q, k, v, do, cu = _packed()
    cache, table, n, q1 = _cache()

    def calls(stream):
        o, lse = fa.fwd_varlen(q, k, v, cu, causal=True, stream=stream)
        grads = fa.bwd_varlen(q, k, v, want[0], do, want[1], cu, causal=True, deterministic=True,
                              stream=stream) if want else ()
        return (o, lse, *grads, *fa.cache4_attend(q1, cache, table, n, stream=stream))

    want = None
    first = calls(None)
    want = first[:2]
    want = calls(None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        got += [calls(None), calls(side)]
    torch.cuda.synchronize()
    for run in got:
        for a, b in zip(want, run):
            assert torch.equal(a, b)


def test_threads_with_streams_of_their_own():
    """Four threads, each on a stream of its own, some of them by stream=."""
    import threading

    q, k, v, do, cu = _packed()
    cache, table, n, q1 = _cache()
    o, lse = fa.fwd_varlen(q, k, v, cu, causal=True)

    def calls(stream=None):
        grads = fa.bwd_varlen(q, k, v, o, do, lse, cu, causal=True, deterministic=True, stream=stream)
        return (*fa.fwd_varlen(q, k, v, cu, causal=True, stream=stream), *grads,
                *fa.cache4_attend(q1, cache, table, n, stream=stream),
                *fa.cache4_read(cache, table, None, n, 1200, D, stream=stream))

    want = calls()
    torch.cuda.synchronize()
    failed = []

    def run(i):
        try:
            side = torch.cuda.Stream()
            for _ in range(15):
                if i % 2:
                    got = calls(side)
                else:
                    with torch.cuda.stream(side):
                        got = calls()
                side.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(want, got)):
                    failed.append((i, "different"))
        except Exception as e:  # reported by the main thread
            failed.append((i, repr(e)))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert fa.fwd_status() == fa.FA_OK and fa.cache4_status() == fa.FA_OK
