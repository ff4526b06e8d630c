"""Operators called on other streams than the one they were made on.

torch.cuda._sleep holds a stream up for about half a second, so that what is not ordered shows."""

import gc

import pytest

pytestmark = pytest.mark.gpu

CYCLES = 1_000_000_000


def attention(rows=4):
    import torch
    from continuous_depth_batching_gb300 import ops
    table = torch.arange(rows * 4, dtype=torch.int32, device="cuda").view(rows, 4)
    cache = ops.PagedCache(torch.randn(rows * 4, 1, 2, 4, 16, 64, device="cuda").bfloat16(), table)
    q = torch.randn(rows, 8 * 64, device="cuda").bfloat16()
    seq = torch.arange(rows, dtype=torch.int32, device="cuda")
    return ops, cache, q, seq, torch.full((rows,), 50, dtype=torch.int32, device="cuda"), torch.zeros_like(q)


def freed_for(numels, dtypes):
    """Addresses of new tensors of the sizes, as many as would take up what was just freed."""
    import torch
    keep = [torch.empty(n, dtype=d, device="cuda") for n, d in zip(numels, dtypes) for _ in range(64)]
    return {t.data_ptr() for t in keep}


def test_a_dropped_object_keeps_its_memory_until_its_calls_are_done():
    import torch
    ops, cache, q, seq, pos, out = attention()
    side = torch.cuda.Stream()
    qkv, x, u, t = torch.zeros(4, 16 * 64, device="cuda"), torch.zeros(4, 1000, device="cuda"), torch.zeros(4, device="cuda"), torch.ones(4, device="cuda")
    for held in (0, CYCLES):  # the first calls load the kernels
        at, w, s = ops.DecodeAttention(cache, 8, 4), ops.CacheWriter(cache, 8), ops.Sampler(4, 1000)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(held)
            at(q, seq, pos, out=out)
            w(qkv, seq, pos, q_out=out)
            s(x, u, t)
    mine = [at.workspace, at.status, w.status, s.token, s.logprob]
    old, sizes, types = {m.data_ptr() for m in mine}, [m.numel() for m in mine], [m.dtype for m in mine]
    del at, w, s, mine
    gc.collect()
    new = freed_for(sizes, types)
    assert not side.query(), "the calls were done too early to show anything"
    assert not old & new
    torch.cuda.synchronize()


def test_check_waits_for_calls_on_any_stream():
    import torch
    ops, cache, q, seq, pos, out = attention()
    at = ops.DecodeAttention(cache, 8, 4)
    w = ops.CacheWriter(cache, 8)
    bad, qkv = torch.full_like(seq, 99), torch.zeros(4, 16 * 64, device="cuda")
    at(q, seq, pos, out=out)
    w(qkv, seq, pos, q_out=out)
    at.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
        at(q, bad, pos, out=out)
        w(qkv, bad, pos, q_out=out)
    for op in (at, w):
        with pytest.raises(ops.CdbError, match="sequence or position"):
            op.check()
        op.check()


def test_an_object_is_ready_on_another_stream():
    # Its status is cleared on the stream it is made on, here behind other work.
    import torch
    ops, cache, q, seq, pos, out = attention()
    bad = torch.full_like(seq, 99)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    at = ops.DecodeAttention(cache, 8, 4)
    with torch.cuda.stream(side):
        at(q, bad, pos, out=out)
    side.synchronize()
    with pytest.raises(ops.CdbError, match="sequence or position"):
        at.check()


def test_streams_in_turn_and_in_a_capture():
    import torch
    ops, cache, q, seq, pos, out = attention()
    at = ops.DecodeAttention(cache, 8, 4)
    want = at(q, seq, pos)
    sides = [torch.cuda.Stream() for _ in range(3)]
    for i in range(9):
        s = sides[i % 3]
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = at(q, seq, pos)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(got, want)
    assert len(at._streams) == 4
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):  # on a stream that the object does not know
        at(q, seq, pos, out=out)
    g.replay()
    assert torch.equal(out, want)
    at.check()
