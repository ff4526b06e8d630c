"""slot_base + depth beyond 32 bits names no slot."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("base,depth", [(-2 ** 31, -2 ** 31), (2 ** 31 - 1, 2 ** 31 - 1), (-2 ** 31, 2 ** 31 - 1), (2 ** 31 - 1, 1)])
def test_sum_of_slot_base_and_depth(base, depth):
    import torch
    from continuous_depth_batching_gb300 import ops
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    pool = torch.full((40, 2, 2, 4, 16, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    cache = ops.PagedCache(pool, table)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    w, at = ops.CacheWriter(cache, 8), ops.DecodeAttention(cache, 8, 2)
    q = torch.full((2, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    w(torch.zeros(2, 1024, device="cuda"), i32(0, 1), i32(5, 300), i32(depth, depth), slot_base=base, q_out=q)
    assert int(w.status.item()) == 2 and bool((q == 3).all()) and bool((pool == 7).all())
    out = torch.full_like(q, 5.0)
    at(q, i32(0, 1), i32(5, 300), i32(depth, depth), slot_base=base, out=out)
    assert int(at.status.item()) == 2 and bool((out == 5).all())
