"""Accepted paths in blocks from 2^27 on, where 16 * block passes 32 bits."""

import pytest

pytestmark = pytest.mark.gpu


def test_paths_in_blocks_behind_2_27():
    import torch
    from continuous_depth_batching_gb300 import ops
    torch.cuda.empty_cache()
    blocks, last = (1 << 27) + 64, 80
    cell = 2 * 16 * 32  # codes of a block: K and V of one head of 32
    if torch.cuda.mem_get_info()[0] < blocks * (cell + 128) + (8 << 30):
        pytest.skip("the pool does not fit")
    pool = torch.empty(blocks, 1, 2, 1, 16, 32, dtype=torch.uint8, device="cuda")
    scales = torch.empty(blocks, 1, 2, 1, 16, device="cuda")
    pool[-last:].random_(0, 256)
    scales[-last:].normal_()
    # sequence 0: the last blocks, on both sides of 2^27; sequence 1: blocks on the other side of it
    table = torch.stack([blocks - 1 - torch.arange(6), (1 << 27) - 3 + torch.arange(6)]).to(torch.int32).cuda()
    at = lambda s, p: (int(table[s, p // 16]), slice(None), slice(None), slice(None), p % 16)  # noqa: E731
    base, paths = (20, 14), ([0, 3, 9, 30, 44], [2, 17, 35, 60, 61])
    shift = blocks - last
    want, want_s = pool[shift:].clone(), scales[shift:].clone()
    for s in range(2):
        for k, p in enumerate(paths[s]):
            a, b = at(s, base[s] + p), at(s, base[s] + k)
            for of in (want, want_s):
                of[(b[0] - shift,) + b[1:]] = of[(a[0] - shift,) + a[1:]].clone()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    keeper = ops.PathKeeper(ops.PagedCache(pool.view(torch.float8_e4m3fn), table, scales))
    keeper(i32(base), i32(paths), i32([5, 5]))
    keeper.check()
    assert torch.equal(pool[shift:], want) and torch.equal(scales[shift:], want_s)
    del pool, scales, keeper
    torch.cuda.empty_cache()
