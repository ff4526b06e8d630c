"""Prompt and draft attention with a row_start that descends: reported, and nothing outside the call's own rows and
workspace is touched, however many tiles the overlapping requests would have."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

GUARD = 1 << 22  # bytes behind the workspace


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("requests", [2, 30, 32, 33, 100, 420])  # up to 32 requests are found by one warp
@pytest.mark.parametrize("skip", [False, True])  # the requests whose rows descend are skipped ones
def test_rows_that_descend(draft, requests, skip):
    import torch
    from continuous_depth_batching_gb300 import ops
    from continuous_depth_batching_gb300.binding import CdbError
    rows, pages, hd = 256 if draft else 2560, 40, 64
    pool = torch.randn(pages, 1, 2, 1, 16, hd, device="cuda").bfloat16()
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(requests, pages).contiguous()
    cache = ops.PagedCache(pool, table)
    op = ops.DraftAttention(cache, 1, rows, requests, 256) if draft else ops.PromptAttention(cache, 1, rows, requests)
    # a workspace of the same size with a guard behind it
    size = op.args.workspace_bytes
    held = torch.full((size + GUARD + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    base = (held.data_ptr() + 255) // 256 * 256
    op.args.workspace = base
    guard = held[base - held.data_ptr() + size:]
    q = torch.randn(rows, hd, device="cuda").bfloat16()
    out = torch.full((rows + 8, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    visible = (torch.full((rows, 4), -1, dtype=torch.int64, device="cuda"),) if draft else ()
    lens = torch.full((requests,), 16 * pages, dtype=torch.int32, device="cuda")
    seq = np.arange(requests)
    if skip:
        seq[1::2] = -1
    seq = torch.tensor(seq, dtype=torch.int32, device="cuda")
    # 0, rows, 0, rows, ..: every other request has all rows
    start = torch.tensor([rows * (i % 2) for i in range(requests + 1)], dtype=torch.int32, device="cuda")
    with pytest.raises(CdbError, match="sequence"):
        op(q, start, lens, *visible, seq=seq, out=out)
        op.check()
    assert (guard == 0x5A).all() and (out[rows:] == 7).all()
    # the object serves its next call
    start = torch.tensor([min(i * 7, rows) for i in range(requests + 1)], dtype=torch.int32, device="cuda")
    n = int(start[-1])
    op(q, start, lens, *visible, seq=seq, out=out)
    op.check()
    assert (guard == 0x5A).all()
    if draft:
        return
    k, v = pool[:, 0, 0, 0].reshape(-1, hd).double(), pool[:, 0, 1, 0].reshape(-1, hd).double()
    x = q[:n].double() @ k.T * hd ** -0.5
    bounds = start.tolist()
    for i in range(0, requests, 2):
        a, b = bounds[i], bounds[i + 1]
        see = torch.ones(b - a, 16 * pages, dtype=torch.bool, device="cuda").tril(16 * pages - (b - a))
        o = torch.softmax(torch.where(see, x[a:b], -torch.inf), -1) @ v
        S = (q[a:b].double().abs() @ k.T.abs()).amax() * hd ** -0.5 if b > a else 0.0
        tol = 2.0 ** -8 * o.abs() + v.abs().max() * (2 * (hd * 2.0 ** -23 * S + 2.0 ** -20 + 2.0 ** -17) + 80 * 2.0 ** -23)
        assert ((out[a:b].double() - o).abs() <= tol).all()
