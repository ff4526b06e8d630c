"""Values and value scales that are not finite, in each block that some rows see and others do not, for every head size:
rows that see them are not finite in the value's element (all elements of the head, if it is the scale) and may be NaN in the
head's others; everything else keeps its bits."""

import numpy as np
import pytest

from tests.test_gpu_prompt_attention import make, run, tree, visible

pytestmark = pytest.mark.gpu

KINDS = {"bf16": ["inf first", "nan last"], "e4m3": ["nan first", "nan last", "scale inf", "scale nan"]}
SHAPES = {"one tile": ([60], [100]), "two items": ([400], [0]), "one tile, three blocks": ([120], [127]), "two tiles": ([250], [127]),
          "cut, one tile": ([60], [3000]), "cut, two tiles": ([250], [3071])}


@pytest.mark.parametrize("dtype,kind", [(d, k) for d in KINDS for k in KINDS[d]])
@pytest.mark.parametrize("hd", [32, 64, 96, 128])
@pytest.mark.parametrize("shape,draft", [(s, d) for s in SHAPES for d in (False, True) if not d or s != "two items"])
def test_values_that_are_not_finite(dtype, kind, hd, shape, draft):
    import torch
    counts, cached = SHAPES[shape]
    heads, hk, n = 2, 2, counts[0]  # a tile holds 128 tokens
    cs = make(dtype, heads, hk, hd, counts, cached, seed=hd + n, **(dict(mask=tree, words=4) if draft else {}))
    clean = run(cs)
    cache, before = cs["cache"], int(cs["L"][0]) - n
    ends = {before // 128 * 128 + 128 * b + o for b in range(4) for o in (0, 127)}
    for pos in sorted({before, before + n // 2, before + n - 1} | {p for p in ends if before <= p < before + n}):
        at = (int(cs["table"][cs["s"][0], pos // 16]), cs["slot"], 1, 1, pos % 16)
        if kind.startswith("scale"):
            t, i, bad = cache.scales, at, float(kind[6:])
        else:
            e = 0 if kind.endswith("first") else hd - 1
            t = cache.pool if dtype == "bf16" else cache.pool.view(torch.uint8)
            i, bad = at + (e,), (float(kind[:3]) if dtype == "bf16" else 0xFF)
        old = t[i].clone()
        t[i] = bad
        got = run(cs)
        t[i] = old
        see = torch.from_numpy(visible(cs, 0)[:, pos]).cuda()
        assert bool(see.any())
        head, was = got[:n, hd:2 * hd][see], clean[:n, hd:2 * hd][see]
        its = torch.ones(hd, dtype=torch.bool, device="cuda") if kind.startswith("scale") else torch.arange(hd, device="cuda") == e
        assert not bool(head[:, its].isfinite().any()), pos
        assert bool((head.isnan() | (head == was))[:, ~its].all()), pos
        rest = torch.ones_like(got, dtype=torch.bool)
        rest[:n, hd:2 * hd][see] = False
        assert torch.equal(got[rest], clean[rest]), pos


@pytest.mark.parametrize("draft", [False, True])
def test_scores_of_minus_infinity_alone_give_zeros(draft):
    """A row that sees one key, whose score is -inf: as a row that sees nothing."""
    import torch
    cs = make("bf16", 2, 1, 64, [1, 3], [0, 0], **(dict(mask=tree) if draft else {}))
    cs["cache"].pool[int(cs["table"][cs["s"][0], 0]), cs["slot"], 0, 0, 0, 9] = float("-inf")
    clean = run(cs)
    cs["q"].view(-1, 2, 64)[0, 0, 9] = 2.0
    cs["q"].view(-1, 2, 64)[0, 1, 9] = -2.0
    got = run(cs)
    assert (got[0, :64] == 0).all() and got[0, 64:128].isnan().all() and torch.equal(got[1:], clean[1:])
