"""Attention of packed prompts and of drafts (include/cdb_ops.h) against float64 restatements.

Everything that no row sees (other slots, pages and positions behind a sequence's end) holds NaN; rows of `out` that
are not a request's hold a sentinel.

Tolerances.  A score is a sum of head_dim exact products, accumulated in fp32 with at most 2^-23 per step of
S = |scale| * sum |q k|; a weight e^s is then off by that (as an exponent) plus 2^-20 for the exponential and its
16-bit form: two numbers within 2^-17 (bf16 cache), or one of weight times value scale within 2^-11 of it or 2^-33
of the largest (e4m3 cache); weights enter twice (numerator, sum).  With an e4m3 cache an element of a query below
2^-8 of the head's largest one may be off by 2^-17 of that.
The weighted sum adds 2^-23 of max |v| per accumulation step (16 keys each) and per joined range.  A bf16 output
adds 2^-8 of its value.
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

SENTINEL = 7.0


def make(dtype, heads, hk, hd, counts, cached, slots=2, slot=1, seed=0, pad=3, extra_pages=3, mask=None, words=1):
    """A call: packed requests of `counts` rows behind `cached` tokens, shuffled pages and sequences."""
    import torch
    from continuous_depth_batching_gb300 import ops
    rng = np.random.default_rng(seed)
    counts, cached = np.asarray(counts), np.asarray(cached)
    n = len(counts)
    lens = np.maximum(counts + cached, 0)
    need = (lens + 15) // 16
    maxb = int(need.max()) + 2
    blocks = int(need.sum()) + extra_pages
    perm = rng.permutation(blocks)
    table = np.full((n, maxb), -1, dtype=np.int32)
    at = 0
    seq = rng.permutation(n)
    for i in range(n):
        table[seq[i], :need[i]] = perm[at:at + need[i]]
        at += need[i]
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (blocks, slots, 2, hk, 16, hd)
    x = torch.randn(shape, generator=g, device="cuda") * (1 + 4 * torch.rand(shape[:-1], generator=g, device="cuda"))[..., None]
    if dtype == "bf16":
        pool, scales = x.bfloat16(), None
        vals = pool.double()
    else:
        scales = (x.abs().amax(-1) / 448).clamp_min(2.0 ** -126)
        pool = (x / scales[..., None]).to(torch.float8_e4m3fn)
        vals = pool.double() * scales.double()[..., None]
    used = torch.zeros(blocks, slots, 16, dtype=torch.bool)
    for i in range(n):
        j = np.arange(lens[i])
        used[table[seq[i], j // 16], slot, j % 16] = True
    hide = ~used.cuda()
    pool.view(torch.uint8).view(*pool.shape[:-1], -1).masked_fill_(hide[:, :, None, None, :, None], 0xFF)  # NaN
    if scales is not None:
        scales.masked_fill_(hide[:, :, None, None, :], float("nan"))
    start = np.concatenate([[0], np.cumsum(counts)])
    rows = int(start[-1]) + pad
    q = (torch.randn(rows, heads * hd, generator=g, device="cuda") * 1.5).bfloat16()
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
    cs = dict(cache=ops.PagedCache(pool, i32(table), scales), vals=vals, q=q, seq=i32(seq), lens=i32(lens), start=i32(start),
              counts=counts, L=lens, table=table, s=seq, slot=slot, heads=heads, hk=hk, hd=hd, dtype=dtype, mask=None,
              max_ctx=min(16 * maxb, int(lens.max()) + 5))
    if mask is not None:
        bits = np.zeros((rows, words), dtype=np.uint64)
        cs["mask"] = []
        for i in range(n):
            m = mask(rng, int(counts[i]))  # [count, count] truth values
            cs["mask"].append(m)
            for u in range(int(counts[i])):
                bits[start[i]:start[i + 1], u // 64] |= m[:, u].astype(np.uint64) << np.uint64(u % 64)
            if counts[i] % 64:  # bits of rows that the request does not have
                bits[start[i]:start[i + 1], counts[i] // 64] |= np.uint64((1 << 64) - (1 << int(counts[i] % 64)))
        cs["visible"], cs["words"] = torch.from_numpy(bits.view(np.int64)).cuda(), words
    return cs


def visible(cs, i):
    c, length = int(cs["counts"][i]), int(cs["L"][i])
    before = length - c
    see = np.zeros((c, length), dtype=bool)
    if cs["mask"] is None:
        for t in range(c):
            see[t, :max(0, before + t + 1)] = True
    else:
        see[:, :max(0, before)] = True
        see[:, max(0, before):] = cs["mask"][i][:, max(0, -before):]
    return see


def expected(cs, i, scale):
    """(output [count, heads, hd] in float64, tolerance) of request i."""
    import torch
    heads, hk, hd = cs["heads"], cs["hk"], cs["hd"]
    length, c = int(cs["L"][i]), int(cs["counts"][i])
    j = np.arange(length)
    blk, off = torch.from_numpy(cs["table"][cs["s"][i], j // 16]).long().cuda(), torch.from_numpy(j % 16).cuda()
    k = cs["vals"][blk, cs["slot"], 0, :, off]  # [length, hk, hd]
    v = cs["vals"][blk, cs["slot"], 1, :, off]
    r0 = int(cs["start"][i])
    q = cs["q"][r0:r0 + c].double().view(c, hk, heads // hk, hd)
    see = torch.from_numpy(visible(cs, i)).cuda()
    x = torch.einsum("tkgd,lkd->tkgl", q, k) * scale
    x = torch.where(see[:, None, None], x, -torch.inf)
    p = torch.nan_to_num(torch.softmax(x, -1))
    v0 = torch.where(see.any(0)[:, None, None], v, 0.0)  # seen by nobody: may be anything
    o = torch.einsum("tkgl,lkd->tkgd", p, v0)
    seen = see.any(1)
    o = torch.where(seen[:, None, None, None], o, 0.0)
    if length == 0 or not bool(seen.any()):
        return o.reshape(c, heads, hd), torch.full((c, heads, hd), 1e-30, dtype=torch.float64, device="cuda")
    fin = torch.nan_to_num(k, 0, 0, 0)
    big = torch.where(see.any(0)[:, None, None], fin.abs(), 0.0)
    S = torch.einsum("tkgd,lkd->tkgl", q.abs(), big).amax() * abs(scale)
    # a row's own largest value
    vm = torch.where(see[..., None], torch.nan_to_num(v, 0, 0, 0).abs().amax(-1)[None], 0.0).amax(1)  # [c, hk]
    steps = 16 + length / 16 + length / 64
    w = 2.0 ** -17
    if cs["dtype"] == "e4m3":
        top = q.abs().amax(-1, keepdim=True)
        small = torch.einsum("tkgd,lkd->tkgl", (q.abs() < 2.0 ** -8 * top).double() * top, big).amax() * abs(scale)
        w = 2.0 ** -11 + length * 2.0 ** -33 + 2.0 ** -17 * small
    tol = 2.0 ** -8 * o.abs() + vm[:, :, None, None] * (2 * (hd * 2.0 ** -23 * S + 2.0 ** -20 + w) + steps * 2.0 ** -23) + 1e-30
    return o.reshape(c, heads, hd), tol.reshape(c, heads, hd)


def run(cs, scale=None, out=None, max_requests=None, op=None):
    import torch
    from continuous_depth_batching_gb300 import ops
    rows, n = cs["q"].shape[0], len(cs["counts"])
    if op is None:
        args = cs["cache"], cs["heads"], rows, max_requests or n
        op = ops.PromptAttention(*args, cs["max_ctx"], scale) if cs["mask"] is None else \
            ops.DraftAttention(*args, 64 * cs["words"], cs["max_ctx"], scale)
    if out is None:
        out = torch.full((rows, cs["heads"] * cs["hd"] + 8), SENTINEL, dtype=torch.bfloat16, device="cuda")
    mask = () if cs["mask"] is None else (cs["visible"],)
    assert op(cs["q"], cs["start"], cs["lens"], *mask, seq=cs["seq"], slot=cs["slot"], out=out) is out
    op.check()
    return out


def check(cs, scale=None, out=None, requests=None):
    out = run(cs, scale, out)
    width = cs["heads"] * cs["hd"]
    assert (out[:, width:] == SENTINEL).all()
    assert (out[int(cs["start"][-1]):] == SENTINEL).all()
    for i in requests if requests is not None else range(len(cs["counts"])):
        if not cs["counts"][i]:
            continue
        o, tol = expected(cs, i, cs["hd"] ** -0.5 if scale is None else scale)
        r0 = int(cs["start"][i])
        got = out[r0:r0 + int(cs["counts"][i]), :width].double().view(o.shape)
        err = (got - o).abs()
        assert not got.isnan().any() and (err <= tol).all(), (i, float((err / tol).max()))
    return out


HEADS = [(16, 16, 128), (8, 2, 128), (7, 7, 32), (14, 2, 64), (10, 2, 96), (128, 1, 64)]
LENGTHS = {
    "one token": ([1], [0]),
    "a token behind a page": ([1], [16]),
    "short": ([5, 1, 0, 16, 17], [0, 3, 40, 0, 127]),
    "around a block": ([128, 127, 129, 1, 2], [0, 0, 0, 127, 128]),
    "behind a block": ([3, 64, 65], [256, 255, 1]),
    "two tiles": ([300, 256, 257], [0, 0, 130]),
    "long": ([700, 30], [900, 2000]),
    "before the start": ([9, 4], [-4, 0]),
}


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,hk,hd", HEADS)
@pytest.mark.parametrize("which", LENGTHS)
def test_prompts(dtype, heads, hk, hd, which):
    counts, cached = LENGTHS[which]
    check(make(dtype, heads, hk, hd, counts, cached, seed=len(which) + hd))


def tree(rng, n):
    m = np.zeros((n, n), dtype=bool)
    for u in range(n):
        p = int(rng.integers(-1, u)) if u else -1
        if p >= 0:
            m[u] = m[p]
        m[u, u] = True
    return m


def scattered(rng, n):
    """Any bits, rows without any among them."""
    m = rng.random((n, n)) < 0.4
    m[rng.random(n) < 0.3] = False
    return m


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,hk,hd", HEADS)
@pytest.mark.parametrize("mask,counts,cached,words", [
    (tree, [1], [0], 1), (tree, [8, 64, 1, 0, 33], [1000, 63, 5, 9, 128], 1), (tree, [256, 100, 3], [130, 0, 700], 4),
    (scattered, [9, 60, 64], [0, 0, 77], 1), (scattered, [130, 31, 5], [0, 250, -2], 3)])
def test_drafts(dtype, heads, hk, hd, mask, counts, cached, words):
    check(make(dtype, heads, hk, hd, counts, cached, seed=sum(counts) + hd, mask=mask, words=words))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0, 1e-3])
def test_scales(dtype, scale):
    check(make(dtype, 8, 2, 64, [40, 200], [100, 0]), scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_many_requests_and_strided_rows(dtype):
    import torch
    rng = np.random.default_rng(5)
    counts = rng.integers(0, 9, 700)
    cs = make(dtype, 4, 2, 64, counts, rng.integers(0, 200, 700), seed=9)
    wide = torch.zeros(cs["q"].shape[0], 3 * 256, dtype=torch.bfloat16, device="cuda")
    wide[:, 256:512] = cs["q"]
    cs["q"] = wide[:, 256:512]
    check(cs, requests=range(0, 700, 13))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("draft", [False, True])
def test_cut_keys(dtype, draft):
    """Few rows behind a long context: the keys are cut among CTAs and joined."""
    kw = dict(mask=tree) if draft else {}
    check(make(dtype, 8, 2, 128, [20, 1, 64], [20000, 3, 5000], seed=3, **kw))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,hk,hd", [(16, 16, 128), (32, 16, 96), (16, 16, 64), (8, 8, 32)])
@pytest.mark.parametrize("most", [3, 200])
def test_long_contexts_that_are_not_cut(dtype, heads, hk, hd, most):
    """Enough requests for the GPU: a CTA takes every block of a request's keys, for one tile or two."""
    rng = np.random.default_rng(hd + most)
    n = 700 // hk
    cs = make(dtype, heads, hk, hd, rng.integers(1, most, n), rng.integers(0, 2500, n), seed=most)
    check(cs, requests=range(0, n, 3))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("draft", [False, True])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(dtype, draft):
    import torch
    from continuous_depth_batching_gb300 import ops
    heads, hk, hd = 4, 2, 64
    for counts, cached, bad_row in (([50], [0], 20), ([64], [100], 63), ([64], [256], 0), ([200], [0], 130)):
        if draft and counts[0] > 64:
            continue
        cs = make(dtype, heads, hk, hd, counts, cached, seed=bad_row, **(dict(mask=tree) if draft else {}))
        pos = int(cs["L"][0]) - counts[0] + bad_row
        blk, off = cs["table"][cs["s"][0], pos // 16], pos % 16
        clean = run(cs)
        cache = cs["cache"]
        if dtype == "bf16":
            cache.pool[blk, cs["slot"], 0, 0, off, 3] = float("inf")   # a key
            cache.pool[blk, cs["slot"], 1, 1, off, 7] = float("nan")   # a value of the other head
        else:
            cache.scales[blk, cs["slot"], 0, 0, off] = float("nan")
            cache.pool.view(torch.uint8)[blk, cs["slot"], 1, 1, off, 7] = 0x7F
        got = run(cs)
        see = torch.from_numpy(visible(cs, 0)[:, pos]).cuda()
        width = heads * hd
        hidden = torch.cat([~see, torch.ones(got.shape[0] - counts[0], dtype=torch.bool, device="cuda")])
        assert torch.equal(got[hidden], clean[hidden])
        half = got[:counts[0], :width][see].float()
        assert half[:, width // 2:].isnan().all()  # the value's rows
        # The key: a score of +inf or NaN makes its row of the head NaN, one of -inf has no weight.
        q = cs["q"][:counts[0]][see].view(-1, heads, hd)[:, :heads // hk, 3]
        want = q >= 0 if dtype == "bf16" else torch.ones_like(q, dtype=torch.bool)
        assert torch.equal(half.view(-1, heads, hd)[:, :heads // hk].isnan(), want[..., None].expand(-1, -1, hd))


def test_weights_keep_their_bits_beside_loud_values():
    """A loud value without weight, and a heavy key with a value near zero, take no bits from the others (e4m3)."""
    import torch
    cs = make("e4m3", 4, 2, 64, [30, 90], [300, 10], seed=11)
    cache, vals = cs["cache"], cs["vals"]
    for i, (p, f) in enumerate(((17, 2.0 ** 60), (40, 2.0 ** -60))):
        for r in range(2):
            blk = int(cs["table"][cs["s"][r], p // 16])
            cache.scales[blk, 1, 1, :, p % 16] *= f
            vals[blk, 1, 1, :, p % 16] *= f
    check(cs)


@pytest.mark.parametrize("draft", [False, True])
def test_bad_requests_are_reported_and_skipped(draft):
    import torch
    from continuous_depth_batching_gb300 import ops
    from continuous_depth_batching_gb300.binding import CdbError
    cs = make("bf16", 4, 2, 64, [10, 20, 30], [5, 50, 7], **(dict(mask=tree) if draft else {}))
    good = run(cs)

    def attempt(match, **kw):
        c = dict(cs, **kw)
        out = torch.full_like(good, SENTINEL)
        with pytest.raises(CdbError, match=match):
            run(c, out=out)
        return out

    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    seq = cs["seq"].tolist()
    out = attempt("sequence", seq=i32([seq[0], 3, seq[2]]))
    assert torch.equal(out[:10], good[:10]) and (out[10:30] == SENTINEL).all() and torch.equal(out[30:60], good[30:60])
    lens = cs["lens"].tolist()
    for bad in (-1, cs["max_ctx"] + 1):
        out = attempt("sequence", lens=i32([lens[0], bad, lens[2]]))
        assert torch.equal(out[:10], good[:10]) and (out[10:30] == SENTINEL).all() and torch.equal(out[30:60], good[30:60])
    attempt("sequence", start=i32([0, 10, 30, 64]))  # past the rows
    attempt("sequence", start=i32([0, 10, 5, 60]))
    attempt("sequence", start=i32([-5, 10, 30, 60]))
    # a sequence below 0 is skipped without a report
    out = run(dict(cs, seq=i32([seq[0], -1, seq[2]])), out=torch.full_like(good, SENTINEL))
    assert torch.equal(out[:10], good[:10]) and (out[10:30] == SENTINEL).all() and torch.equal(out[30:60], good[30:60])
    # a block out of range
    table = cs["cache"].block_table
    at = (seq[1], 1)
    keep = int(table[at])
    for bad in (-1, 10 ** 6):
        table[at] = bad
        attempt("block table")
        table[at] = keep


def test_arguments_are_refused():
    import torch
    from continuous_depth_batching_gb300 import ops
    cs = make("bf16", 4, 2, 64, [10, 20], [5, 50], mask=tree)
    rows = cs["q"].shape[0]
    p = ops.PromptAttention(cs["cache"], 4, rows, 2)
    d = ops.DraftAttention(cs["cache"], 4, rows, 2, 64)
    q, start, lens, vis = cs["q"], cs["start"], cs["lens"], cs["visible"]
    more = torch.zeros(rows + 1, 256, dtype=torch.bfloat16, device="cuda")
    for call, what in ((lambda: p(q.float(), start, lens), "q:"), (lambda: p(q[:, :200], start, lens), "q:"),
                       (lambda: p(more, start, lens), "workspace"), (lambda: p(q, start, torch.cat([lens, lens])), "workspace"),
                       (lambda: p(q, start[:2], lens), "row_start"), (lambda: p(q, start, lens.long()), "lens"),
                       (lambda: p(q, start, lens, seq=lens[:1]), "seq"), (lambda: p(q, start, lens, out=q.float()), "out"),
                       (lambda: d(q, start, lens, None), "visible"), (lambda: d(q, start, lens, vis.int()), "visible"),
                       (lambda: d(q, start, lens, vis[:5]), "visible"), (lambda: d(q, start, lens, torch.cat([vis, vis], 1)), "visible"),
                       (lambda: ops.DraftAttention(cs["cache"], 4, rows, 2, 257), "max_draft"),
                       (lambda: ops.PromptAttention(cs["cache"], 3, rows, 2), "not supported")):
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(Exception, match="slot"):
        p(q, start, lens, slot=2)
    empty = torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda")
    assert p(empty, start, lens).shape == (0, 256)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert (p(q, start, none, out=torch.full_like(q, SENTINEL)) == SENTINEL).all()


@pytest.mark.parametrize("draft", [False, True])
def test_the_same_call_gives_the_same_bits_captured_too(draft):
    import torch
    from continuous_depth_batching_gb300 import ops
    cs = make("bf16", 8, 2, 128, [20, 64, 40], [5000, 300, 0], **(dict(mask=tree) if draft else {}))
    rows = cs["q"].shape[0]
    op = ops.DraftAttention(cs["cache"], 8, rows, 3, 64, cs["max_ctx"]) if draft else \
        ops.PromptAttention(cs["cache"], 8, rows, 3, cs["max_ctx"])
    first = run(cs, op=op)
    for _ in range(3):
        assert torch.equal(run(cs, op=op), first)
    out = torch.full_like(first, SENTINEL)
    mask = (cs["visible"],) if draft else ()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op(cs["q"], cs["start"], cs["lens"], *mask, seq=cs["seq"], slot=1, out=out)
    for _ in range(3):
        out.fill_(SENTINEL)
        graph.replay()
        assert torch.equal(out, first)
    # other lengths in the same graph
    cs["lens"].copy_(cs["lens"] - 17)
    shorter = run(cs, op=op)
    out.fill_(SENTINEL)
    graph.replay()
    assert torch.equal(out, shorter) and not torch.equal(out, first)
