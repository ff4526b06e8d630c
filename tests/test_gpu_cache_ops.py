"""The paged-cache operators (include/cdb_ops.h) against float64 restatements.

Everything the operators must not touch or use (padding rows, unused positions,
pages behind a sequence's end) holds NaN or a sentinel.

Tolerances.  A stored bf16 value is within 2^-8 of its fp32 value, an e4m3 code
within 2^-4 of the scaled value or half a step of 2^-9 near zero, so a cached
value within 2^-4 |x| + 2^-10 s.  fp32 norms and rotations: a handful of
roundings of 2^-24 of the head's largest value, 2^-20 in all.

Attention: a score is a sum of head_dim exact products, accumulated in fp32 with
at most 2^-23 per step of S = |scale| * sum |q k|; a weight e^s is then off by that
(as an exponent) plus 2^-20 for the exponential and 2^-17 for its two-part 16-bit
form; weights enter twice (numerator, sum).  The weighted sum adds 2^-23 of max
|v| per accumulation step (16 keys each) and per joined split.
"""

import itertools

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def make_cache(dtype, blocks, slots, hk, hd, table, seed=0, fill=True):
    """A pool of random keys on the GPU; and its values in float64."""
    import torch
    from continuous_depth_batching_gb300 import ops
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
    return ops.PagedCache(pool, table, scales), vals


def poison(cache, vals, used):
    """NaN into every (block, slot, offset) that no row reads."""
    import torch
    m = ~used.cuda()
    raw = cache.pool.view(torch.uint8).view(*cache.pool.shape[:-1], -1)
    raw.masked_fill_(m[:, :, None, None, :, None], 0xFF)  # NaN in bf16 and in e4m3
    if cache.scales is not None:
        cache.scales.masked_fill_(m[:, :, None, None, :], float("nan"))


def attention_case(dtype, H, hk, hd, lengths, slots=1, shared=0, seed=0, extra_pages=3):
    """Rows with these own lengths (behind `shared` common positions) over shuffled pages."""
    import torch
    rng = np.random.default_rng(seed)
    rows = len(lengths)
    sp = shared // 16
    need = [(n + 15) // 16 for n in lengths]
    maxb = sp + max(need) + 2
    blocks = sp + sum(need) + extra_pages
    perm = rng.permutation(blocks)
    table = np.full((rows, maxb), -1, dtype=np.int32)
    at = sp
    for i, n in enumerate(need):
        table[i, :sp] = perm[:sp]
        table[i, sp:sp + n] = perm[at:at + n]
        at += n
    seq = rng.permutation(rows).astype(np.int32)
    pos = np.array([shared + lengths[s] - 1 for s in seq], dtype=np.int32)
    depth = rng.integers(0, slots, rows).astype(np.int32)
    t = torch.from_numpy(table).cuda()
    cache, vals = make_cache(dtype, blocks, slots, hk, hd, t, seed)
    used = torch.zeros(blocks, slots, 16, dtype=torch.bool)
    for i in range(rows):
        j = np.arange(pos[i] + 1)
        used[table[seq[i], j // 16], depth[i], j % 16] = True
    poison(cache, vals, used)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = (torch.randn(rows, H * hd, generator=g, device="cuda") * 1.5).bfloat16()
    return dict(cache=cache, vals=vals, q=q, seq=torch.from_numpy(seq).cuda(), pos=torch.from_numpy(pos).cuda(),
                depth=torch.from_numpy(depth).cuda(), table=table, H=H, hk=hk, hd=hd, shared=shared,
                max_ctx=int(pos.max()) + 1 + int(rng.integers(0, 17)))


def expected(cs, row, scale):
    """(output [H, hd] in float64, its tolerance) of one row."""
    import torch
    H, hk, hd = cs["H"], cs["hk"], cs["hd"]
    s, L, d = int(cs["seq"][row]), int(cs["pos"][row]) + 1, int(cs["depth"][row])
    j = np.arange(L)
    blk, off = torch.from_numpy(cs["table"][s, j // 16]).long().cuda(), torch.from_numpy(j % 16).cuda()
    k = cs["vals"][blk, d, 0, :, off].repeat_interleave(H // hk, 1)  # [L, H, hd]
    v = cs["vals"][blk, d, 1, :, off].repeat_interleave(H // hk, 1)
    q = cs["q"][row].double().view(H, hd)
    p = torch.softmax(torch.einsum("hd,lhd->hl", q, k) * scale, -1)
    o = torch.einsum("hl,lhd->hd", p, v)
    S = torch.einsum("hd,lhd->hl", q.abs(), k.abs()).max() * abs(scale)
    steps = 16 + L / 16 + L / 128
    tol = 2.0 ** -8 * o.abs() + v.abs().max() * (2 * (hd * 2.0 ** -23 * S + 2.0 ** -20 + 2.0 ** -17) + steps * 2.0 ** -23)
    return o, tol


def check_attention(cs, rows=None, scale=None, **kw):
    import torch
    from continuous_depth_batching_gb300 import ops
    n = cs["q"].shape[0]
    at = ops.DecodeAttention(cs["cache"], cs["H"], n, min(cs["max_ctx"], cs["cache"].max_ctx), scale=scale)
    args = dict(depth=cs["depth"]) if not cs["shared"] else dict(shared_len=cs["shared"])
    args.update(kw)
    out = at(cs["q"], cs["seq"], cs["pos"], **args)
    at.check()
    for i in rows if rows is not None else range(n):
        o, tol = expected(cs, i, scale if scale is not None else cs["hd"] ** -0.5)
        err = (out[i].double().view(cs["H"], cs["hd"]) - o).abs()
        assert bool((err <= tol).all()), (i, float((err / tol).max()), int(cs["pos"][i]))
    return out


LENGTHS = [1, 2, 15, 16, 17, 31, 33, 64, 100, 127, 128, 129, 255, 256, 257, 300, 511, 513, 700]
HEADS = [(16, 16), (8, 2), (12, 4), (5, 5), (6, 1), (20, 2), (17, 1), (9, 3)]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd", [32, 64, 96, 128])
@pytest.mark.parametrize("heads", HEADS)
def test_attention_shapes(dtype, hd, heads):
    check_attention(attention_case(dtype, *heads, hd, LENGTHS, slots=3, seed=hd + heads[0]))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attention_long(dtype):
    cs = attention_case(dtype, 8, 2, 128, [8191, 20000, 4097, 1, 12345], slots=1, seed=5)
    check_attention(cs)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attention_scale_and_sharp_scores(dtype):
    # Large scores: one key takes the whole weight; the running maximum moves often.
    cs = attention_case(dtype, 4, 4, 64, [600, 77, 1], seed=6)
    check_attention(cs, scale=1.0)
    check_attention(cs, scale=0.0)
    check_attention(cs, scale=-0.3)


def test_value_scales_over_many_orders():
    # Weights of e4m3 values are relative to the largest value scale so far: scales that
    # grow by 2^40 inside one row, and values that vanish beside a later one.
    import torch
    cs = attention_case("e4m3", 4, 4, 128, [300, 130, 40], seed=7)
    sc = cs["cache"].scales
    g = torch.Generator(device="cuda").manual_seed(1)
    f = torch.exp2(torch.randint(-20, 21, sc[:, :, 1].shape, generator=g, device="cuda").float())
    sc[:, :, 1] *= f
    cs["vals"][:, :, 1] *= f.double()[..., None]
    check_attention(cs)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_padding_empty_rows_and_strides(dtype):
    import torch
    from continuous_depth_batching_gb300 import ops
    cs = attention_case(dtype, 8, 4, 64, [50, 200, 3, 129], slots=2, seed=8)
    want = check_attention(cs)
    w = 8 * 64
    n = 7
    q = torch.full((n, w + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    seq = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    pos = torch.full((n,), 1 << 30, dtype=torch.int32, device="cuda")
    depth = torch.full((n,), 99, dtype=torch.int32, device="cuda")
    live = torch.tensor([1, 2, 4, 5], device="cuda")
    q[live, :w] = cs["q"]
    seq[live], pos[live], depth[live] = cs["seq"], cs["pos"], cs["depth"]
    seq[6], pos[6], depth[6] = 2, -1, 1  # a row without keys
    q[6, :w] = 1.0
    out = torch.full((n, w + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    at = ops.DecodeAttention(cs["cache"], 8, n)
    at(q[:, :w], seq, pos, depth, out=out[:, :w])
    at.check()
    assert torch.equal(out[live, :w], want)
    assert bool((out[6, :w] == 0).all())
    assert bool((out[[0, 3]] == 7).all()) and bool((out[:, w:] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_row_does_not_depend_on_the_batch(dtype):
    import torch
    from continuous_depth_batching_gb300 import ops
    cs = attention_case(dtype, 16, 4, 128, LENGTHS, slots=2, seed=9)
    want = check_attention(cs, rows=[0])
    for i in (0, 7, 18):
        at = ops.DecodeAttention(cs["cache"], 16, 1, cs["cache"].max_ctx)
        one = at(cs["q"][i:i + 1].clone(), cs["seq"][i:i + 1].clone(), cs["pos"][i:i + 1].clone(),
                 cs["depth"][i:i + 1].clone())
        assert torch.equal(one[0], want[i])


def test_pool_offsets_past_32_bits():
    import torch
    from continuous_depth_batching_gb300 import ops
    hk, hd, blocks = 8, 128, 140000  # 4.6 GB of codes
    table = torch.tensor([[blocks - 1, 0, blocks - 2], [5, blocks - 3, -1]], dtype=torch.int32, device="cuda")
    pool = torch.zeros(blocks, 1, 2, hk, 16, hd, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros(blocks, 1, 2, hk, 16, device="cuda")
    cache = ops.PagedCache(pool, table, scales)
    rows = 2
    w = ops.CacheWriter(cache, 16)
    g = torch.Generator(device="cuda").manual_seed(3)
    lens = [40, 29]
    ks = torch.zeros(2, 48, hk, hd, dtype=torch.float64, device="cuda")
    vs = torch.zeros_like(ks)
    seq = torch.arange(2, dtype=torch.int32, device="cuda")
    for p in range(max(lens)):
        qkv = torch.randn(rows, (16 + 2 * hk) * hd, generator=g, device="cuda")
        live = torch.tensor([s if p < lens[s] else -1 for s in range(2)], dtype=torch.int32, device="cuda")
        q = w(qkv, live, torch.full((2,), p, dtype=torch.int32, device="cuda"))
        kv = qkv.double().view(rows, -1, hd)
        ks[:, p], vs[:, p] = kv[:, 16:16 + hk], kv[:, 16 + hk:]
    w.check()
    q = torch.randn(rows, 16 * hd, generator=g, device="cuda").bfloat16()
    at = ops.DecodeAttention(cache, 16, rows)
    out = at(q, seq, torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda"))
    at.check()
    for i in range(rows):
        k, v = (x[i, :lens[i]].repeat_interleave(2, 1) for x in (ks, vs))
        s = torch.einsum("hd,lhd->hl", q[i].double().view(16, hd), k) * hd ** -0.5
        o = torch.einsum("hl,lhd->hd", torch.softmax(s, -1), v)
        # Keys and values are within 2^-4 of theirs; a score's error is then normal-sized sums of those.
        assert float((out[i].double().view(16, hd) - o).norm() / o.norm()) < 2.0 ** -4


SHARED_HEADS = [(16, 16), (8, 2), (9, 3), (5, 1), (24, 4)]


def check_shared(cs, kw=None):
    """A batch behind a common prefix.  The prefix's weights are bf16, each off by 2^-8 of itself: 2^-8 max |v|
    beside what expected() allows.  Over a row those errors are independent: the norm stays within 2^-7."""
    import torch
    from continuous_depth_batching_gb300 import ops
    n = cs["q"].shape[0]
    at = ops.DecodeAttention(cs["cache"], cs["H"], n + 3, min(cs["max_ctx"], cs["cache"].max_ctx))
    out = at(cs["q"], cs["seq"], cs["pos"], shared_len=cs["shared"], **(kw or {}))
    at.check()
    total = [0.0, 0.0]
    for i in range(n):
        if int(cs["seq"][i]) < 0:
            continue
        o, tol = expected(cs, i, cs["hd"] ** -0.5)
        err = (out[i].double().view(cs["H"], cs["hd"]) - o).abs()
        tol = tol + 2.0 ** -8 * cs["vals"][:, :, 1].nan_to_num().abs().max()
        assert bool((err <= tol).all()), (i, float((err / tol).max()), int(cs["pos"][i]))
        total[0] += float(err.square().sum())
        total[1] += float(o.square().sum())
    assert total[0] ** 0.5 <= 2.0 ** -7 * total[1] ** 0.5
    return out


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd", [32, 64, 96, 128])
@pytest.mark.parametrize("heads", SHARED_HEADS)
def test_shared_prefix_shapes(dtype, hd, heads):
    rng = np.random.default_rng(hd)
    for shared, rows in ((16, 2), (64, 5), (112, 33), (336, 3), (1040, 20)):
        lengths = [int(v) for v in rng.integers(1, 150, rows)]
        check_shared(attention_case(dtype, *heads, hd, lengths, shared=shared, seed=shared))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,shared", [(1, 512), (129, 256), (300, 2064), (40, 9008)])
def test_shared_prefix_large(dtype, rows, shared):
    rng = np.random.default_rng(rows)
    check_shared(attention_case(dtype, 8, 4, 128, [int(v) for v in rng.integers(1, 300, rows)], shared=shared, seed=rows))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_shared_prefix_rows_inside_it_and_padding(dtype):
    # Rows that end inside the prefix, at its end, without keys, and padding before the first live row.
    import torch
    cs = attention_case(dtype, 8, 2, 64, [1, 20, 3, 90, 7, 16, 1, 2], shared=208, seed=3)
    pos = cs["pos"]
    pos[1], pos[2], pos[3] = 207, 100, 0
    cs["seq"][0] = cs["seq"][5] = -1
    out = torch.full((8, 8 * 64 + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    check_shared(cs, dict(out=out[:, :512]))
    assert bool((out[[0, 5]] == 7).all()) and bool((out[:, 512:] == 7).all())
    pos[4] = -1
    from continuous_depth_batching_gb300 import ops
    at = ops.DecodeAttention(cs["cache"], 8, 8)
    at(cs["q"], cs["seq"], pos, shared_len=208, out=out[:, :512])
    at.check()
    assert bool((out[4, :512] == 0).all())
    cs["seq"].fill_(-1)
    out.fill_(3.0)
    at(cs["q"], cs["seq"], pos, shared_len=208, out=out[:, :512])
    at.check()
    assert bool((out == 3).all())


@pytest.mark.parametrize("shared", [0, 208])
def test_rows_without_keys_at_any_negative_position(shared):
    import torch
    from continuous_depth_batching_gb300 import ops
    cs = attention_case("bf16", 8, 2, 64, [20, 30, 3, 90], shared=208, seed=4)
    cs["pos"][1], cs["pos"][2] = -2 ** 31, -1000
    at = ops.DecodeAttention(cs["cache"], 8, 4)
    out = at(cs["q"], cs["seq"], cs["pos"], shared_len=shared)
    at.check()
    assert bool((out[1:3] == 0).all()) and bool((out[[0, 3]] != 0).any(1).all())


def test_shared_prefix_exactly_the_context():
    # No row has keys of its own.
    cs = attention_case("bf16", 4, 4, 128, [1, 1, 1], shared=128, seed=2)
    cs["pos"].fill_(127)
    cs["max_ctx"] = 128
    check_shared(cs)


def test_shared_prefix_of_other_blocks_is_reported():
    from continuous_depth_batching_gb300 import ops
    cs = attention_case("bf16", 4, 4, 64, [5, 9, 3], shared=64, seed=4)
    t = cs["cache"].block_table
    t[int(cs["seq"][2]), 1] = t[int(cs["seq"][2]), 4]
    at = ops.DecodeAttention(cs["cache"], 4, 3)
    at(cs["q"], cs["seq"], cs["pos"], shared_len=64)
    assert int(at.status.item()) == 128


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [1.0, 0.0, -0.3])
def test_shared_prefix_scales(dtype, scale):
    # Sharp scores, none, and turned-round ones.
    import torch
    from continuous_depth_batching_gb300 import ops
    cs = attention_case(dtype, 4, 2, 64, [30, 7, 1, 90], shared=320, seed=11)
    at = ops.DecodeAttention(cs["cache"], 4, 4, scale=scale)
    out = at(cs["q"], cs["seq"], cs["pos"], shared_len=320)
    at.check()
    v = cs["vals"][:, :, 1].nan_to_num().abs().max()
    for i in range(4):
        o, tol = expected(cs, i, scale)
        assert bool(((out[i].double().view(4, 64) - o).abs() <= tol + 2.0 ** -8 * v).all())


def test_shared_value_scales_over_many_orders():
    import torch
    from continuous_depth_batching_gb300 import ops
    cs = attention_case("e4m3", 4, 4, 128, [30, 40], shared=1024, seed=12)
    sc = cs["cache"].scales
    g = torch.Generator(device="cuda").manual_seed(1)
    f = torch.exp2(torch.randint(-20, 21, sc[:, :, 1].shape, generator=g, device="cuda").float())
    sc[:, :, 1] *= f
    cs["vals"][:, :, 1] *= f.double()[..., None]
    at = ops.DecodeAttention(cs["cache"], 4, 2)
    out = at(cs["q"], cs["seq"], cs["pos"], shared_len=1024)
    at.check()
    v = cs["vals"][:, :, 1].nan_to_num().abs().max()
    for i in range(2):
        o, tol = expected(cs, i, 128 ** -0.5)
        assert bool(((out[i].double().view(4, 128) - o).abs() <= tol + 2.0 ** -8 * v).all())


def test_zero_values_in_the_cache():
    # Pages of zeros: codes 0 with the smallest scale; the output of such keys alone is 0.
    import torch
    for shared in (0, 64):
        cs = attention_case("e4m3", 4, 4, 64, [20, 33], shared=shared, seed=13)
        cs["cache"].pool.view(torch.uint8)[:, :, 1] = 0
        cs["cache"].scales[:, :, 1] = 2.0 ** -126
        from continuous_depth_batching_gb300 import ops
        at = ops.DecodeAttention(cs["cache"], 4, 2)
        out = at(cs["q"], cs["seq"], cs["pos"], shared_len=shared)
        at.check()
        assert bool((out == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_shared_prefix_in_a_graph_and_on_a_side_stream(dtype):
    import torch
    from continuous_depth_batching_gb300 import ops
    cs = attention_case(dtype, 8, 4, 128, [40, 300, 7, 19, 120], shared=528, seed=14)
    plain = ops.DecodeAttention(cs["cache"], 8, 5)
    at = ops.DecodeAttention(cs["cache"], 8, 5)
    q, out = cs["q"].clone(), torch.zeros_like(cs["q"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        at(q, cs["seq"], cs["pos"], shared_len=528, out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            for _ in range(3):  # back to back on one workspace
                at(q, cs["seq"], cs["pos"], shared_len=528, out=out)
    torch.cuda.synchronize()
    for seed in range(5):
        q.copy_(torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        g.replay()
        got = out.clone()
        assert torch.equal(got, plain(q, cs["seq"], cs["pos"], shared_len=528))
    at.check()


def test_a_decode_step_of_all_operators():
    # Project, write, attend behind a shared prompt, project to logits, sample: against the same step in float64.
    import torch
    from continuous_depth_batching_gb300 import ops
    from tests.test_gpu_sample import reference
    H, hk, hd, d, vocab, rows, shared = 8, 4, 64, 256, 1000, 6, 64
    g = torch.Generator(device="cuda").manual_seed(21)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    cs = attention_case("e4m3", H, hk, hd, [5, 17, 1, 40, 16, 33], shared=shared, seed=22)
    cache, vals = cs["cache"], cs["vals"]
    h, wqkv, head = rnd(rows, d), rnd((H + 2 * hk) * hd, d) / 16, rnd(vocab, H * hd) / 8
    rope, gain = ops.rope_table(256, hd), 1 + 0.1 * rnd(hd)
    seq, pos = cs["seq"], cs["pos"]  # the last position of each sequence is this step's
    w = ops.CacheWriter(cache, H, rope, gain, gain)
    at, s = ops.DecodeAttention(cache, H, rows), ops.Sampler(rows, vocab)
    u, t = torch.rand(rows, generator=g, device="cuda"), torch.full((rows,), 0.9, device="cuda")
    p = torch.full((rows,), 0.8, device="cuda")
    qkv = h @ wqkv.T
    q = w(qkv, seq, pos)
    o = at(q, seq, pos, shared_len=shared)
    logits = o.float() @ head.T
    token, _ = s(logits, u, t, top_p=p)
    w.check()
    at.check()
    # Reference: the written row's key and value from the cache they went to, everything before it as it was.
    blk, off = cache.block_table[seq.long(), pos.long() // 16].long(), pos.long() % 16
    vals[blk, 0, :, :, off] = cache.pool[blk, 0, :, :, off].double() * cache.scales[blk, 0, :, :, off].double()[..., None]
    x = qkv.double().view(rows, H + 2 * hk, hd)
    y = x[:, :H + hk] / torch.sqrt((x[:, :H + hk] ** 2).mean(-1, keepdim=True) + 1e-6) * gain.double()
    c = torch.view_as_complex(rope.double().contiguous())[pos.long()][:, None]
    z = torch.complex(y[..., :hd // 2].contiguous(), y[..., hd // 2:].contiguous()) * c
    y = torch.cat([z.real, z.imag], -1)
    assert bool(((q.double().view(rows, H, hd) - y[:, :H]).abs() <= 2.0 ** -8 * y[:, :H].abs() + 2.0 ** -18).all())
    new = vals[blk, 0, :, :, off]
    want = torch.stack([y[:, H:], x[:, H + hk:]], 1)
    big = want.abs().amax(-1, keepdim=True)
    assert bool(((new - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 * big / 448 + 2.0 ** -18 * big).all())
    cs = dict(cs, q=q)
    for i in range(rows):
        e, tol = expected(cs, i, hd ** -0.5)
        tol = tol + 2.0 ** -8 * vals[:, :, 1].nan_to_num().abs().max()
        assert bool(((o[i].double().view(H, hd) - e).abs() <= tol).all())
        assert int(token[i]) == reference(logits[i].cpu().numpy(), float(u[i]), np.float32(0.9), None, np.float32(0.8))[0]


def write_reference(cs):
    """Float64 queries [rows, H, hd], keys and values [rows, 2, hk, hd]."""
    import torch
    H, hk, hd, rot = cs["H"], cs["hk"], cs["hd"], cs["rot"]
    x = cs["qkv"].double()[:, :(H + 2 * hk) * hd].view(-1, H + 2 * hk, hd)
    q, k, v = x[:, :H], x[:, H:H + hk], x[:, H + hk:]
    if cs["q_gain"] is not None:
        norm = lambda y, w: y / torch.sqrt((y * y).mean(-1, keepdim=True) + cs["eps"]) * w.double()
        q, k = norm(q, cs["q_gain"]), norm(k, cs["k_gain"])
    if rot:
        pos = cs["pos"].double()[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, device="cuda").double() / rot)
        c, s = pos.cos()[:, None], pos.sin()[:, None]

        def turn(y):
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            return torch.cat([a * c - b * s, b * c + a * s, y[..., rot:]], -1)
        q, k = turn(q), turn(k)
    return q, torch.stack([k, v], 1)


def write_case(dtype, src, H, hk, hd, rows, rot=None, norm=True, slots=2, seed=0, pad=0):
    import torch
    from continuous_depth_batching_gb300 import ops
    rng = np.random.default_rng(seed)
    rot = hd if rot is None else rot
    nseq, maxb = max(1, rows // 3), 9
    table = torch.from_numpy(rng.permutation(nseq * maxb + 2)[:nseq * maxb].reshape(nseq, maxb).astype(np.int32)).cuda()
    blocks = nseq * maxb + 2
    cells = rng.choice(nseq * maxb * 16 * slots, rows, replace=False)  # distinct (sequence, position, slot)
    seq, rest = np.divmod(cells, maxb * 16 * slots)
    pos, depth = np.divmod(rest, slots)
    shape = (blocks, slots, 2, hk, 16, hd)
    if dtype == "e4m3":
        pool = torch.full(shape, 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        scales = torch.full(shape[:-1], -3.0, device="cuda")
    else:
        pool, scales = torch.full(shape, 77.0, dtype=torch.bfloat16, device="cuda"), None
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(rows, (H + 2 * hk) * hd + 8, generator=g, device="cuda") * 3
    qkv = qkv.to(torch.bfloat16 if src == "bf16" else torch.float32)
    gain = [1 + 0.3 * torch.randn(hd, generator=g, device="cuda") for _ in range(2)] if norm else [None, None]
    i32 = lambda v: torch.from_numpy(np.asarray(v, dtype=np.int32)).cuda()
    return dict(cache=ops.PagedCache(pool, table, scales), qkv=qkv, q_gain=gain[0], k_gain=gain[1], eps=1e-5, rot=rot,
                rope=ops.rope_table(maxb * 16, rot) if rot else None, seq=i32(seq), pos=i32(pos), depth=i32(depth),
                H=H, hk=hk, hd=hd, rows=rows)


def run_write(cs, seq=None):
    import torch
    from continuous_depth_batching_gb300 import ops
    w = ops.CacheWriter(cs["cache"], cs["H"], cs["rope"], cs["q_gain"], cs["k_gain"], cs["eps"])
    width = cs["H"] * cs["hd"]
    q = torch.full((cs["rows"], width + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    w(cs["qkv"][:, :-8], cs["seq"] if seq is None else seq, cs["pos"], cs["depth"], q_out=q[:, :width])
    w.check()
    assert bool((q[:, width:] == 5).all())
    return q[:, :width]


def check_write(cs):
    import torch
    q = run_write(cs)
    wq, wkv = write_reference(cs)
    c, hd = cs["cache"], cs["hd"]
    got = q.double().view(wq.shape)
    tol = 2.0 ** -8 * wq.abs() + 2.0 ** -20 * wq.abs().amax(-1, keepdim=True)
    assert bool(((got - wq).abs() <= tol).all())
    blk = c.block_table[cs["seq"].long(), cs["pos"].long() // 16].long()
    at = (blk, cs["depth"].long(), slice(None), slice(None), cs["pos"].long() % 16)
    raw = c.pool.view(torch.uint8)[at].view(c.pool.dtype)
    big = wkv.abs().amax(-1, keepdim=True)
    if c.scales is None:
        assert bool(((raw.double() - wkv).abs() <= 2.0 ** -8 * wkv.abs() + 2.0 ** -20 * big).all())
    else:
        s = c.scales[at].double()[..., None]
        want = (big / 448).clamp_min(2.0 ** -126)
        assert bool(((s - want).abs() <= 2.0 ** -20 * want).all())
        assert bool(((raw.double() * s - wkv).abs() <= 2.0 ** -4 * wkv.abs() + 2.0 ** -10 * s + 2.0 ** -20 * big).all())
    # Nothing else changed.
    touched = torch.zeros(c.pool.shape[0], c.n_slots, 16, dtype=torch.bool, device="cuda")
    touched[blk, cs["depth"].long(), cs["pos"].long() % 16] = True
    keep = (~touched)[:, :, None, None, :].expand(c.pool.shape[:-1])
    if c.scales is None:
        assert bool((c.pool[keep] == 77).all())
    else:
        assert bool((c.pool.view(torch.uint8)[keep] == 0x55).all()) and bool((c.scales[keep] == -3).all())


@pytest.mark.parametrize("dtype,src", list(itertools.product(["bf16", "e4m3"], ["fp32", "bf16"])))
@pytest.mark.parametrize("hd", [32, 64, 96, 128])
@pytest.mark.parametrize("heads", [(16, 16), (8, 2), (7, 7), (5, 1), (55, 11)])
def test_write_shapes(dtype, src, hd, heads):
    check_write(write_case(dtype, src, *heads, hd, 37, seed=hd + heads[0]))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("rot,norm", [(0, True), (0, False), (128, False), (64, True), (16, True), (96, False)])
def test_write_without_norm_or_with_partial_rotation(dtype, rot, norm):
    check_write(write_case(dtype, "fp32", 8, 4, 128, 50, rot=rot, norm=norm, seed=rot))


def test_write_one_row_and_many():
    check_write(write_case("e4m3", "fp32", 16, 16, 128, 1))
    check_write(write_case("e4m3", "bf16", 4, 2, 64, 3000, seed=2))


def test_write_leaves_padding_rows():
    import torch
    cs = write_case("e4m3", "fp32", 8, 2, 64, 20, seed=4)
    before = cs["cache"].pool.view(torch.uint8).clone()
    cs["qkv"].fill_(float("nan"))
    q = run_write(cs, torch.full_like(cs["seq"], -1))
    assert bool((q == 5).all()) and torch.equal(before, cs["cache"].pool.view(torch.uint8))


def test_write_extreme_values():
    # All zeros, values below the smallest scale, the largest floats, infinities and NaN.
    import torch
    cs = write_case("e4m3", "fp32", 2, 1, 32, 6, rot=0, norm=False, seed=5)
    x = cs["qkv"][:, :-8].view(6, 4, 32)
    x[0] = 0.0
    x[1] = 1e-42
    x[2] = 3e38
    x[3, :, 3] = float("inf")
    x[4, :, 5] = float("nan")
    run_write(cs)
    c = cs["cache"]
    blk = c.block_table[cs["seq"].long(), cs["pos"].long() // 16].long()
    at = (blk, cs["depth"].long(), slice(None), slice(None), cs["pos"].long() % 16)
    s = c.scales[at].double()[..., None]
    v = c.pool.view(torch.uint8)[at].view(torch.float8_e4m3fn).double() * s
    assert bool((v[0] == 0).all()) and bool((s[:2] == 2.0 ** -126).all())
    assert float((v[1] - 1e-42).abs().max()) <= 2.0 ** -10 * 2.0 ** -126
    assert float((v[2] / 3e38 - 1).abs().max()) <= 2.0 ** -20
    assert bool(torch.isnan(v[3]).all())           # an infinity leaves no number in its head
    assert bool(torch.isnan(v[4, :, :, 5]).all())  # a NaN stays one; its neighbours are numbers
    assert bool(torch.isfinite(v[4, :, :, :5]).all())


def test_indexes_out_of_range_are_reported():
    import torch
    from continuous_depth_batching_gb300 import ops
    from continuous_depth_batching_gb300.binding import CdbError
    for dtype in ("bf16", "e4m3"):
        cs = write_case(dtype, "fp32", 4, 2, 64, 8, seed=6)
        c = cs["cache"]
        table0 = c.block_table.clone()
        w = ops.CacheWriter(c, 4, cs["rope"])
        at = ops.DecodeAttention(c, 4, 8)
        q = torch.ones(8, 256, dtype=torch.bfloat16, device="cuda")
        maxb = c.block_table.shape[1]
        bad = [("seq", c.block_table.shape[0], 8), ("pos", maxb * 16, 8), ("depth", 2, 2), ("depth", -1, 2),
               ("block", -1, 1), ("block", c.pool.shape[0], 1)]
        for what, value, bit in bad:
            v = {k: cs[k].clone() for k in ("seq", "pos", "depth")}
            c.block_table.copy_(table0)
            if what == "block":
                c.block_table[int(cs["seq"][3]), int(cs["pos"][3]) // 16] = value
            else:
                v[what][3] = value
            out = torch.full_like(q, 9.0)
            qo = torch.full_like(q, 9.0)
            w(cs["qkv"][:, :-8], v["seq"], v["pos"], v["depth"], q_out=qo)
            assert int(w.status.item()) == bit and bool((qo[3] == 9).all()) and bool((qo[2] != 9).any())
            with pytest.raises(CdbError):
                w.check()
            w.check()  # reported once
            at(q, v["seq"], v["pos"], v["depth"], out=out)
            assert int(at.status.item()) == bit
            if what != "block":
                assert bool((out[3] == 9).all())
            with pytest.raises(CdbError):
                at.check()
        c.block_table.copy_(table0)


def test_write_then_attend_in_a_graph():
    # A decode step captured once and replayed with new inputs in the same buffers.
    import torch
    from continuous_depth_batching_gb300 import ops
    H, hk, hd, rows, steps = 8, 4, 128, 5, 40
    table = torch.arange(rows * 4, dtype=torch.int32, device="cuda").view(rows, 4)
    cache = ops.PagedCache(torch.zeros(rows * 4, 1, 2, hk, 16, hd, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                           table, torch.zeros(rows * 4, 1, 2, hk, 16, device="cuda"))
    rope = ops.rope_table(64, hd)
    gain = torch.ones(hd, device="cuda")
    w = ops.CacheWriter(cache, H, rope, gain, gain)
    at = ops.DecodeAttention(cache, H, rows)
    qkv = torch.zeros(rows, (H + 2 * hk) * hd, device="cuda")
    seq = torch.arange(rows, dtype=torch.int32, device="cuda")
    pos = torch.zeros(rows, dtype=torch.int32, device="cuda")
    q = torch.zeros(rows, H * hd, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    w(qkv, seq, pos, q_out=q)
    at(q, seq, pos, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w(qkv, seq, pos, q_out=q)
        at(q, seq, pos, out=out)
    gen = torch.Generator(device="cuda").manual_seed(2)
    for p in range(steps):
        qkv.normal_(generator=gen)
        pos.fill_(p)
        g.replay()
        got = out.clone()
        at(q, seq, pos, out=out)
        assert torch.equal(got, out)
    at.check()
    w.check()
    used = torch.zeros(rows * 4, 1, 16, dtype=torch.bool)
    vals = cache.pool.double() * cache.scales.double()[..., None]
    cs = dict(q=q, seq=seq, pos=pos, depth=torch.zeros_like(pos), table=table.cpu().numpy(), H=H, hk=hk, hd=hd, vals=vals)
    for i in range(rows):
        o, tol = expected(cs, i, hd ** -0.5)
        assert bool(((out[i].double().view(H, hd) - o).abs() <= tol).all())


def test_value_codes_are_rounded_once():
    """Codes of values (no norm, no rotation) equal the quotients' in 64 bits, also next to the borders between codes.

    x 448 against a border times max|x| is exact in float64 (24 + 9 bits), and differs from it by 2^-34 of its value
    at least, or not at all: far more than what the kernel's remainders are off by (2^-48).  Subnormal codes (|x| below
    2^-6 of the scale) are off by at most one."""
    import torch
    from continuous_depth_batching_gb300 import ops
    rows, hk, hd = 600, 2, 128
    rng = np.random.default_rng(11)
    table = torch.arange(rows // 16 + 1, dtype=torch.int32, device="cuda")[None].contiguous()
    pool = torch.zeros(rows // 16 + 1, 1, 2, hk, 16, hd, dtype=torch.float8_e4m3fn, device="cuda")
    c = ops.PagedCache(pool, table, torch.zeros(pool.shape[:-1], dtype=torch.float32, device="cuda"))
    x = rng.standard_normal((rows, hk, hd)).astype(np.float32)
    big = (np.abs(x).max(-1, keepdims=True) * rng.uniform(1, 2, (rows, hk, 1))).astype(np.float32)
    border = (2 * rng.integers(8, 15, (rows, hk, hd)) + 1) * 2.0 ** rng.integers(-9, 4, (rows, hk, hd))  # 1.mmm1 in binary
    near = (border * big.astype(np.float64) / 448).astype(np.float32)
    near = np.nextafter(near, np.where(rng.random(near.shape) < 0.5, np.float32(0), np.float32(np.inf)), dtype=np.float32)
    near = np.where(rng.random(near.shape) < 0.5, near, (border * big.astype(np.float64) / 448).astype(np.float32))
    x = np.where(rng.random(x.shape) < 0.7, near * rng.choice([-1, 1], x.shape), x).astype(np.float32)
    x[..., 5] = big[..., 0]  # the largest
    x[::50, :, :] = np.round(x[::50] * 64) * 2.0 ** -6  # exact borders among them
    x[::50, :, 5] = 7.0  # 448 / 64
    x[::50] = np.clip(x[::50], -7, 7)
    qkv = torch.zeros(rows, 3 * hk * hd, device="cuda")
    qkv[:, 2 * hk * hd:] = torch.from_numpy(x.reshape(rows, -1)).cuda()
    w = ops.CacheWriter(c, hk)
    zero = torch.zeros(rows, dtype=torch.int32, device="cuda")
    w(qkv, zero, torch.arange(rows, dtype=torch.int32, device="cuda"))
    w.check()
    got = pool[:, 0, 1].permute(0, 2, 1, 3).reshape(-1, hk, hd)[:rows].double().cpu().numpy()
    x = x.astype(np.float64)
    z = x * 448 / np.abs(x).max(-1, keepdims=True)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(z), 1e-30))), -6) - 3)
    want = np.rint(z / step) * step
    normal = np.abs(z) >= 2.0 ** -6
    assert (got[normal] == want[normal]).all(), int((got != want)[normal].sum())
    assert (np.abs(got - want)[~normal] <= 2.0 ** -9).all()
