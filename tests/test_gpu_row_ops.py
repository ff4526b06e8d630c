"""Pages and rows, rotation and accepted paths (include/cdb_ops.h) against plain restatements.

Tolerances.  Rotation: the norm (a sum of head_dim squares, a root, two products) and the turn (a sine and
a cosine within 2^-23, two products, a sum) are a handful of roundings of 2^-24 of the pair's size, 2^-20 in
all; the angle is exact to 2^-40 of a turn.  A bf16 output adds 2^-8 of its value.  The rest are whole numbers
and copies.
"""

import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# pages and rows
# ---------------------------------------------------------------------------

class Pages:
    """The operator's meaning, one request after the other."""

    def __init__(self, n_seqs, max_blocks, blocks, head=0):
        self.table = np.full((n_seqs, max_blocks), -1, dtype=np.int64)
        self.ring = np.full(blocks, -1, dtype=np.int64)
        self.ring[(head + np.arange(blocks)) % blocks] = np.arange(blocks)[::-1]
        self.head, self.tail = head, head + blocks

    def step(self, lens, new, seq, max_rows):
        start, rows, give = [0], [], []
        out = list(lens)
        for i, (l, d) in enumerate(zip(lens, new)):
            after = max(0, l + d)
            have, want = -(-l // 16), -(-after // 16)
            for p in range(have, want):
                self.table[seq[i], p] = self.ring[self.head % len(self.ring)]
                self.head += 1
            for p in range(want, have):
                give.append(self.table[seq[i], p])
            for pos in range(l, l + max(0, d)):
                rows.append((seq[i], pos, self.table[seq[i], pos // 16] * 16 + pos % 16))
            start.append(len(rows))
            out[i] = after
        for b in give:
            self.ring[self.tail % len(self.ring)] = b
            self.tail += 1
        rows += [(-1, -1, -1)] * (max_rows - len(rows))
        return out, start, rows


def upload(x, dtype=None):
    import torch
    return torch.tensor(np.asarray(x), dtype=dtype or torch.int32, device="cuda")


@pytest.mark.parametrize("n,max_rows", [(1, 5), (1, 5000), (64, 300), (513, 4000), (3000, 40000)])
def test_pages_over_many_steps(n, max_rows):
    import torch
    from continuous_depth_batching_gb300 import ops
    rng = np.random.default_rng(n)
    seqs, max_blocks = n + 3, 400
    blocks = 40 * n + 400
    ref = Pages(seqs, max_blocks, blocks, head=7 * blocks - 3)
    table, ring = upload(ref.table), upload(ref.ring)
    state = upload([ref.head, ref.tail], torch.int64)
    seq = rng.permutation(seqs)[:n]
    lens = [0] * n
    plan = ops.PagePlanner(table, ring, n, max_rows)
    d_lens = upload(lens)
    for step in range(6):
        most = max(1, max_rows // n)
        new = rng.integers(0, most + 1, n)
        if step == 2:
            new[:] = 0
        if step >= 3:
            new = np.where(rng.random(n) < 0.4, -rng.integers(1, 40, n), new)
        lens, start, rows = ref.step(lens, new.tolist(), seq, max_rows)
        got = plan(state, d_lens, upload(new), seq=upload(seq))
        plan.check()
        rows = np.array(rows).reshape(max_rows, 3)
        assert got.row_start.tolist() == start
        assert np.array_equal(got.seq.cpu().numpy(), rows[:, 0])
        assert np.array_equal(got.pos.cpu().numpy(), rows[:, 1])
        assert np.array_equal(got.slot.cpu().numpy(), rows[:, 2])
        assert d_lens.tolist() == lens and state.tolist() == [ref.head, ref.tail]
        assert np.array_equal(table.cpu().numpy(), ref.table)
        assert np.array_equal(ring.cpu().numpy(), ref.ring)


@pytest.mark.parametrize("new,seq,lens,what", [
    ([30, 40], [0, 1], [0, 0], "free blocks"),          # 5 pages of 4
    ([20, 20], [0, 1], [0, 0], "rows"),                 # 40 rows of 32
    ([5, 5], [0, 4], [0, 0], "sequence"),
    ([5, 5], [0, -1], [0, 0], "sequence"),
    ([5, 5], [0, 1], [-1, 0], "sequence"),
    ([5, 1], [0, 1], [0, 160], "sequence"),             # an eleventh page
    ([2147483647, 2147483647], [0, 1], [5, 5], "sequence"),
])
def test_pages_change_nothing_where_they_cannot_be_served(new, seq, lens, what):
    import torch
    from continuous_depth_batching_gb300 import ops
    from continuous_depth_batching_gb300.binding import CdbError
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(4, 10).contiguous()
    ring = upload([3, 1, 2, 0, 9, 9, 9, 9])
    state, d_lens = upload([8, 12], torch.int64), upload(lens)
    plan = ops.PagePlanner(table, ring, 2, 32)
    before = [x.clone() for x in (table, ring, state, d_lens)]
    got = plan(state, d_lens, upload(np.array(new)), seq=upload(seq))
    with pytest.raises(CdbError, match=what):
        plan.check()
    plan.check()  # reported once
    for x, y in zip((table, ring, state, d_lens), before):
        assert torch.equal(x, y)
    assert got.row_start.tolist() == [0, 0, 0]
    assert (got.seq == -1).all() and (got.pos == -1).all() and (got.slot == -1).all()


def test_pages_apart_from_their_inputs_and_without_requests():
    import torch
    from continuous_depth_batching_gb300 import ops
    table, ring = torch.full((3, 4), -1, dtype=torch.int32, device="cuda"), upload([4, 5, 6, 7])
    state, lens = upload([0, 4], torch.int64), upload([15, 0])
    so, lo = torch.zeros_like(state), torch.zeros_like(lens)
    table[0, 0] = 9
    plan = ops.PagePlanner(table, ring, 2, 8)
    for _ in range(2):  # the same answer twice
        got = plan(state, lens, upload([2, 1]), state_out=so, lens_out=lo)
        plan.check()
        assert state.tolist() == [0, 4] and lens.tolist() == [15, 0]
        assert so.tolist() == [2, 4] and lo.tolist() == [17, 1]
        assert got.slot.tolist() == [9 * 16 + 15, 4 * 16, 5 * 16] + [-1] * 5
        assert got.seq.tolist() == [0, 0, 1] + [-1] * 5 and got.pos.tolist() == [15, 16, 0] + [-1] * 5
    none = upload([])
    got = plan(state, none, none, state_out=so, lens_out=none)
    assert got.row_start.tolist() == [0] and (got.seq == -1).all() and so.tolist() == [0, 4]
    with pytest.raises(ValueError, match="at most 2"):
        plan(state, upload([1, 2, 3]), upload([1, 2, 3]))
    with pytest.raises(ValueError, match="state"):
        plan(lens, lens, upload([1, 2]))
    with pytest.raises(ValueError, match="new_tokens"):
        plan(state, lens, upload([1]))


# ---------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------

def rotated(x, pos, heads, kv, hd, inv, inter, factor, gains, eps):
    """float64 [rows, (heads + kv) * hd], and each element's pair size."""
    rows, rot = x.shape[0], 2 * len(inv)
    y = x[:, :(heads + kv) * hd].astype(np.float64).reshape(rows, heads + kv, hd).copy()
    if gains:
        y /= np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        y[:, :heads] *= gains[0]
        y[:, heads:] *= gains[1]
    a = pos[:, None] * inv
    c, s = np.cos(a)[:, None] * factor, np.sin(a)[:, None] * factor
    one = slice(0, rot, 2) if inter else slice(0, rot // 2)
    two = slice(1, rot, 2) if inter else slice(rot // 2, rot)
    u, v = y[..., one].copy(), y[..., two].copy()
    y[..., one], y[..., two] = u * c - v * s, v * c + u * s
    size = np.abs(y)
    size[..., one] = size[..., two] = np.hypot(u, v) * abs(factor)
    return y.reshape(rows, -1), size.reshape(rows, -1)


ROT = [(hd, rot) for hd in (32, 64, 96, 128) for rot in sorted({16, 16 * (hd // 32), hd})]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("hd,rot", ROT)
def test_rotation(dtype, inter, hd, rot):
    import torch
    from continuous_depth_batching_gb300 import ops
    for rows, heads, kv, norm, far, factor in ((1, 16, 16, True, 100, 1.0), (37, 5, 1, False, 2 ** 31 - 50, 1.3), (700, 3, 0, True, 10 ** 6, -0.5)):
        g = torch.Generator(device="cuda").manual_seed(rows + hd + rot)
        width = (heads + kv) * hd
        x = torch.randn(rows, width + 64, generator=g, device="cuda") * 3
        x = x.to(torch.float32 if dtype == "fp32" else torch.bfloat16)
        pos = torch.randint(0, far, (rows,), generator=g, device="cuda").to(torch.int32)
        pos[rows // 2:rows // 2 + rows // 8] = -1
        gains = [1 + 0.3 * torch.randn(hd, generator=g, device="cuda") for _ in range(2)] if norm else None
        steps, _ = ops.rope_steps(rot, theta=50000.0)
        inv = 50000.0 ** (-np.arange(rot // 2) * 2 / rot)
        op = ops.Rotary(heads, kv, hd, steps, interleaved=inter, factor=factor, q_gain=gains and gains[0],
                        k_gain=gains and gains[1], eps=1e-5)
        out = torch.full((rows, width + 8), 7.0, dtype=x.dtype, device="cuda")
        keep = x.clone()
        assert op(x, pos, out=out) is out
        assert torch.equal(x, keep)
        want, size = rotated(x.double().cpu().numpy(), pos.cpu().numpy().astype(np.float64), heads, kv, hd, inv, inter, factor,
                             gains and [v.double().cpu().numpy() for v in gains], 1e-5)
        got = out.double().cpu().numpy()
        pad = (pos < 0).cpu().numpy()
        assert (got[:, width:] == 7).all() and (got[pad] == 7).all()
        # float64 angles of the reference: 2^-52 of up to 2^31 radians
        tol = size * (2.0 ** -20 + 2.0 ** -20) + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0) + 1e-30
        err = np.abs(got[:, :width] - want)[~pad]
        assert (err <= tol[~pad]).all(), (err / tol[~pad]).max()
        assert op(x, pos) is x  # in place
        assert torch.equal(x[:, :width][pos >= 0], out[:, :width][pos >= 0])
        assert torch.equal(x[:, width:], keep[:, width:]) and torch.equal(x[pos < 0], keep[pos < 0])


def test_rotation_refuses_tensors():
    import torch
    from continuous_depth_batching_gb300 import ops
    steps, _ = ops.rope_steps(64)
    op = ops.Rotary(4, 2, 64, steps)
    x, pos = torch.zeros(3, 384, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    for args, what in (((x.half(), pos), "x:"), ((x[:, :380], pos), "x:"), ((x, pos.long()), "pos:"), ((x, pos[:2]), "pos:"),
                       ((x.cpu(), pos), "x:"), ((x, pos, x.bfloat16()), "out:"), ((x, pos, x[:2]), "out:"),
                       ((x.expand(3, 384)[:, ::2], pos), "x:")):
        with pytest.raises(ValueError, match=what):
            op(*args)
    with pytest.raises(ValueError, match="steps"):
        ops.Rotary(4, 2, 64, steps.cpu())
    with pytest.raises(ValueError, match="come together"):
        ops.Rotary(4, 2, 64, steps, q_gain=torch.ones(64, device="cuda"))


# ---------------------------------------------------------------------------
# accepted paths
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("slots,hk,hd", [(1, 1, 32), (3, 5, 96), (24, 2, 64), (2, 4, 128)])
def test_paths(dtype, slots, hk, hd):
    import torch
    from continuous_depth_batching_gb300 import ops
    rng = np.random.default_rng(hd + slots)
    n, nodes, most, max_blocks = 9, 100, 40, 30
    base = rng.integers(0, 16 * max_blocks - nodes + 1, n)
    base[1] = 16 * max_blocks - nodes  # up to the last position
    keep = rng.integers(0, most + 1, n)
    keep[2], keep[3] = 0, most
    path = np.full((n, most + 3), 77)
    for i in range(n):
        path[i, :keep[i]] = np.sort(rng.permutation(nodes)[:keep[i]])
    path[4, :keep[4]] = np.arange(keep[4])  # in place already
    seq = rng.permutation(n + 2)[:n]
    seq[5] = -1
    table = rng.permutation((n + 2) * max_blocks).reshape(n + 2, max_blocks)
    shape = (table.size, slots, 2, hk, 16, hd)
    bits = torch.from_numpy(rng.integers(0, 256, shape + (2 if dtype == "bf16" else 1,), dtype=np.uint8)).cuda()
    if dtype == "bf16":
        pool, scales = bits.view(torch.bfloat16).view(shape), None
    else:
        pool = bits.view(torch.float8_e4m3fn).view(shape)
        scales = torch.from_numpy(rng.standard_normal(shape[:-1]).astype(np.float32)).cuda()
    cache = ops.PagedCache(pool, upload(table), scales)
    want = bits.cpu().numpy().copy()
    want_s = scales.cpu().numpy().copy() if scales is not None else None
    for i in range(n):
        if seq[i] < 0:
            continue
        for k in range(keep[i]):
            a, b = base[i] + path[i, k], base[i] + k
            src, dst = (table[seq[i], a // 16], a % 16), (table[seq[i], b // 16], b % 16)
            want[dst[0], :, :, :, dst[1]] = want[src[0], :, :, :, src[1]]
            if want_s is not None:
                want_s[dst[0], :, :, :, dst[1]] = want_s[src[0], :, :, :, src[1]]
    op = ops.PathKeeper(cache)
    op(upload(base), upload(path)[:, :most], upload(keep), seq=upload(seq))
    op.check()
    assert np.array_equal(bits.cpu().numpy(), want)
    if want_s is not None:
        assert np.array_equal(scales.cpu().numpy(), want_s)


@pytest.mark.parametrize("base,path,keep,seq,what", [
    (10, [0, 0, 3], 3, 0, "sequence"), (10, [2, 1], 2, 0, "sequence"), (10, [-1, 3], 2, 0, "sequence"), (60, [1, 4], 2, 0, "sequence"),
    (-1, [1, 2], 2, 0, "sequence"), (10, [1, 2], 4, 0, "sequence"), (10, [1, 2], -1, 0, "sequence"), (10, [1, 2], 2, 2, "sequence"),
    (40, [1, 9], 2, 1, "block table")])
def test_paths_that_are_refused_move_nothing(base, path, keep, seq, what):
    import torch
    from continuous_depth_batching_gb300 import ops
    from continuous_depth_batching_gb300.binding import CdbError
    pool = torch.randn(8, 2, 2, 3, 16, 64, device="cuda").bfloat16()
    cache = ops.PagedCache(pool, upload([[0, 1, 2, 3], [4, 5, 6, 99]]), None)
    op = ops.PathKeeper(cache)
    before = pool.clone()
    p = upload([path + [50] * (3 - len(path))])
    op(upload([base]), p, upload([keep]), seq=upload([seq]))
    with pytest.raises(CdbError, match=what):
        op.check()
    assert torch.equal(pool, before)
    with pytest.raises(ValueError, match="path"):
        op(upload([base]), p.long(), upload([1]))
    with pytest.raises(ValueError, match="keep"):
        op(upload([base]), p, upload([]))
