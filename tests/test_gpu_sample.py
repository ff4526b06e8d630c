"""Sampling (include/cdb_ops.h) against a float64 restatement of its definition.

Tokens must be equal: the kernel's weights are within 2^-33 of their values, so
over every row of this file (below 4000) a running sum is on the wrong side of
its border with probability below 4000 * 2 * sqrt(262144) * 2^-33 = 4.8e-4.
logprob: a float32 sum of a quotient and a logarithm, each within 2^-22 of its
value, the quotient's operand below 90 in magnitude: 90 * 2^-22 + 2^-22 * |log|.
The reference rounds each weight to the operator's unit and adds integers: with
float64 sums it misses borders that u meets exactly (200 weights of 1 and 800 of
e^-0.75, u = 1/8: the running mass 100 e^-0.75 + 25 is u times the total).
"""

import math
from fractions import Fraction

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def reference(x, u, t, k=None, p=None, mp=None):
    """Token and log probability of one row (float64, lists in index order)."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    if not np.any(x > -np.inf):
        return -1, -np.inf
    m = x.max()
    if not t > 0:
        return int(np.argmax(x)), 0.0
    with np.errstate(invalid="ignore"):
        z = np.where(x == m, 0.0, (x - m) / np.float64(t))
    valid = np.nonzero(x > -np.inf)[0] if m < np.inf else np.nonzero(x == m)[0]
    order = valid[np.lexsort((valid, -x[valid]))]
    if k is not None and 0 < k < len(x):
        order = order[:k]
    w = np.exp(z[order])
    mass = lambda v: np.cumsum(np.rint(v * 2.0 ** 44).astype(np.int64))  # < 2^62: exact sums
    if p is not None and p < 1:
        c = mass(w)
        need = max(1, math.ceil(Fraction(float(p)) * int(c[-1])))
        order = order[:int(np.searchsorted(c, need, side="left")) + 1]
        w = w[:len(order)]
    if mp is not None and mp > 0:
        order = order[w >= min(float(mp), 1.0)]
    kept = np.sort(order)
    w = np.exp(z[kept])
    c = mass(w)
    u = min(max(float(u), 0.0), 1 - 2.0 ** -24)
    if u > 0:
        at = int(np.searchsorted(c, math.floor(Fraction(u) * int(c[-1])), side="right"))
    else:
        at = int(np.argmax(z[kept] > -700))
    return int(kept[at]), float(z[kept[at]] - np.log(w.sum()))


def check(x, u, t, k=None, p=None, mp=None, bf16=False, pad=0):
    import torch
    from continuous_depth_batching_gb300 import ops
    x = torch.as_tensor(np.asarray(x, dtype=np.float32))
    if bf16:
        x = x.bfloat16()
    rows, vocab = x.shape
    wide = torch.full((rows, vocab + pad), 1e9).to(x.dtype).cuda()  # never read behind the vocabulary
    wide[:, :vocab] = x.cuda()
    f = lambda v: None if v is None else torch.as_tensor(np.asarray(v, dtype=np.float32)).cuda()
    kk = None if k is None else torch.as_tensor(np.asarray(k, dtype=np.int32)).cuda()
    s = ops.Sampler(rows, vocab)
    token, logprob = s(wide[:, :vocab], f(u), f(t), kk, f(p), f(mp))
    token, logprob = token.cpu().numpy(), logprob.cpu().numpy().astype(np.float64)
    xs = x.float().numpy()
    pick = lambda v, i: None if v is None else v[i]
    f32 = lambda v: None if v is None else np.asarray(v, dtype=np.float32)
    u, t, p, mp = f32(u), f32(t), f32(p), f32(mp)
    for i in range(rows):
        want, lp = reference(xs[i], u[i], t[i], pick(k, i), pick(p, i), pick(mp, i))
        assert token[i] == want, (i, token[i], want, t[i], pick(k, i), pick(p, i), pick(mp, i))
        if np.isinf(lp):
            assert logprob[i] == lp
        else:
            assert abs(logprob[i] - lp) <= 90 * 2.0 ** -22 + 2.0 ** -22 * abs(lp), (i, logprob[i], lp)
    return token


def settings(rng, rows, vocab):
    t = rng.uniform(0.2, 2.0, rows).astype(np.float32)
    k = rng.integers(1, max(2, min(vocab, 500)), rows).astype(np.int32)
    p = rng.uniform(0.3, 1.0, rows).astype(np.float32)
    mp = rng.uniform(0.0, 0.3, rows).astype(np.float32)
    off = rng.random((3, rows)) < 0.4
    return t, np.where(off[0], 0, k), np.where(off[1], 1.0, p).astype(np.float32), np.where(off[2], 0, mp).astype(np.float32)


@pytest.mark.parametrize("vocab", [1, 2, 31, 33, 500, 1023, 4097, 16384, 16389, 49152, 65536, 131075, 262144])
@pytest.mark.parametrize("bf16", [False, True])
def test_all_filters(vocab, bf16):
    rng = np.random.default_rng(vocab + bf16)
    rows = 24 if vocab < 100000 else 8
    x = rng.standard_normal((rows, vocab)) * rng.uniform(0.3, 6, (rows, 1))
    t, k, p, mp = settings(rng, rows, vocab)
    check(x, rng.random(rows), t, k, p, mp, bf16=bf16, pad=rng.integers(0, 9))


@pytest.mark.parametrize("rows", [1, 3, 64, 200, 700])
def test_row_counts(rows):
    # The cluster size follows the number of rows; the tokens must not.
    rng = np.random.default_rng(rows)
    vocab = 5003
    x = rng.standard_normal((rows, vocab)) * 2
    t, k, p, mp = settings(rng, rows, vocab)
    u = rng.random(rows)
    token = check(x, u, t, k, p, mp)
    assert check(x[:1], u[:1], t[:1], k[:1], p[:1], mp[:1])[0] == token[0]


@pytest.mark.parametrize("only", ["t", "k", "p", "mp"])
def test_one_filter(only):
    rng = np.random.default_rng(7)
    rows, vocab = 40, 20000
    x = rng.standard_normal((rows, vocab)) * 2.5
    t, k, p, mp = settings(rng, rows, vocab)
    kw = {"k": np.maximum(k, 1), "p": np.minimum(p, 0.99).astype(np.float32), "mp": mp}
    check(x, rng.random(rows), t, **({only: kw[only]} if only in kw else {}))


def test_equal_logits():
    # Every border is a tie: by index, and k, p and u at exact fractions.
    rows, vocab = 16, 4096
    x = np.full((rows, vocab), 3.25)
    u = np.arange(rows) / rows
    token = check(x, u, np.ones(rows))
    assert list(token) == [int(vocab * v) for v in u]
    k = np.arange(1, rows + 1) * 7
    token = check(x, u, np.ones(rows), k=k)
    assert list(token) == [int(u[i] * k[i]) for i in range(rows)]
    check(x, u, np.ones(rows), p=np.linspace(0, 1, rows))
    check(x, u, np.ones(rows), mp=np.full(rows, 1.0))
    x[:, 100:300] = 4.0
    for n in (1, 150, 200, 201, 1000):
        check(x, u, np.ones(rows), k=np.full(rows, n))
        check(x, u, np.ones(rows), k=np.full(rows, n), p=np.full(rows, 0.5))


def test_few_values():
    # bf16 logits of a coarse grid: thresholds inside groups of equal values.
    rng = np.random.default_rng(3)
    rows, vocab = 48, 9001
    x = np.round(rng.standard_normal((rows, vocab)) * 2) / 2
    t, k, p, mp = settings(rng, rows, vocab)
    for bf16 in (False, True):
        check(x, rng.random(rows), t, k, p, mp, bf16=bf16)


def test_extremes():
    rng = np.random.default_rng(4)
    vocab, inf, nan = 3000, np.inf, np.nan
    base = rng.standard_normal(vocab)
    rows = []
    rows.append(np.full(vocab, -inf))                                  # nothing to choose from
    rows.append(np.full(vocab, nan))
    rows.append(np.where(np.arange(vocab) == 2999, -5.0, -inf))        # one token left by a mask
    rows.append(np.where(np.arange(vocab) % 7 == 3, base, -inf))
    rows.append(np.where(np.arange(vocab) % 5 == 3, nan, base))
    rows.append(np.where(np.arange(vocab) % 1000 == 17, inf, base))    # +inf takes the mass
    rows.append(np.where(np.arange(vocab) == 0, 3.4e38, -3.4e38))      # spans the whole range
    rows.append(np.where(np.arange(vocab) < 4, base, np.finfo(np.float32).min))  # a mask of the lowest value
    rows.append(np.where(np.arange(vocab) % 2, 0.0, -0.0))             # equal zeros
    rows.append(base * 1e-30)
    rows.append(base * 1e30)
    rows.append(base - 1e6)
    x = np.array(rows, dtype=np.float32)
    n = len(rows)
    for u in (0.0, 0.37, 0.9999999, 1.0, 5.0, -1.0):
        for t in (0.0, -1.0, nan, 1e-38, 0.05, 1.0, 100.0):
            check(x, np.full(n, u), np.full(n, t))
            check(x, np.full(n, u), np.full(n, t), k=np.full(n, 5), p=np.full(n, 0.8), mp=np.full(n, 0.05))
    check(x, np.full(n, 0.5), np.ones(n), k=np.full(n, vocab), p=np.full(n, 1.5), mp=np.full(n, -1.0))
    check(x, np.full(n, 0.5), np.ones(n), k=np.full(n, -3), p=np.full(n, 0.0), mp=np.full(n, 7.0))
    check(x, np.full(n, 0.5), np.ones(n), k=np.full(n, vocab - 1), p=np.full(n, 1e-30))


def test_frequencies():
    # Evenly spaced numbers hit each token in proportion to its probability, to one count.
    import torch
    from continuous_depth_batching_gb300 import ops
    rows, vocab = 4096, 37
    x = np.linspace(0, 3, vocab).astype(np.float32)[::-1].copy()
    s = ops.Sampler(rows, vocab)
    lg = torch.from_numpy(x).cuda().expand(rows, vocab).contiguous()
    u = (torch.arange(rows, device="cuda") / rows).float()
    token, _ = s(lg, u, torch.ones(rows, device="cuda"))
    p = np.exp(x.astype(np.float64))
    p /= p.sum()
    n = np.bincount(token.cpu().numpy(), minlength=vocab)
    assert np.all(np.abs(n - p * rows) <= 1.0 + 1e-9)


def test_replay_in_a_graph_and_side_stream():
    import torch
    from continuous_depth_batching_gb300 import ops
    rng = np.random.default_rng(8)
    rows, vocab = 6, 30000
    x = torch.from_numpy(rng.standard_normal((rows, vocab)).astype(np.float32)).cuda()
    u = torch.rand(rows, device="cuda")
    t = torch.ones(rows, device="cuda")
    p = torch.full((rows,), 0.9, device="cuda")
    plain = ops.Sampler(rows, vocab)
    want = [v.clone() for v in plain(x, u, t, top_p=p)]
    s = ops.Sampler(rows, vocab)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        s(x, u, t, top_p=p)
        with torch.cuda.graph(g, stream=side):
            out = s(x, u, t, top_p=p)
    torch.cuda.synchronize()
    for _ in range(3):
        s.token.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    u.copy_(torch.rand(rows, device="cuda"))
    g.replay()
    again = plain(x, u, t, top_p=p)
    torch.cuda.synchronize()
    assert torch.equal(out[0], again[0])


@pytest.mark.parametrize("near", [1, 2, 127, 128, 129, 300])
@pytest.mark.parametrize("vocab", [700, 20000])
def test_many_logits_close_together(near, vocab):
    """`near` logits a few ulps apart, some of them equal, behind a larger one: thresholds fall between and inside them."""
    rng = np.random.default_rng(near * 7 + vocab)
    rows = 16
    x = rng.standard_normal((rows, vocab)) - 9
    for i in range(rows):
        at = rng.permutation(vocab)[:near + 1]
        x[i, at[1:]] = 3.0 + rng.integers(0, max(1, near // 3), near) * 2.0 ** -21
        x[i, at[0]] = 4.0
    k = rng.integers(1, near + 2, rows)
    k[::3] = 0
    p = rng.uniform(0.1, 0.99, rows)
    p[1::3] = 1.0
    check(x, rng.random(rows), rng.uniform(0.5, 2.0, rows), k, p)


@pytest.mark.parametrize("vocab", [3000, 24001])
def test_bf16_rows_of_every_scale(vocab):
    """Rows in one or two thread blocks; thresholds among positive, negative, tiny, zero, equal and huge logits."""
    rng = np.random.default_rng(vocab)
    rows = 160
    x = rng.standard_normal((rows, vocab)) * 10.0 ** rng.uniform(-7, 4, (rows, 1))
    x += np.where(rng.random((rows, 1)) < 0.3, 10.0 ** rng.uniform(-2, 3, (rows, 1)) * rng.choice([-1, 1], (rows, 1)), 0)
    x[::7] = np.round(x[::7])
    x[3::11, ::2] = 0.0
    x[5::13, 1::3] = -np.inf
    x[6::17] = -1.25
    t = np.maximum(np.abs(x[np.isfinite(x).all(1)]).mean(), 1e-6) * 10.0 ** rng.uniform(-3, 1, rows)
    s = np.where(np.isfinite(x), x, 0).std(1) + 1e-3
    t = np.where(rng.random(rows) < 0.8, s * rng.uniform(0.1, 3, rows), t)
    p = rng.uniform(0.02, 0.999, rows)
    k = np.where(rng.random(rows) < 0.5, 0, rng.integers(1, 2 * vocab // 3, rows))
    k[1::5] = rng.integers(1, 60, len(k[1::5]))
    mp = np.where(rng.random(rows) < 0.8, 0, rng.uniform(0, 0.3, rows))
    check(x, rng.random(rows), t, k, p, mp, bf16=True)
    check(x[:, :vocab // 2], rng.random(rows), t, None, p, None, bf16=True, pad=3)
