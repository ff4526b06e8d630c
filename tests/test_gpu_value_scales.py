"""e4m3 attention where a row's value scales lie far apart, against float64.

Tolerance, per output element: test_gpu_cache_ops.py's bound on the scores, counted relative to the sum of
p_j |v_j| instead of the largest |v|.  A weight is off by 2^-17 (the exponent's argument is below 2^7 in magnitude and
is rounded by 2^-18 then; the exponential 2^-22) and, between numerator and sum, by twice what its score is off.  The
16-bit form of weight times scale is within 2^-22 of it or 2^-33 of the row's largest one, behind a shared prefix
(one fp16 number) within 2^-11 or 2^-33; times the code, added over the keys.  Sums are fp32: 2^-23 per step.  The
output is rounded by 2^-8.
"""

import numpy as np
import pytest

from tests.test_gpu_cache_ops import attention_case

pytestmark = pytest.mark.gpu


def bound(cs, row, scale):
    """(output [H, hd], tolerance) in float64."""
    import torch
    H, hk, hd, c = cs["H"], cs["hk"], cs["hd"], cs["cache"]
    s, L, d = int(cs["seq"][row]), int(cs["pos"][row]) + 1, int(cs["depth"][row])
    j = np.arange(L)
    blk, off = torch.from_numpy(cs["table"][s, j // 16]).long().cuda(), torch.from_numpy(j % 16).cuda()
    rep = lambda x: x.repeat_interleave(H // hk, 1)
    pool, sc = c.pool.view(torch.uint8)[blk, d, :, :, off].view(torch.float8_e4m3fn).double(), c.scales[blk, d, :, :, off].double()
    k, code, vs = rep(pool[:, 0] * sc[:, 0, :, None]), rep(pool[:, 1]), rep(sc[:, 1])
    q = cs["q"][row].double().view(H, hd)
    p = torch.softmax(torch.einsum("hd,lhd->hl", q, k) * scale, -1)
    w = p * vs.T
    o = torch.einsum("hl,lhd->hd", w, code)
    mass = torch.einsum("hl,lhd->hd", w.abs(), code.abs())
    S = torch.einsum("hd,lhd->hl", q.abs(), k.abs()).amax(1, keepdim=True) * abs(scale)
    part = 2.0 ** -11 if cs["shared"] else 2.0 ** -22
    rel = 2 * (hd * 2.0 ** -23 * S + 2.0 ** -17 + 2.0 ** -22) + part + (16 + L / 16 + L / 64) * 2.0 ** -23
    floor = 2.0 ** -33 * w.abs().amax(1, keepdim=True) * code.abs().sum(0)
    return o, 2.0 ** -8 * o.abs() + rel * mass + floor


def case(H, hk, hd, lengths, shared, keys, seed, q0=16.0):
    """A cache whose first key element decides the scores: `keys(L, rng)` gives, for the L keys of a row (in order),
    that element's score (natural logarithm) and the exponent of the value scale (None: a zero value)."""
    import torch
    cs = attention_case("e4m3", H, hk, hd, lengths, shared=shared, seed=seed)
    c, rng = cs["cache"], np.random.default_rng(seed)
    step = 2.0 ** -4
    cs["q"].view(len(lengths), H, hd)[..., 0] = q0
    cs["q"].view(len(lengths), H, hd)[..., 1:] /= 16
    raw = c.pool.view(torch.uint8)
    for i in range(len(lengths)):
        L = int(cs["pos"][i]) + 1
        score, ex = keys(L, rng)
        for j in range(L):
            b, o = int(cs["table"][int(cs["seq"][i]), j // 16]), j % 16
            if j < shared and i > 0:
                continue  # written with the first row
            c.scales[b, 0, 0, :, o] = step
            code = torch.tensor(score[j] * hd ** 0.5 / q0 / step).clamp(-448, 448).to(torch.float8_e4m3fn)
            raw[b, 0, 0, :, o] = torch.randn(hk, hd, generator=torch.Generator().manual_seed(j)).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
            raw[b, 0, 0, :, o, 0] = int(code.view(torch.uint8))
            if ex[j] is None:
                raw[b, 0, 1, :, o] = 0
                c.scales[b, 0, 1, :, o] = 2.0 ** -126
            else:
                c.scales[b, 0, 1, :, o] = 2.0 ** float(ex[j])
    return cs


def check(cs):
    import torch
    from continuous_depth_batching_gb300 import ops
    n = cs["q"].shape[0]
    at = ops.DecodeAttention(cs["cache"], cs["H"], n)
    out = at(cs["q"], cs["seq"], cs["pos"], shared_len=cs["shared"])
    at.check()
    for i in range(n):
        o, tol = bound(cs, i, cs["hd"] ** -0.5)
        err = (out[i].double().view(cs["H"], cs["hd"]) - o).abs()
        assert bool((err <= tol).all()), (i, float((err / tol).max()))


def loud(L, rng):
    """Keys of every second page: a value 2^26 as loud at a score of -30, which has no weight."""
    far = (np.arange(L) // 16 % 2 == 1) & (rng.random(L) < 0.3)
    return np.where(far, -30.0, rng.uniform(-1, 1, L)), np.where(far, 16, -10)


def sink(L, rng):
    """The first key takes all but 2^-22 of the weight and has a value of zero."""
    s = rng.uniform(-1, 1, L)
    ex = [-8.0] * L
    if L > 1:
        s[0], ex[0] = 15.0, None
    return s, ex


def far_sink(L, rng):
    """A zero value in the middle of the keys that is 2^75 times as heavy as the others."""
    s = rng.uniform(-1, 1, L)
    ex = list(rng.uniform(-12, -6, L).round())
    if L > 2:
        s[L // 2], ex[L // 2] = 52.0, None
    return s, ex


def spread(L, rng):
    """Scores and scales of many sizes, against each other."""
    s = rng.uniform(-20, 20, L)
    return s, (-s * rng.uniform(0.5, 1.8)).round()


def climb(L, rng):
    """Scores and scales that rise all along."""
    return np.linspace(-40, 40, L), np.linspace(-30, 20, L).round()


def fall(L, rng):
    s, ex = climb(L, rng)
    return s[::-1].copy(), ex[::-1].copy()


KINDS = [loud, sink, far_sink, spread, climb, fall]


@pytest.mark.parametrize("keys", KINDS)
@pytest.mark.parametrize("heads", [(4, 4, 64), (12, 2, 128), (6, 1, 96), (8, 4, 32), (20, 2, 64)])
def test_own_keys(keys, heads):
    check(case(*heads, [1, 40, 130, 300, 700], 0, keys, seed=heads[0]))


@pytest.mark.parametrize("keys", KINDS)
@pytest.mark.parametrize("heads", [(4, 4, 64), (12, 2, 128), (20, 2, 64), (8, 8, 128)])
def test_shared_prefix(keys, heads):
    for shared, lengths in ((48, [1, 40, 3]), (720, [20, 1, 90, 2, 33])):
        check(case(*heads, lengths, shared, keys, seed=heads[0] + shared))


def test_negative_scales():
    """A value's scale may be negative; its magnitude is what counts."""
    for shared, heads in ((0, (12, 2, 128)), (320, (8, 4, 64))):
        cs = case(*heads, [70, 20, 5], shared, climb, seed=3)
        cs["cache"].scales[:, :, 1, :, ::3] *= -1
        check(cs)
