"""The sines and cosines of the rotation (cdb_rotate), read off by turning (1, 0) and (0, 1) in fp32.

Tolerance: an angle is an exact 64-bit fraction of a turn; its distance from the nearest quarter of a turn, at most 1/8 turn or
1/4 half turn, is rounded to fp32, by 2^-27 half turns at most, hence pi 2^-27 in sine and cosine.  These are within one ulp,
at most 2^-24 below 1.  A factor rounds once more, 2^-24 of the product."""

import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("far", [5000, 2 ** 31 - 5000])
@pytest.mark.parametrize("factor", [1.0, -0.75])
def test_sines_and_cosines(inter, far, factor):
    import torch
    from continuous_depth_batching_gb300 import ops
    hd, rows = 128, 5000
    steps, _ = ops.rope_steps(hd, theta=50000.0)
    pos = np.arange(far - rows, far, dtype=np.int64)
    # quarters of a turn, exactly: 1/4, 1/2, 1/8 and 3/8 of a turn a position
    steps[:4] = torch.tensor([1 << 62, -(1 << 63), 1 << 61, 3 << 61], device="cuda")
    x = torch.zeros(rows, 2 * hd, device="cuda")
    one = torch.arange(0, hd, 2) if inter else torch.arange(hd // 2)
    two = one + (1 if inter else hd // 2)
    x[:, one], x[:, hd + two] = 1.0, 1.0
    op = ops.Rotary(1, 1, hd, steps, interleaved=inter, factor=factor)
    got = op(x, torch.tensor(pos, dtype=torch.int32, device="cuda")).double().cpu().numpy()
    with np.errstate(over="ignore"):
        phase = steps.cpu().numpy().view(np.uint64)[None] * pos.astype(np.uint64)[:, None]
    a = 2 * math.pi * (phase.view(np.int64).astype(np.float64) / 2.0 ** 64)
    c, s = np.cos(a) * factor, np.sin(a) * factor
    tol = abs(factor) * (math.pi * 2.0 ** -27 + 2.0 ** -24) + (0 if factor == 1 else 2.0 ** -24 * abs(factor)) + 2.0 ** -50
    for have, want in ((got[:, one], c), (got[:, two], s), (got[:, hd + one], -s), (got[:, hd + two], c)):
        err = np.abs(have - want)
        assert err.max() <= tol, (err.max() / tol, np.unravel_index(err.argmax(), err.shape))
    # at whole quarters the numbers are exact
    q = np.round(a[:, :2] / (math.pi / 2)).astype(int) % 4
    assert np.array_equal(got[:, one[:2]], np.array([1, 0, -1, 0])[q] * factor)
    assert np.array_equal(got[:, two[:2]], np.array([0, 1, 0, -1])[q] * factor)
