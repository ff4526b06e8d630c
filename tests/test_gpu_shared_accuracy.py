"""Attention behind a shared prefix is as near to float64 as attention over a row's own keys.

Element by element, bf16 cache: test_gpu_cache_ops.py's tolerance for own keys as it is (two-part weights, 2^-17).
e4m3: beside it 2^-11 of sum p_j |v_j| for the one fp16 number that a weight times scale is.

Over all elements: rounding an output in [2^e, 2^(e+1)) to bf16 leaves up to 2^(e-8), in the mean square 2^(2e-16) / 3.
What comes before it is far less: weights to 2^-17 (fp16: 2^-11, 3% of the rounding's square), scores to some 2^-20.
So the squares add up to that, give or take the spread of a sum over n elements, 0.9 / sqrt(n) of it were all in one
binade and about twice that as they are: 3% for the 4096 elements and more asked for here, and 25% are allowed.  One
bf16 number per weight would add 2^-16 / 3 of the outputs' square, about as much again.
"""

import numpy as np
import pytest

from tests.test_gpu_cache_ops import attention_case, expected

pytestmark = pytest.mark.gpu


def mass(cs, row, scale):
    import torch
    H, hk, hd = cs["H"], cs["hk"], cs["hd"]
    s, j, d = int(cs["seq"][row]), np.arange(int(cs["pos"][row]) + 1), int(cs["depth"][row])
    blk, off = torch.from_numpy(cs["table"][s, j // 16]).long().cuda(), torch.from_numpy(j % 16).cuda()
    k, v = (cs["vals"][blk, d, n, :, off].repeat_interleave(H // hk, 1) for n in (0, 1))
    p = torch.softmax(torch.einsum("hd,lhd->hl", cs["q"][row].double().view(H, hd), k) * scale, -1)
    return torch.einsum("hl,lhd->hd", p, v.abs())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [(8, 2, 64), (16, 16, 128), (9, 3, 128), (24, 4, 64)])
@pytest.mark.parametrize("rows,shared", [(2, 16), (5, 64), (33, 112), (20, 1040), (140, 2064)])
def test_shared_prefix(dtype, heads, rows, shared):
    import torch
    from continuous_depth_batching_gb300 import ops
    rng = np.random.default_rng(rows)
    cs = attention_case(dtype, *heads, [int(v) for v in rng.integers(1, 60, rows)], shared=shared, seed=rows + heads[0])
    cs["q"] /= 16  # many keys with a weight: their roundings do not stand behind one that is 1
    scale = cs["hd"] ** -0.5
    out = ops.DecodeAttention(cs["cache"], cs["H"], rows)(cs["q"], cs["seq"], cs["pos"], shared_len=shared)
    square = rounding = 0.0
    for i in range(rows):
        o, tol = expected(cs, i, scale)
        if dtype == "e4m3":
            tol = tol + 2.0 ** -11 * mass(cs, i, scale)
        err = (out[i].double().view(o.shape) - o).abs()
        assert bool((err <= tol).all()), (i, float((err / tol).max()))
        square += float(err.square().sum())
        rounding += float(torch.exp2(2 * torch.floor(torch.log2(o.abs())) - 16).sum()) / 3
    if out.numel() >= 4096:
        assert square <= 1.25 * rounding, square / rounding
