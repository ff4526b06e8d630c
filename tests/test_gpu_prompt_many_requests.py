"""Prompt and draft attention of more than 32 requests in calls whose keys are cut: items are found by all threads of a
CTA, in one round of them or two.  Against float64, with the tolerances of tests/test_gpu_prompt_attention.py."""

import numpy as np
import pytest

from tests.test_gpu_prompt_attention import check, make, tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])  # 384 and 512 threads
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("requests,hk,hd", [(33, 2, 128), (33, 1, 32), (100, 2, 96), (100, 1, 128), (450, 1, 64), (560, 1, 32)])
def test_cut_keys_of_many_requests(dtype, draft, requests, hk, hd):
    rng = np.random.default_rng(requests + hd)
    counts = rng.integers(0, 5, requests)
    cached = rng.integers(0, 200, requests)
    long = rng.permutation(requests)[:5]
    counts[long] = 3, 40, 64, 1, 7
    cached[long] = 20000, 5000, 300, 9000, 1000
    counts[-1], cached[-1] = 2, 2000
    group = 4
    assert hk * (counts.sum() // (2 * (128 // group)) + requests) < 608  # such calls are cut
    cs = make(dtype, group * hk, hk, hd, counts, cached, seed=requests, **(dict(mask=tree) if draft else {}))
    some = set(range(0, requests, 11)) | set(int(i) for i in long) | {requests - 1}
    check(cs, requests=sorted(some))
