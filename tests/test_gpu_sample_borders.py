"""Sampling where a border falls beside the key of -0, against the float64 restatement of test_gpu_sample.py.

Tokens must be equal, log probabilities within that file's bound.
"""

import numpy as np
import pytest

from tests.test_gpu_sample import check

pytestmark = pytest.mark.gpu


def zero_rows(rng, rows, vocab, negative):
    """Few positive logits of a value of their own in [4, 8) per row (every bf16 number of it in 128 rows), zeros,
    logits `negative(n)` just below them, and a far rest; with the number of logits >= 0."""
    x = np.full((rows, vocab), -10.0)
    top = 4 + np.arange(rows) % 128 / 32
    n0 = rng.integers(130, 300, rows)
    for i in range(rows):
        at = rng.permutation(vocab)
        x[i, at[:3]] = top[i]
        x[i, at[3:3 + n0[i]]] = 0.0
        x[i, at[600:900]] = negative(300)
    return x, n0 + 3


@pytest.mark.parametrize("vocab", [2048, 9000])
@pytest.mark.parametrize("bf16", [False, True])
def test_top_k_ends_with_the_zeros(vocab, bf16):
    rng = np.random.default_rng(vocab)
    rows = 256
    for n, negative in enumerate((lambda n: np.full(n, -0.001), lambda n: -0.25 * rng.random(n) - 2.0 ** -20)):
        x, k = zero_rows(rng, rows, vocab, negative)
        u, t = rng.random(rows), np.full(rows, 10.0)
        check(x, u, t, k=k, bf16=bf16)
        check(x, u, t, k=k, p=np.full(rows, 0.97), bf16=bf16)
        check(x, u, t, k=k + rng.integers(-1, 2, rows), bf16=bf16)


def test_zeros_behind_one_large_logit():
    x = np.concatenate([[7.0], np.zeros(300), np.full(300, -0.01), [-7.0]])[None]
    for bf16 in (False, True):
        for u in (0.0, 0.01, 0.5, 0.99):
            check(x, [u], [10.0], k=[301], bf16=bf16)
            check(x, [u], [10.0], k=[301], p=[0.9], bf16=bf16)


@pytest.mark.parametrize("bf16", [False, True])
def test_thresholds_among_subnormal_logits(bf16):
    # Keys next to the one of -0, on both sides: a group of keys can end there.
    rng = np.random.default_rng(5)
    rows, vocab = 256, 2048
    size = 2.0 ** -133 if bf16 else 2.0 ** -149
    most = 32 if bf16 else 1 << 22
    x, k = zero_rows(rng, rows, vocab, lambda n: -size * rng.integers(1, most, n))
    x[:, ::9] = np.where(x[:, ::9] == 0, size * rng.integers(1, most, x[:, ::9].shape), x[:, ::9])
    more = rng.integers(1, 299, rows)
    u, t = rng.random(rows), np.full(rows, 10.0)
    check(x, u, t, k=k + more, bf16=bf16)
    check(x, u, t, k=k + more, p=rng.uniform(0.5, 0.999, rows), bf16=bf16)
    check(x, u, t, p=rng.uniform(0.05, 0.7, rows), bf16=bf16)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("vocab", [700, 20000])
def test_u_zero_takes_a_far_tie_of_top_k(vocab, bf16):
    # The ties weigh e^-50 of the largest logit, far below the unit of the masses, and one of them is the first token kept.
    rows = 8
    x = np.full((rows, vocab), -200.0)
    x[:, 5::7] = -50.0
    x[:, [40, 300]] = 0.0
    k = np.array([1, 2, 3, 4, 5, 40, 99, 102])  # the two largest, then ties
    token = check(x, np.zeros(rows), np.ones(rows), k=k, bf16=bf16)
    # Of 700 tokens 99 are ties (index 40, the 100th, holds one of the largest): the 102nd token kept is then one of -200, index 0.
    assert list(token) == [40, 40] + [5] * 5 + [0 if vocab == 700 else 5]
    check(x, np.full(rows, -1.0), np.ones(rows), k=k, p=np.full(rows, 1.0), bf16=bf16)
    token = check(x, np.zeros(rows), np.full(rows, 0.05), k=k, bf16=bf16)  # e^-1000: no weight left
    assert list(token) == [40] * 8
    assert list(check(x, np.zeros(rows), np.ones(rows), k=k, mp=np.full(rows, 1e-9), bf16=bf16)) == [40] * 8


@pytest.mark.parametrize("bf16", [False, True])
def test_u_zero_keeps_to_a_tiny_min_p(bf16):
    # min_p below the unit of the masses still rules out what weighs less: e^-60 < 1e-20 < e^-40.
    rows = 5
    x = np.full((rows, 3000), -60.0)
    x[:, 100:200] = -40.0
    x[:, 2000] = 0.0
    mp = np.array([1e-20, 1e-30, 1e-10, 1e-44, 0.0])
    token = check(x, np.zeros(rows), np.ones(rows), mp=mp, bf16=bf16)
    assert list(token) == [100, 0, 2000, 0, 0]
    # With top_k too, whose threshold is a tie.
    token = check(x, np.zeros(rows), np.ones(rows), k=np.full(rows, 150), mp=mp, bf16=bf16)
    assert list(token) == [100, 0, 2000, 0, 0]
    check(x, np.full(rows, 0.5), np.ones(rows), mp=mp, bf16=bf16)
