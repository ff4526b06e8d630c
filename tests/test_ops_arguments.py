"""Refusals of the decode-step operators: C entry points, before any CUDA call."""

import ctypes as C

import pytest

from continuous_depth_batching_gb300 import ops

ARG = -1


@pytest.fixture(scope="module")
def L():
    return ops._lib()


def sample_args(**kw):
    p = 0x1000  # never dereferenced: the call is refused
    a = ops.SampleArgs(rows=4, vocab=100, logits=p, dtype=0, ld=100, u=p, temperature=p, token=p)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(vocab=0), dict(vocab=262145, ld=262145), dict(ld=99), dict(dtype=2),
                                 dict(dtype=-1), dict(logits=None), dict(u=None), dict(temperature=None),
                                 dict(token=None), dict(logits=0x1002), dict(rows=(1 << 31) - 1)])
def test_sample_refuses(L, bad):
    assert L.cdb_sample(C.byref(sample_args(**bad)), None) == ARG
    assert L.cdb_ops_last_error()


def test_sample_refuses_no_arguments(L):
    assert L.cdb_sample(None, None) == ARG


def test_sample_takes_an_empty_batch(L):
    assert L.cdb_sample(C.byref(sample_args(rows=0)), None) == 0
    assert L.cdb_ops_last_error() == b""
