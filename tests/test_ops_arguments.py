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


def cache_desc(**kw):
    c = ops.Cache(pool=0x1000, scales=0x1000, block_table=0x1000, dtype=2, kv_blocks=8, n_kv_slots=1, n_kv_heads=4,
                  head_dim=64, n_seqs=2, max_blocks=4)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


CACHE_BAD = [dict(dtype=0), dict(dtype=3), dict(head_dim=48), dict(head_dim=256), dict(kv_blocks=0), dict(n_kv_slots=0),
             dict(n_kv_heads=0), dict(n_seqs=0), dict(max_blocks=0), dict(pool=None), dict(pool=0x1008),
             dict(block_table=None), dict(scales=None), dict(scales=0x1004), dict(max_blocks=1 << 28)]


def write_args(**kw):
    p = 0x1000
    a = ops.CacheWriteArgs(cache=cache_desc(), rows=3, n_heads=8, qkv=p, dtype=0, ldqkv=1024, q_gain=p, k_gain=p, eps=1e-6,
                           rope=p, rope_positions=64, rot_dim=64, seq=p, pos=p, q=p, ldq=512)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [dict(cache=cache_desc(**b)) for b in CACHE_BAD] +
                         [dict(rows=-1), dict(n_heads=0), dict(dtype=2), dict(ldqkv=1023), dict(ldqkv=1026), dict(qkv=None),
                          dict(qkv=0x1004), dict(q=None), dict(q=0x1002), dict(ldq=504), dict(ldq=516), dict(q_gain=None),
                          dict(k_gain=None), dict(q_gain=0x1004), dict(eps=-1.0), dict(eps=float("nan")), dict(rot_dim=8),
                          dict(rot_dim=24), dict(rot_dim=80), dict(rot_dim=0), dict(rope_positions=0), dict(rope=0x1008),
                          dict(seq=None), dict(pos=None)])
def test_cache_write_refuses(L, bad):
    assert L.cdb_cache_write(C.byref(write_args(**bad)), None) == ARG
    assert L.cdb_ops_last_error()


def attention_args(**kw):
    p = 0x1000
    a = ops.AttentionArgs(cache=cache_desc(), rows=3, n_heads=8, q=p, ldq=512, seq=p, pos=p, scale=0.125, max_ctx=64, out=p,
                          ldo=512, workspace=p, workspace_bytes=1 << 30)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [dict(cache=cache_desc(**b)) for b in CACHE_BAD] +
                         [dict(rows=-1), dict(rows=(1 << 31) - 1), dict(n_heads=0), dict(n_heads=6), dict(q=None), dict(q=0x1008),
                          dict(ldq=504), dict(ldq=516), dict(out=None), dict(out=0x1002), dict(ldo=504), dict(ldo=518),
                          dict(seq=None), dict(pos=None), dict(max_ctx=0), dict(max_ctx=65), dict(shared_len=8),
                          dict(shared_len=-16), dict(shared_len=80), dict(shared_len=16, depth=0x1000),
                          dict(workspace=None), dict(workspace=0x1010), dict(workspace_bytes=0),
                          dict(cache=cache_desc(kv_blocks=1 << 25))])
def test_attention_refuses(L, bad):
    assert L.cdb_attention(C.byref(attention_args(**bad)), None) == ARG
    assert L.cdb_ops_last_error()


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_attention_refuses_scales_that_are_not_finite(L, scale):
    assert L.cdb_attention(C.byref(attention_args(scale=scale)), None) == ARG
    assert b"scale" in L.cdb_ops_last_error()


def test_empty_batches(L):
    assert L.cdb_sample(C.byref(sample_args(rows=0, logits=None, u=None, token=None)), None) == 0
    assert L.cdb_attention(C.byref(attention_args(rows=0, q=None, seq=None, workspace=None, workspace_bytes=0)), None) == 0
    assert L.cdb_cache_write(C.byref(write_args(rows=0)), None) == 0
    assert L.cdb_attention(C.byref(attention_args(rows=0)), None) == 0


def test_attention_workspace_sizes(L):
    assert L.cdb_attention_workspace(4, 8, 3, 64, 100, 0) == 0   # heads do not divide
    assert L.cdb_attention_workspace(4, 8, 8, 64, 100, 8) == 0
    one, two = (L.cdb_attention_workspace(r, 8, 8, 128, 4096, 0) for r in (1, 2))
    assert 0 < one < two <= 2 * one
    any_prefix = L.cdb_attention_workspace(64, 16, 4, 128, 4096, -1)
    for rows in (1, 2, 3, 31, 32, 33, 64):
        for shared in range(0, 4097, 16):
            assert L.cdb_attention_workspace(rows, 16, 4, 128, 4096, shared) <= any_prefix


def test_matrices_whose_rows_overlap_are_refused():
    """A broadcast row has stride 0, which the operators' row stride cannot say."""
    import torch
    op = object.__new__(ops._Op)
    op.dev = -1  # where CPU tensors are
    x = torch.zeros(4, 32)
    assert op._mat("x", x, (torch.float32,), 4, 32) == (x.data_ptr(), 32)
    assert op._mat("x", x[:, :24], (torch.float32,), 4, 24) == (x.data_ptr(), 32)
    assert op._mat("x", x[:1].expand(1, 32), (torch.float32,), 1, 32)[1] == 32
    for bad in (x[:1].expand(4, 32), x.as_strided((4, 32), (16, 1)), x.t(), x[0], x[:, ::2]):
        with pytest.raises(ValueError):
            op._mat("x", bad, (torch.float32,), bad.shape[0], bad.shape[-1])


def on_cpu(cls, args, **attrs):
    """An operator object whose device is the CPU; its argument structure is one that the C call refuses."""
    op = object.__new__(cls)
    import torch
    op._t, op.L, op.dev, op.args = torch, ops._lib(), -1, args
    op._device, op._raw_stream = lambda: -1, lambda dev: 0
    for k, v in attrs.items():
        setattr(op, k, v)
    return op


def test_sampler_checks_its_tensors():
    import torch
    op = on_cpu(ops.Sampler, ops.SampleArgs(vocab=64), max_rows=8, vocab=64)  # no output: refused
    op._bind("cdb_sample", "sample")
    f, i = torch.zeros(8), torch.zeros(8, dtype=torch.int32)
    x = torch.zeros(8, 80)[:, :64]
    for logits in (x, x.bfloat16(), x[:5], x[7:]):
        with pytest.raises(ops.CdbError, match="are needed"):
            op(logits, f, f, i, f, None)
        a = op.args
        assert (a.rows, a.logits, a.ld) == (logits.shape[0], logits.data_ptr(), max(logits.stride(0), 64))
        assert a.dtype == (logits.dtype is torch.bfloat16)
        assert (a.u, a.temperature, a.top_k, a.top_p, a.min_p) == (f.data_ptr(),) * 2 + (i.data_ptr(), f.data_ptr(), None)
    for bad in (x[:, :63], torch.zeros(9, 64), x.half(), x[0], x[:1].expand(4, 64), x.t().contiguous().t(), torch.zeros(8, 65)):
        with pytest.raises(ValueError):
            op(bad, f, f)
    for bad in (f[:7], f.double(), f.repeat(2)[::2], i, None):
        for args in ((bad, f), (f, bad), (f, f, i, bad) if bad is not None else (bad, f)):
            with pytest.raises(ValueError):
                op(x, *args)
    for bad in (f, i[:3], i.long()):
        with pytest.raises(ValueError):
            op(x, f, f, bad)
    with pytest.raises(ValueError):
        op(torch._neg_view(x), f, f)
    with pytest.raises((TypeError, AttributeError)):
        op([1.0], f, f)


def test_cache_operators_check_their_tensors():
    import torch
    cache = ops._CacheOp.__new__(ops._CacheOp)
    cache.n_kv_heads, cache.head_dim = 4, 64
    wr = on_cpu(ops.CacheWriter, write_args(eps=-1.0), cache=cache, width=512)  # refused behind the tensors' checks
    at = on_cpu(ops.DecodeAttention, attention_args(workspace=None), cache=cache, width=512, max_rows=8)
    wr._bind("cdb_cache_write", "cache_write")
    at._bind("cdb_attention", "attention")
    qkv, q, v = torch.zeros(8, 1032), torch.zeros(8, 520, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32)
    for n in (8, 5, 1):
        with pytest.raises(ops.CdbError, match="eps"):
            wr(qkv[:n], v, v, None, 3, q)
        a = wr.args
        assert (a.rows, a.qkv or 0, a.ldqkv, a.dtype) == (n, qkv[:n].data_ptr(), 1032, 0)
        assert (a.seq, a.pos, a.depth, a.slot_base, a.q, a.ldq) == (v.data_ptr(), v.data_ptr(), None, 3, q.data_ptr(), 520)
    for n in (8, 5, 1):
        with pytest.raises(ops.CdbError, match="workspace"):
            at(q[:n, :512], v, v, None, 0, 32, q)
        a = at.args
        assert (a.rows, a.q, a.ldq, a.seq, a.pos, a.depth) == (n, q.data_ptr(), 520, v.data_ptr(), v.data_ptr(), None)
        assert (a.slot_base, a.shared_len, a.out, a.ldo) == (0, 32, q.data_ptr(), 520)
    for bad in (qkv[:, :1023], qkv.double(), qkv[:1].expand(8, 1032), qkv[0], torch.zeros(1032, 8).t()):
        with pytest.raises(ValueError):
            wr(bad, v, v, q_out=q)
    for bad in (q[:, :511], q.float(), q[:1].expand(8, 520), q[:7]):
        with pytest.raises(ValueError):
            wr(qkv, v, v, q_out=bad)
        with pytest.raises(ValueError):
            at(q, v, v, out=bad)
    for bad in (q[:, :511], q.float(), q[:1].expand(8, 520), torch.zeros(9, 512, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            at(bad, v, v, out=torch.zeros(9, 512, dtype=torch.bfloat16))
    for bad in (v[:7], v.long(), v.repeat(2)[::2], v.float()):
        for args in ((bad, v), (v, bad), (v, v, bad)):
            with pytest.raises(ValueError):
                wr(qkv, *args, q_out=q)
            with pytest.raises(ValueError):
                at(q, *args, out=q)
    with pytest.raises(ValueError, match="seq is needed"):
        wr(qkv, None, v, q_out=q)
    for call in (lambda: wr(qkv, v, v, None, 1 << 40, q), lambda: at(q, v, v, None, 0, 1 << 31, q)):
        with pytest.raises(OverflowError):
            call()
