"""Two host threads that call one operator object: each call gets its own arguments.

The entry point is replaced by a callback, which runs while the first call has let go of the interpreter and makes the
second thread's call in between."""

import ctypes as C

from continuous_depth_batching_gb300 import ops
from tests.test_ops_arguments import attention_args, on_cpu, write_args


def interrupted(what, call, args, first, second, seen):
    """Arguments that the entry point finds for `first`, when `second` is called inside its call."""
    op = on_cpu(ops._Op, args)
    op._bind(what, call)
    inner = []

    @C.CFUNCTYPE(C.c_int, C.POINTER(type(args)), C.c_void_p)
    def entry(a, stream):
        if not inner:
            inner.append(1)
            run(second)
        else:
            inner.append(seen(a.contents))
            return 0
        inner.append(seen(a.contents))
        return 0

    def run(v):
        return op._call(C.cast(entry, C.c_void_p).value, op._ref, 0, -1, *v)

    assert run(first) == 0
    return inner[2], inner[1]


def test_arguments_of_interleaved_calls():
    import torch
    f = torch.ones(8)
    x, y = torch.zeros(8, 64), torch.zeros(3, 64)
    got = interrupted("cdb_sample", "sample", ops.SampleArgs(vocab=64), (8, x, f, f, None, None, None),
                      (8, y, f, f, None, None, None), lambda a: (a.rows, a.logits))
    assert got == ((8, x.data_ptr()), (3, y.data_ptr()))
    v = torch.zeros(8, dtype=torch.int32)
    x, y, q = torch.zeros(8, 1024), torch.zeros(2, 1024), torch.zeros(8, 512, dtype=torch.bfloat16)
    got = interrupted("cdb_cache_write", "cache_write", write_args(), (x, v, v, None, 0, q), (y, v, v, None, 1, q),
                      lambda a: (a.rows, a.qkv, a.slot_base))
    assert got == ((8, x.data_ptr(), 0), (2, y.data_ptr(), 1))
    x, y = torch.zeros(8, 512, dtype=torch.bfloat16), torch.zeros(5, 512, dtype=torch.bfloat16)
    got = interrupted("cdb_attention", "attention", attention_args(), (8, x, v, v, None, 0, 16, q),
                      (8, y, v, v, None, 0, 32, q), lambda a: (a.rows, a.q, a.shared_len))
    assert got == ((8, x.data_ptr(), 16), (5, y.data_ptr(), 32))
