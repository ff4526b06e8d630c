"""Operators of one decode step (include/cdb_ops.h) on PyTorch tensors.

For programs that drive the model themselves instead of through
``binding.Engine``.  Each class checks its arguments, keeps the argument
structure and the output buffers of its operator, and enqueues one call on the
current CUDA stream; nothing synchronizes, and every call can be captured into
a CUDA graph.  An object's default outputs are overwritten by its next call,
so one object serves one stream at a time.
"""

from __future__ import annotations

import ctypes as C

from .binding import CdbError, lib

FP32, BF16, E4M3 = 0, 1, 2


class SampleArgs(C.Structure):
    _fields_ = [("rows", C.c_int), ("vocab", C.c_int), ("logits", C.c_void_p), ("dtype", C.c_int),
                ("ld", C.c_int64), ("u", C.c_void_p), ("temperature", C.c_void_p), ("top_k", C.c_void_p),
                ("top_p", C.c_void_p), ("min_p", C.c_void_p), ("token", C.c_void_p), ("logprob", C.c_void_p)]


def _lib():
    L = lib()
    if L.cdb_sample.argtypes is None:
        L.cdb_ops_last_error.restype = C.c_char_p
        L.cdb_ops_last_error.argtypes = []
        L.cdb_sample.argtypes = [C.c_void_p, C.c_void_p]
    return L


def _fail(L, rc, what):
    raise CdbError(rc, f"{what}: {L.cdb_ops_last_error().decode()}")


class _Op:
    """Shared argument checks; the device is the current one when the object is made."""

    def __init__(self):
        import torch
        self._t = torch
        self.L = _lib()
        self.dev = torch.cuda.current_device()

    def _stream(self):
        return self._t.cuda.current_stream(self.dev).cuda_stream

    def _vec(self, name, t, dtype, n):
        """Device pointer of a contiguous vector of at least n elements."""
        if t is None:
            return None
        if t.dtype != dtype or t.device.index != self.dev or t.dim() != 1 or t.shape[0] < n or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous {dtype} vector of at least {n} on cuda:{self.dev}, got "
                             f"{tuple(t.shape)} {t.dtype} on {t.device}")
        return t.data_ptr()

    def _mat(self, name, t, dtypes, rows, cols):
        """Device pointer and row stride of a [>= rows, >= cols] matrix with contiguous rows."""
        if (t.dtype not in dtypes or t.device.index != self.dev or t.dim() != 2 or t.shape[0] < rows or
                t.shape[1] < cols or (t.stride(1) != 1 and t.shape[1] > 1)):
            raise ValueError(f"{name}: expected [{rows}, {cols}] with contiguous rows of {dtypes} on cuda:{self.dev}, "
                             f"got {tuple(t.shape)} {t.dtype} on {t.device}")
        return t.data_ptr(), max(t.stride(0), t.shape[1])


class Sampler(_Op):
    """Temperature, top-k, top-p and min-p sampling from given uniform numbers (cdb_sample).

    One token per row of logits [rows, vocab] (fp32 or bf16, rows may be strided); u,
    temperature, top_p, min_p float32 [rows], top_k int32 [rows], the filters None for off.
    A temperature that is not > 0 takes the argmax.  Returns (token int32 [rows], logprob
    float32 [rows]); a row with nothing to choose from gets token -1, logprob -inf.
    """

    def __init__(self, max_rows, vocab):
        super().__init__()
        t = self._t
        if max_rows < 1:
            raise ValueError("max_rows must be >= 1")
        self.max_rows, self.vocab = int(max_rows), int(vocab)
        self.token = t.empty(self.max_rows, dtype=t.int32, device=f"cuda:{self.dev}")
        self.logprob = t.empty(self.max_rows, dtype=t.float32, device=f"cuda:{self.dev}")
        self.args = SampleArgs(vocab=self.vocab)
        self._ref = C.byref(self.args)

    def __call__(self, logits, u, temperature, top_k=None, top_p=None, min_p=None):
        t, a = self._t, self.args
        rows = logits.shape[0]
        if rows > self.max_rows or logits.shape[-1] != self.vocab:
            raise ValueError(f"logits {tuple(logits.shape)}: at most {self.max_rows} rows of {self.vocab}")
        a.rows = rows
        a.logits, a.ld = self._mat("logits", logits, (t.float32, t.bfloat16), rows, self.vocab)
        a.dtype = BF16 if logits.dtype == t.bfloat16 else FP32
        a.u = self._vec("u", u, t.float32, rows)
        a.temperature = self._vec("temperature", temperature, t.float32, rows)
        a.top_k = self._vec("top_k", top_k, t.int32, rows)
        a.top_p = self._vec("top_p", top_p, t.float32, rows)
        a.min_p = self._vec("min_p", min_p, t.float32, rows)
        a.token, a.logprob = self.token.data_ptr(), self.logprob.data_ptr()
        rc = self.L.cdb_sample(self._ref, self._stream())
        if rc != 0:
            _fail(self.L, rc, "cdb_sample")
        return self.token[:rows], self.logprob[:rows]
