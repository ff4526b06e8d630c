"""Operators of one decode step (include/cdb_ops.h) on PyTorch tensors.

For programs that drive the model themselves instead of through
``binding.Engine``.  Each class checks its arguments, keeps the argument
structure and the output buffers of its operator, and enqueues one call on the
current CUDA stream; nothing synchronizes, and every call can be captured into
a CUDA graph.  An object's default outputs and its workspace are overwritten by
its next call, so one object serves one stream at a time.  It may be called on
other streams than the one it was made on, and dropped while a call is in
flight: its own memory (default outputs, status, workspace) waits for every
stream that called it.  A graph that captured its calls needs the object for as
long as it is replayed.  Tensors that the caller gives are the caller's to
order and to keep.  An object works on the device that was current when it was
made; no gradients are recorded.
"""

from __future__ import annotations

import ctypes as C
import importlib.util
import os

from .binding import CdbError, lib

FP32, BF16, E4M3 = 0, 1, 2


class SampleArgs(C.Structure):
    _fields_ = [("rows", C.c_int), ("vocab", C.c_int), ("logits", C.c_void_p), ("dtype", C.c_int),
                ("ld", C.c_int64), ("u", C.c_void_p), ("temperature", C.c_void_p), ("top_k", C.c_void_p),
                ("top_p", C.c_void_p), ("min_p", C.c_void_p), ("token", C.c_void_p), ("logprob", C.c_void_p)]


class Cache(C.Structure):
    _fields_ = [("pool", C.c_void_p), ("scales", C.c_void_p), ("block_table", C.c_void_p), ("dtype", C.c_int),
                ("kv_blocks", C.c_int), ("n_kv_slots", C.c_int), ("n_kv_heads", C.c_int), ("head_dim", C.c_int),
                ("n_seqs", C.c_int), ("max_blocks", C.c_int)]


class CacheWriteArgs(C.Structure):
    _fields_ = [("cache", Cache), ("rows", C.c_int), ("n_heads", C.c_int), ("qkv", C.c_void_p), ("dtype", C.c_int),
                ("ldqkv", C.c_int64), ("q_gain", C.c_void_p), ("k_gain", C.c_void_p), ("eps", C.c_float),
                ("rope", C.c_void_p), ("rope_positions", C.c_int), ("rot_dim", C.c_int), ("seq", C.c_void_p),
                ("pos", C.c_void_p), ("depth", C.c_void_p), ("slot_base", C.c_int), ("q", C.c_void_p),
                ("ldq", C.c_int64), ("status", C.c_void_p)]


class AttentionArgs(C.Structure):
    _fields_ = [("cache", Cache), ("rows", C.c_int), ("n_heads", C.c_int), ("q", C.c_void_p), ("ldq", C.c_int64),
                ("seq", C.c_void_p), ("pos", C.c_void_p), ("depth", C.c_void_p), ("slot_base", C.c_int),
                ("scale", C.c_float), ("max_ctx", C.c_int), ("shared_len", C.c_int), ("out", C.c_void_p),
                ("ldo", C.c_int64), ("status", C.c_void_p), ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t)]


STATUS = {1: "block table entry out of range", 2: "slot out of range", 8: "sequence or position out of range",
          32: "bounded wait expired", 128: "rows do not share the prefix's blocks"}


def _lib():
    L = lib()
    if L.cdb_sample.argtypes is None:
        L.cdb_cache_write.argtypes = [C.c_void_p, C.c_void_p]
        L.cdb_attention.argtypes = [C.c_void_p, C.c_void_p]
        L.cdb_attention_workspace.restype = C.c_size_t
        L.cdb_attention_workspace.argtypes = [C.c_int] * 6
        L.cdb_ops_last_error.restype = C.c_char_p
        L.cdb_ops_last_error.argtypes = []
        L.cdb_sample.argtypes = [C.c_void_p, C.c_void_p]
    return L


_calls = None


def _tensor_calls():
    """The module of csrc/tensor_calls.cpp: checks of tensors and calls."""
    global _calls
    if _calls is None:
        import torch  # noqa: F401  (its libraries have to be loaded)

        from .build import CALLS
        if not os.path.exists(CALLS):
            raise RuntimeError(f"CDB library not built ({CALLS}); run continuous_depth_batching_gb300.build.build()")
        spec = importlib.util.spec_from_file_location("cdb_tensor_calls", CALLS)
        _calls = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(_calls)
    return _calls


class _Op:
    """Shared argument checks; the device is the current one when the object is made."""

    _at = 0  # handle of the last call's stream

    def __init__(self):
        import torch
        self._t = torch
        self.L = _lib()
        self.dev = torch.cuda.current_device()
        self._device, self._raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        self._streams = [torch.cuda.current_stream(self.dev)]  # the one it was made on, then others that called it
        self._memory = []  # the object's own tensors
        self._at = self._raw_stream(self.dev)

    def _bind(self, what, call):
        """The C entry point and the argument structure that self._call fills in."""
        self._what, self._call = what, getattr(_tensor_calls(), call)
        self._fn, self._ref = C.cast(getattr(self.L, what), C.c_void_p).value, C.addressof(self.args)

    def _stream(self):
        if self._device() != self.dev:
            raise ValueError(f"made on cuda:{self.dev}, the current device is cuda:{self._device()}")
        at = self._raw_stream(self.dev)
        if at != self._at:
            self._moved()
            self._at = at
        return at

    def _moved(self):
        """The first call on a stream: the object's memory is allocated and cleared on the stream it was made on."""
        t = self._t
        stream = t.cuda.current_stream(self.dev)
        if stream in self._streams:
            return
        if not t.cuda.is_current_stream_capturing():  # a capture starts behind all work of the device
            stream.wait_stream(self._streams[0])
        for m in self._memory:
            m.record_stream(stream)
        self._streams.append(stream)

    def _fail(self, rc):
        if rc is None:
            raise ValueError(f"{self._what}: a tensor has no memory or is a view that negates its values")
        raise CdbError(rc, f"{self._what}: {self.L.cdb_ops_last_error().decode()}")

    def _vec(self, name, t, dtype, n, needed=False):
        """Device pointer of a contiguous vector of at least n elements."""
        if t is None:
            if needed:
                raise ValueError(f"{name} is needed")
            return None
        if t.dtype is not dtype or t.get_device() != self.dev or t.numel() < n or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous {dtype} vector of at least {n} on cuda:{self.dev}, got "
                             f"{tuple(t.shape)} {t.dtype} on {t.device}")
        return t.data_ptr()

    def _mat(self, name, t, dtypes, rows, cols):
        """Device pointer and row stride of a [>= rows, >= cols] matrix with contiguous rows."""
        shape, stride = t.shape, t.stride()
        if (t.dtype not in dtypes or t.get_device() != self.dev or len(shape) != 2 or shape[0] < rows or
                shape[1] < cols or (stride[1] != 1 and shape[1] > 1) or (stride[0] < shape[1] and shape[0] > 1)):
            raise ValueError(f"{name}: expected [{rows}, {cols}] with contiguous rows, one behind another, of {dtypes} "
                             f"on cuda:{self.dev}, got {tuple(shape)} with strides {tuple(stride)} {t.dtype} on {t.device}")
        return t.data_ptr(), max(stride[0], shape[1])  # one row: its stride says nothing


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
        self._memory += [self.token, self.logprob]
        self.args = SampleArgs(vocab=self.vocab, token=self.token.data_ptr(), logprob=self.logprob.data_ptr())
        self._bind("cdb_sample", "sample")
        self._out = self.token, self.logprob  # of the last number of rows

    def __call__(self, logits, u, temperature, top_k=None, top_p=None, min_p=None):
        rc = self._call(self._fn, self._ref, self._stream(), self.dev, self.max_rows, logits, u, temperature, top_k,
                        top_p, min_p)
        if rc != 0:
            if rc is None:
                self._explain(logits, u, temperature, top_k, top_p, min_p)
            self._fail(rc)
        rows, out = logits.shape[0], self._out
        if out[0].shape[0] != rows:
            out = self._out = self.token[:rows], self.logprob[:rows]
        return out

    def _explain(self, logits, u, temperature, top_k, top_p, min_p):
        t, rows = self._t, logits.shape[0]
        if rows > self.max_rows or logits.shape[-1] != self.vocab:
            raise ValueError(f"logits {tuple(logits.shape)}: at most {self.max_rows} rows of {self.vocab}")
        self._mat("logits", logits, (t.float32, t.bfloat16), rows, self.vocab)
        self._vec("u", u, t.float32, rows, True)
        self._vec("temperature", temperature, t.float32, rows, True)
        self._vec("top_k", top_k, t.int32, rows)
        self._vec("top_p", top_p, t.float32, rows)
        self._vec("min_p", min_p, t.float32, rows)


class PagedCache:
    """A paged KV cache in the engine's layout, over tensors the caller owns.

    pool [kv_blocks, n_slots, 2, n_kv_heads, 16, head_dim], bfloat16 or float8_e4m3fn (then
    scales float32 of the pool's shape without its last axis); block_table int32
    [n_seqs, max_blocks].
    """

    def __init__(self, pool, block_table, scales=None):
        import torch
        if pool.dim() != 6 or pool.shape[2] != 2 or pool.shape[4] != 16 or not pool.is_contiguous():
            raise ValueError(f"pool: expected contiguous [kv_blocks, n_slots, 2, n_kv_heads, 16, head_dim], got "
                             f"{tuple(pool.shape)}")
        if pool.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError(f"pool: {pool.dtype}, expected bfloat16 or float8_e4m3fn")
        e4m3 = pool.dtype == torch.float8_e4m3fn
        if e4m3 != (scales is not None):
            raise ValueError("an e4m3 pool needs scales, a bf16 pool has none")
        if e4m3 and (scales.dtype != torch.float32 or scales.shape != pool.shape[:-1] or not scales.is_contiguous()):
            raise ValueError(f"scales: expected contiguous float32 {tuple(pool.shape[:-1])}, got {tuple(scales.shape)}")
        if block_table.dtype != torch.int32 or block_table.dim() != 2 or not block_table.is_contiguous():
            raise ValueError("block_table: expected contiguous int32 [n_seqs, max_blocks]")
        for t in (block_table,) + ((scales,) if e4m3 else ()):
            if t.device != pool.device:
                raise ValueError(f"pool is on {pool.device}, block_table or scales on {t.device}")
        if pool.device.type != "cuda":
            raise ValueError(f"pool is on {pool.device}, expected a CUDA device")
        self.pool, self.block_table, self.scales = pool, block_table, scales
        nb, ns, _, hk, _, hd = pool.shape
        self.n_kv_heads, self.head_dim, self.n_slots = hk, hd, ns
        self.max_ctx = 16 * block_table.shape[1]
        self.desc = Cache(pool.data_ptr(), scales.data_ptr() if e4m3 else None, block_table.data_ptr(),
                          E4M3 if e4m3 else BF16, nb, ns, hk, hd, block_table.shape[0], block_table.shape[1])


class _CacheOp(_Op):
    def __init__(self, cache, n_heads):
        super().__init__()
        if cache.pool.device.index != self.dev:
            raise ValueError(f"the cache is on {cache.pool.device}, the current device is cuda:{self.dev}")
        self.cache, self.n_heads = cache, int(n_heads)
        self.width = self.n_heads * cache.head_dim
        self.status = self._t.zeros(1, dtype=self._t.int32, device=cache.pool.device)
        self._memory.append(self.status)

    def _rows(self, rows, seq, pos, depth):
        for name, v, needed in (("seq", seq, True), ("pos", pos, True), ("depth", depth, False)):
            self._vec(name, v, self._t.int32, rows, needed)

    def check(self):
        """Wait for the object's calls, on whichever streams, and raise if one found an index out of range."""
        now = self._t.cuda.current_stream(self.dev)
        for s in self._streams:
            if s != now:
                now.wait_stream(s)
        st = int(self.status.item())
        if st:
            self.status.zero_()
            now.synchronize()  # before the next call, on whichever stream
            raise CdbError(-5, "; ".join(v for k, v in STATUS.items() if st & k) or f"status {st}")


class CacheWriter(_CacheOp):
    """Query / key norm, rotation and the cache write of a step's rows, in one pass (cdb_cache_write).

    qkv [rows, (n_heads + 2 n_kv_heads) head_dim] fp32 or bf16: query heads, key heads, value
    heads.  rope: float32 [positions, rot_dim / 2, 2] (cos, sin), see rope_table, or None;
    q_gain, k_gain: float32 [head_dim] norm weights, or None.  Returns the queries, bf16
    [rows, n_heads head_dim]; rows with seq < 0 are padding and left alone.
    """

    def __init__(self, cache, n_heads, rope=None, q_gain=None, k_gain=None, eps=1e-6):
        super().__init__(cache, n_heads)
        t = self._t
        a = self.args = CacheWriteArgs(cache=cache.desc, n_heads=self.n_heads, eps=eps)
        hd = cache.head_dim
        if (q_gain is None) != (k_gain is None):
            raise ValueError("q_gain and k_gain come together")
        a.q_gain, a.k_gain = self._vec("q_gain", q_gain, t.float32, hd), self._vec("k_gain", k_gain, t.float32, hd)
        if rope is not None:
            if (rope.dtype != t.float32 or rope.dim() != 3 or rope.shape[2] != 2 or not rope.is_contiguous() or
                    rope.device.index != self.dev):
                raise ValueError(f"rope: expected contiguous float32 [positions, rot_dim / 2, 2], got {tuple(rope.shape)}")
            a.rope, a.rope_positions, a.rot_dim = rope.data_ptr(), rope.shape[0], 2 * rope.shape[1]
        self._keep = (rope, q_gain, k_gain)
        a.status = self.status.data_ptr()
        self._bind("cdb_cache_write", "cache_write")

    def __call__(self, qkv, seq, pos, depth=None, slot_base=0, q_out=None):
        if q_out is None:
            q_out = self._t.zeros(qkv.shape[0], self.width, dtype=self._t.bfloat16, device=qkv.device)
        rc = self._call(self._fn, self._ref, self._stream(), self.dev, qkv, seq, pos, depth, slot_base, q_out)
        if rc != 0:
            if rc is None:
                t, rows = self._t, qkv.shape[0]
                self._mat("qkv", qkv, (t.float32, t.bfloat16), rows,
                          self.width + 2 * self.cache.n_kv_heads * self.cache.head_dim)
                self._rows(rows, seq, pos, depth)
                self._mat("q_out", q_out, (t.bfloat16,), rows, self.width)
            self._fail(rc)
        return q_out


class DecodeAttention(_CacheOp):
    """Attention of one query token per row over the paged cache (cdb_attention).

    q bf16 [rows, n_heads head_dim]; row i attends to positions 0..pos[i] of sequence seq[i]
    in slot slot_base + depth[i].  shared_len: positions that every row's sequence shares
    (same blocks), read once for all rows.  Rows with seq < 0 are left alone.  max_ctx bounds
    every position (+ 1), by default the whole block table; the workspace is sized for max_rows
    rows of it, and every call takes time for it, reached or not (128 rows of 1000 keys, 32/8
    heads: 82 us with max_ctx 1024, 252 us and 1.1 GB of workspace with 131072).  Give the
    longest row that its calls will see; objects of several lengths can share a cache.
    """

    def __init__(self, cache, n_heads, max_rows, max_ctx=None, scale=None):
        super().__init__(cache, n_heads)
        self.max_rows, self.max_ctx = int(max_rows), int(max_ctx or cache.max_ctx)
        hd = cache.head_dim
        n = self.L.cdb_attention_workspace(self.max_rows, self.n_heads, cache.n_kv_heads, hd, self.max_ctx, -1)
        if n == 0:
            raise ValueError(f"n_heads {n_heads}, max_rows {max_rows}, max_ctx {max_ctx}: not supported with "
                             f"{cache.n_kv_heads} KV heads of {hd}")
        t = self._t
        self.workspace = t.empty(n + 256, dtype=t.uint8, device=cache.pool.device)
        self._memory.append(self.workspace)
        base = (self.workspace.data_ptr() + 255) // 256 * 256
        self.args = AttentionArgs(cache=cache.desc, n_heads=self.n_heads, scale=hd ** -0.5 if scale is None else scale,
                                  max_ctx=self.max_ctx, status=self.status.data_ptr(), workspace=base,
                                  workspace_bytes=n)
        self._bind("cdb_attention", "attention")

    def __call__(self, q, seq, pos, depth=None, slot_base=0, shared_len=0, out=None):
        if out is None:
            out = self._t.zeros(q.shape[0], self.width, dtype=self._t.bfloat16, device=q.device)
        rc = self._call(self._fn, self._ref, self._stream(), self.dev, self.max_rows, q, seq, pos, depth, slot_base,
                        shared_len, out)
        if rc != 0:
            if rc is None:
                t, rows = self._t, q.shape[0]
                if rows > self.max_rows:
                    raise ValueError(f"{rows} rows, the workspace holds {self.max_rows}")
                self._mat("q", q, (t.bfloat16,), rows, self.width)
                self._rows(rows, seq, pos, depth)
                self._mat("out", out, (t.bfloat16,), rows, self.width)
            self._fail(rc)
        return out


def rope_table(positions, rot_dim, theta=10000.0, device="cuda"):
    """(cos, sin) of pos * theta^(-2j / rot_dim), float32 [positions, rot_dim / 2, 2], angles in float64."""
    import torch
    inv = theta ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()
