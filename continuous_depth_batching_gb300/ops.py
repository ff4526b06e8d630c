"""Operators of a step (include/cdb_ops.h) on PyTorch tensors.

For programs that drive the model themselves instead of through
``binding.Engine``.  Each class checks its arguments, keeps the argument
structure of its operator, its workspace and what it returns (the tokens of
Sampler, the rows of PagePlanner), and enqueues one call on the current CUDA
stream; nothing synchronizes, and every call can be captured into a CUDA graph.
What an object keeps is overwritten by its next call, so one object serves one
stream at a time.  CacheWriter and the attentions keep no output: without q_out
or out they allocate a new tensor of zeros in every call, which costs a pass
over it (8192 rows of 32 heads of 128: 67 MB), so give one where time counts.
An object may be called on other streams than the one it was made on, and
dropped while a call is in flight: its own memory (what it returns, status,
workspace) waits for every stream that called it.  A graph that captured its
calls needs the object for as long as it is replayed.  Tensors that the caller
gives are the caller's to order and to keep.  An object works on the device
that was current when it was made; no gradients are recorded.
"""

from __future__ import annotations

import ctypes as C
import importlib.util
import math
import os
from collections import namedtuple

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


class PlanPagesArgs(C.Structure):
    _fields_ = [("requests", C.c_int), ("lens", C.c_void_p), ("new_tokens", C.c_void_p), ("seq", C.c_void_p),
                ("block_table", C.c_void_p), ("n_seqs", C.c_int), ("max_blocks", C.c_int), ("free_blocks", C.c_void_p),
                ("free_slots", C.c_int), ("state", C.c_void_p), ("state_out", C.c_void_p), ("lens_out", C.c_void_p),
                ("row_start", C.c_void_p), ("row_seq", C.c_void_p), ("row_pos", C.c_void_p), ("row_slot", C.c_void_p),
                ("max_rows", C.c_int), ("status", C.c_void_p)]


class RotateArgs(C.Structure):
    _fields_ = [("rows", C.c_int), ("n_heads", C.c_int), ("n_kv_heads", C.c_int), ("head_dim", C.c_int), ("x", C.c_void_p),
                ("dtype", C.c_int), ("ldx", C.c_int64), ("pos", C.c_void_p), ("steps", C.c_void_p), ("rot_dim", C.c_int),
                ("interleaved", C.c_int), ("factor", C.c_float), ("q_gain", C.c_void_p), ("k_gain", C.c_void_p),
                ("eps", C.c_float), ("out", C.c_void_p), ("ldo", C.c_int64)]


class PromptAttentionArgs(C.Structure):
    _fields_ = [("cache", Cache), ("rows", C.c_int), ("n_heads", C.c_int), ("q", C.c_void_p), ("ldq", C.c_int64),
                ("requests", C.c_int), ("row_start", C.c_void_p), ("lens", C.c_void_p), ("seq", C.c_void_p),
                ("slot", C.c_int), ("scale", C.c_float), ("max_ctx", C.c_int), ("visible", C.c_void_p),
                ("mask_words", C.c_int), ("out", C.c_void_p), ("ldo", C.c_int64), ("status", C.c_void_p),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t)]


class KeepPathArgs(C.Structure):
    _fields_ = [("cache", Cache), ("requests", C.c_int), ("base", C.c_void_p), ("path", C.c_void_p), ("ld_path", C.c_int64),
                ("max_path", C.c_int), ("keep", C.c_void_p), ("seq", C.c_void_p), ("status", C.c_void_p)]


STATUS = {1: "block table entry out of range", 2: "slot out of range", 8: "sequence or position out of range",
          32: "bounded wait expired", 128: "rows do not share the prefix's blocks", 256: "too few free blocks",
          512: "more new tokens than rows"}


def _lib():
    L = lib()
    if L.cdb_sample.argtypes is None:
        L.cdb_cache_write.argtypes = [C.c_void_p, C.c_void_p]
        L.cdb_attention.argtypes = [C.c_void_p, C.c_void_p]
        L.cdb_attention_workspace.restype = C.c_size_t
        L.cdb_attention_workspace.argtypes = [C.c_int] * 6
        L.cdb_ops_last_error.restype = C.c_char_p
        L.cdb_ops_last_error.argtypes = []
        L.cdb_prompt_attention_workspace.restype = C.c_size_t
        L.cdb_prompt_attention_workspace.argtypes = [C.c_int] * 6
        for f in (L.cdb_plan_pages, L.cdb_rotate, L.cdb_prompt_attention, L.cdb_draft_attention, L.cdb_keep_path):
            f.argtypes = [C.c_void_p, C.c_void_p]
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


class _StatusOp(_Op):
    """An operator whose kernels report what they refuse."""

    def __init__(self):
        super().__init__()
        self.status = self._t.zeros(1, dtype=self._t.int32, device=f"cuda:{self.dev}")
        self._memory.append(self.status)

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


class _CacheOp(_StatusOp):
    def __init__(self, cache, n_heads):
        super().__init__()
        if cache.pool.device.index != self.dev:
            raise ValueError(f"the cache is on {cache.pool.device}, the current device is cuda:{self.dev}")
        self.cache, self.n_heads = cache, int(n_heads)
        self.width = self.n_heads * cache.head_dim

    def _rows(self, rows, seq, pos, depth):
        for name, v, needed in (("seq", seq, True), ("pos", pos, True), ("depth", depth, False)):
            self._vec(name, v, self._t.int32, rows, needed)


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


class _PackedAttention(_CacheOp):
    """What prompts and drafts share (cdb_prompt_attention, cdb_draft_attention)."""

    def __init__(self, what, cache, n_heads, max_rows, max_requests, max_ctx, scale, mask_words):
        super().__init__(cache, n_heads)
        self.max_rows, self.max_requests = int(max_rows), int(max_requests)
        self.max_ctx = int(max_ctx or cache.max_ctx)
        hd = cache.head_dim
        n = self.L.cdb_prompt_attention_workspace(self.max_rows, self.max_requests, self.n_heads, cache.n_kv_heads, hd,
                                                  self.max_ctx)
        if n == 0:
            raise ValueError(f"n_heads {n_heads}, max_rows {max_rows}, max_requests {max_requests}, max_ctx {max_ctx}: not "
                             f"supported with {cache.n_kv_heads} KV heads of {hd}")
        t = self._t
        self.workspace = t.empty(n + 256, dtype=t.uint8, device=cache.pool.device)
        self._memory.append(self.workspace)
        base = (self.workspace.data_ptr() + 255) // 256 * 256
        self.args = PromptAttentionArgs(cache=cache.desc, n_heads=self.n_heads, scale=hd ** -0.5 if scale is None else scale,
                                        max_ctx=self.max_ctx, mask_words=mask_words, status=self.status.data_ptr(),
                                        workspace=base, workspace_bytes=n)
        self._bind(what, "prompt_attention")

    def _attend(self, q, row_start, lens, visible, seq, slot, out):
        if out is None:
            out = self._t.zeros(q.shape[0], self.width, dtype=self._t.bfloat16, device=q.device)
        rc = self._call(self._fn, self._ref, self._stream(), self.dev, self.max_rows, self.max_requests, q, row_start, lens,
                        visible, seq, slot, out)
        if rc != 0:
            if rc is None:
                self._explain(q, row_start, lens, visible, seq, out)
            self._fail(rc)
        return out

    def _explain(self, q, row_start, lens, visible, seq, out):
        t, rows, n = self._t, q.shape[0], lens.numel()
        if rows > self.max_rows or n > self.max_requests:
            raise ValueError(f"{rows} rows of {n} requests, the workspace holds {self.max_rows} of {self.max_requests}")
        if lens.dim() != 1:
            raise ValueError(f"lens: expected one length per request, got {tuple(lens.shape)}")
        self._mat("q", q, (t.bfloat16,), rows, self.width)
        self._vec("lens", lens, t.int32, n, True)
        self._vec("row_start", row_start, t.int32, n + 1, True)
        self._vec("seq", seq, t.int32, n)
        words = self.args.mask_words
        if words and (visible is None or visible.dtype != t.int64 or visible.dim() != 2 or visible.shape[0] < rows or
                      visible.shape[1] != words or not visible.is_contiguous() or visible.get_device() != self.dev):
            raise ValueError(f"visible: expected contiguous int64 [{rows}, {words}] on cuda:{self.dev}, got "
                             f"{None if visible is None else (tuple(visible.shape), visible.dtype, visible.device)}")
        self._mat("out", out, (t.bfloat16,), rows, self.width)


class PromptAttention(_PackedAttention):
    """Causal attention of packed prompts over the paged cache (cdb_prompt_attention).

    q bf16 [rows, n_heads head_dim], request i's tokens in rows row_start[i] .. row_start[i + 1] - 1
    (int32 [requests + 1]); lens int32 [requests] counts its cached tokens, these last ones among
    them, so a prompt may come in chunks or behind tokens cached before.  seq int32 [requests]:
    their sequences in the block table, by default 0, 1, ..  Rows behind the last request are left alone;
    a row at a negative position gives zeros.  Keys and values have to be in the cache before the call.
    """

    def __init__(self, cache, n_heads, max_rows, max_requests, max_ctx=None, scale=None):
        super().__init__("cdb_prompt_attention", cache, n_heads, max_rows, max_requests, max_ctx, scale, 0)

    def __call__(self, q, row_start, lens, seq=None, slot=0, out=None):
        return self._attend(q, row_start, lens, None, seq, slot, out)


class DraftAttention(_PackedAttention):
    """Attention of drafted tokens over the paged cache (cdb_draft_attention).

    As PromptAttention, for requests of at most max_draft rows, with a mask among each request's own
    rows: bit u of visible[row] (int64 [rows, ceil(max_draft / 64)]) says that the row sees the request's
    row u, see draft_mask.  Every row sees all tokens before the request's rows.
    """

    def __init__(self, cache, n_heads, max_rows, max_requests, max_draft, max_ctx=None, scale=None):
        if not 1 <= max_draft <= 256:
            raise ValueError(f"max_draft must be in 1..256, got {max_draft}")
        self.max_draft = int(max_draft)
        super().__init__("cdb_draft_attention", cache, n_heads, max_rows, max_requests, max_ctx, scale,
                         (self.max_draft + 63) // 64)

    def __call__(self, q, row_start, lens, visible, seq=None, slot=0, out=None):
        return self._attend(q, row_start, lens, visible, seq, slot, out)


class Rotary(_Op):
    """Query / key norm and rotary positions (cdb_rotate), for rows that CacheWriter's table does not serve.

    steps, factor: of rope_steps.  x [rows, (n_heads + n_kv_heads) head_dim and more] fp32 or bf16, query
    heads, then key heads; pos int32 [rows], < 0 padding.  In place unless `out` is given.  interleaved:
    a pair is two neighbours, not an element of each half.
    """

    def __init__(self, n_heads, n_kv_heads, head_dim, steps, interleaved=False, factor=1.0, q_gain=None, k_gain=None, eps=1e-6):
        super().__init__()
        t = self._t
        if steps.dtype != t.int64 or steps.dim() != 1 or not steps.is_contiguous() or steps.get_device() != self.dev:
            raise ValueError(f"steps: expected a contiguous int64 vector on cuda:{self.dev}, got {tuple(steps.shape)} {steps.dtype} "
                             f"on {steps.device}")
        if (q_gain is None) != (k_gain is None):
            raise ValueError("q_gain and k_gain come together")
        a = self.args = RotateArgs(n_heads=n_heads, n_kv_heads=n_kv_heads, head_dim=head_dim, steps=steps.data_ptr(),
                                   rot_dim=2 * steps.numel(), interleaved=bool(interleaved), factor=factor, eps=eps)
        a.q_gain = self._vec("q_gain", q_gain, t.float32, head_dim)
        a.k_gain = self._vec("k_gain", k_gain, t.float32, head_dim)
        self._keep = (steps, q_gain, k_gain)
        self.width = (n_heads + n_kv_heads) * head_dim
        self._bind("cdb_rotate", "rotate")

    def __call__(self, x, pos, out=None):
        if out is None:
            out = x
        rc = self._call(self._fn, self._ref, self._stream(), self.dev, x, pos, out)
        if rc != 0:
            if rc is None:
                t, rows = self._t, x.shape[0]
                self._mat("x", x, (t.float32, t.bfloat16), rows, self.width)
                self._vec("pos", pos, t.int32, rows, True)
                self._mat("out", out, (x.dtype,), rows, self.width)
            self._fail(rc)
        return out


Rows = namedtuple("Rows", "row_start seq pos slot")


class PagePlanner(_StatusOp):
    """Block tables and packed rows from the lengths of a step's requests (cdb_plan_pages).

    block_table int32 [n_seqs, max_blocks] and free_blocks int32 [free_slots], a ring of free blocks, are
    updated in place; state int64 [2] counts the blocks taken and given so far: a new pool of n blocks has
    free_blocks = 0 .. n - 1 and state (0, n).  lens int32 [requests] are the cached tokens, new_tokens int32
    [requests] those to add, or, negative, to drop.  state and lens are updated in place unless state_out
    and lens_out are given.  Returns Rows(row_start, seq, pos, slot): int32 [requests + 1], int32 and int32
    [max_rows], int64 [max_rows]; rows without a token are -1.  check() raises if a call could not be
    served; such a call changed nothing.
    """

    def __init__(self, block_table, free_blocks, max_requests, max_rows):
        super().__init__()
        t, dev = self._t, f"cuda:{self.dev}"
        if max_requests < 1 or max_rows < 0:
            raise ValueError("max_requests must be >= 1, max_rows >= 0")
        if block_table.dtype != t.int32 or block_table.dim() != 2 or not block_table.is_contiguous() or \
                block_table.get_device() != self.dev:
            raise ValueError(f"block_table: expected contiguous int32 [n_seqs, max_blocks] on {dev}, got "
                             f"{tuple(block_table.shape)} {block_table.dtype} on {block_table.device}")
        self._vec("free_blocks", free_blocks, t.int32, 1, True)
        self.max_requests, self.max_rows = int(max_requests), int(max_rows)
        self.row_start = t.empty(self.max_requests + 1, dtype=t.int32, device=dev)
        self.seq, self.pos = (t.empty(self.max_rows, dtype=t.int32, device=dev) for _ in range(2))
        self.slot = t.empty(self.max_rows, dtype=t.int64, device=dev)
        self._memory += [self.row_start, self.seq, self.pos, self.slot]
        self._out = Rows(self.row_start, self.seq, self.pos, self.slot)  # of the last number of requests
        self._keep = (block_table, free_blocks)
        self.args = PlanPagesArgs(block_table=block_table.data_ptr(), n_seqs=block_table.shape[0],
                                  max_blocks=block_table.shape[1], free_blocks=free_blocks.data_ptr(),
                                  free_slots=free_blocks.numel(), row_start=self.row_start.data_ptr(),
                                  row_seq=self.seq.data_ptr(), row_pos=self.pos.data_ptr(),
                                  row_slot=self.slot.data_ptr(), max_rows=self.max_rows, status=self.status.data_ptr())
        self._bind("cdb_plan_pages", "plan_pages")

    def __call__(self, state, lens, new_tokens, seq=None, state_out=None, lens_out=None):
        n = lens.numel()
        if n > self.max_requests:
            raise ValueError(f"{n} requests, at most {self.max_requests}")
        state_out = state if state_out is None else state_out
        lens_out = lens if lens_out is None else lens_out
        rc = self._call(self._fn, self._ref, self._stream(), self.dev, state, lens, new_tokens, seq, state_out, lens_out)
        if rc != 0:
            if rc is None:
                t = self._t
                if lens.dim() != 1:
                    raise ValueError(f"lens: expected one length per request, got {tuple(lens.shape)}")
                for name, v, needed in (("lens", lens, True), ("new_tokens", new_tokens, True), ("seq", seq, False),
                                        ("lens_out", lens_out, True)):
                    self._vec(name, v, t.int32, n, needed)
                self._vec("state", state, t.int64, 2, True)
                self._vec("state_out", state_out, t.int64, 2, True)
            self._fail(rc)
        out = self._out
        if out.row_start.shape[0] != n + 1:
            out = self._out = Rows(self.row_start[:n + 1], self.seq, self.pos, self.slot)
        return out


class PathKeeper(_CacheOp):
    """Moves a draft's accepted nodes to their places in the text (cdb_keep_path).

    In every slot of the cache, entry k < keep[i] of request i goes from position base[i] + path[i, k] to
    base[i] + k.  base, keep int32 [requests], path int32 [requests, max_path], ascending in a row; seq
    int32 [requests], by default 0, 1, ..
    """

    def __init__(self, cache):
        super().__init__(cache, 1)
        self.args = KeepPathArgs(cache=cache.desc, status=self.status.data_ptr())
        self._bind("cdb_keep_path", "keep_path")

    def __call__(self, base, path, keep, seq=None):
        rc = self._call(self._fn, self._ref, self._stream(), self.dev, base, path, keep, seq)
        if rc != 0:
            if rc is None:
                t, n = self._t, base.numel()
                if base.dim() != 1:
                    raise ValueError(f"base: expected one position per request, got {tuple(base.shape)}")
                self._vec("base", base, t.int32, n, True)
                self._mat("path", path, (t.int32,), n, 1)
                self._vec("keep", keep, t.int32, n, True)
                self._vec("seq", seq, t.int32, n)
            self._fail(rc)


def draft_mask(parent, words=None, device="cuda"):
    """DraftAttention's mask of one request's tree: parent[u] < u is the node that node u follows, -1 the text.

    int64 [len(parent), words]: node u's bits are u's, its parent's, and so on."""
    import torch
    n = len(parent)
    words = words or max(1, (n + 63) // 64)
    rows = []
    for u, p in enumerate(int(p) for p in parent):
        if not -1 <= p < u or u >= 64 * words:
            raise ValueError(f"node {u}: parent {p}, {words} words")
        rows.append((rows[p] if p >= 0 else 0) | 1 << u)
    bits = [[(r >> 64 * w & (1 << 64) - 1) - ((r >> 64 * w + 63 & 1) << 64) for w in range(words)] for r in rows]
    return torch.tensor(bits, dtype=torch.int64, device=device).reshape(n, words)


def rope_steps(rot_dim, theta=10000.0, scaling="none", factor=1.0, trained=None, low=1.0, high=32.0, device="cuda"):
    """(steps, factor) of Rotary: turns per position of each pair, times 2^64, as int64 [rot_dim / 2].

    The plain rotation turns pair j by theta^(-2j / rot_dim) per position.  scaling, to reach `factor` times
    further than a model was trained: "linear": positions divided by factor; "base": theta times
    factor^(rot_dim / (rot_dim - 2)), so that the slowest pair turns factor times slower; "parts": a pair that
    turns fewer than `low` times over `trained` positions turns factor times slower, one of more than `high` as before,
    a linear ramp between them in the number of turns (not in j, as some checkpoints have it), and cos and sin are
    multiplied by 0.1 ln(factor) + 1, the factor returned (else 1)."""
    import torch
    if rot_dim < 2 or rot_dim % 2 or theta <= 0 or factor < 1 or scaling not in ("none", "linear", "base", "parts"):
        raise ValueError(f"rot_dim {rot_dim}, theta {theta}, scaling {scaling!r}, factor {factor}")
    if scaling == "parts" and (not trained or not 0 <= low < high):
        raise ValueError('"parts" needs trained, and low < high')
    if scaling == "base":
        theta *= factor ** (rot_dim / max(rot_dim - 2, 1))
    steps = []
    for j in range(rot_dim // 2):
        inv = theta ** (-2.0 * j / rot_dim)
        if scaling == "linear":
            inv /= factor
        elif scaling == "parts":
            keep = min(1.0, max(0.0, (trained * inv / (2 * math.pi) - low) / (high - low)))
            inv *= keep + (1 - keep) / factor
        n = round(inv / (2 * math.pi) * 2.0 ** 64) & (1 << 64) - 1
        steps.append(n - (1 << 64) if n >> 63 else n)
    gain = 0.1 * math.log(factor) + 1 if scaling == "parts" else 1.0
    return torch.tensor(steps, dtype=torch.int64, device=device), gain


def rope_table(positions, rot_dim, theta=10000.0, device="cuda"):
    """(cos, sin) of pos * theta^(-2j / rot_dim), float32 [positions, rot_dim / 2, 2], angles in float64."""
    import torch
    inv = theta ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()
