"""Refusals of the operators for pages, rotation, prompts, drafts and accepted paths: C entry points, before any CUDA
call; and the helpers that need no GPU."""

import ctypes as C
import math

import numpy as np
import pytest
import torch

from continuous_depth_batching_gb300 import ops

ARG = -1
P = 0x1000  # never dereferenced: the call is refused


@pytest.fixture(scope="module")
def L():
    return ops._lib()


def filled(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def cache_desc(**kw):
    return filled(ops.Cache(pool=P, scales=P, block_table=P, dtype=2, kv_blocks=8, n_kv_slots=2, n_kv_heads=4, head_dim=64,
                            n_seqs=2, max_blocks=4), kw)


CACHE_BAD = [dict(dtype=0), dict(head_dim=48), dict(kv_blocks=0), dict(n_kv_slots=0), dict(n_seqs=0), dict(max_blocks=0),
             dict(pool=None), dict(pool=P + 8), dict(block_table=None), dict(scales=None), dict(scales=P + 4)]


def refused(call, a):
    assert call(C.byref(a), None) == ARG
    assert ops._lib().cdb_ops_last_error()


def pages_args(**kw):
    return filled(ops.PlanPagesArgs(requests=3, lens=P, new_tokens=P, seq=P, block_table=P, n_seqs=4, max_blocks=8,
                                    free_blocks=P, free_slots=32, state=P, state_out=P, lens_out=P, row_start=P, row_seq=P,
                                    row_pos=P, row_slot=P, max_rows=16), kw)


@pytest.mark.parametrize("bad", [dict(requests=-1), dict(requests=8193), dict(max_rows=-1), dict(n_seqs=0), dict(max_blocks=0),
                                 dict(max_blocks=1 << 28), dict(free_slots=0), dict(block_table=None), dict(free_blocks=None),
                                 dict(state=None), dict(state=P + 4), dict(state_out=None), dict(state_out=P + 4),
                                 dict(row_start=None), dict(lens=None), dict(new_tokens=None), dict(lens_out=None),
                                 dict(row_seq=None), dict(row_pos=None), dict(row_slot=P + 4)])
def test_plan_pages_refuses(L, bad):
    refused(L.cdb_plan_pages, pages_args(**bad))


@pytest.mark.parametrize("bad", [dict(max_rows=2**30 + 1), dict(max_rows=2**31 - 1), dict(free_slots=2**28 + 1),
                                 dict(free_slots=2**31 - 1)])
def test_plan_pages_refuses_what_32_bit_indices_do_not_hold(L, bad):
    refused(L.cdb_plan_pages, pages_args(**bad))


def rotate_args(**kw):
    return filled(ops.RotateArgs(rows=3, n_heads=8, n_kv_heads=4, head_dim=64, x=P, dtype=0, ldx=768, pos=P, steps=P, rot_dim=64,
                                 factor=1.0, q_gain=P, k_gain=P, eps=1e-6, out=P, ldo=768), kw)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(head_dim=48), dict(n_heads=-1), dict(n_heads=0, n_kv_heads=0), dict(dtype=2),
                                 dict(rot_dim=8), dict(rot_dim=24), dict(rot_dim=80), dict(rot_dim=0), dict(factor=math.inf),
                                 dict(factor=math.nan), dict(q_gain=None), dict(k_gain=None), dict(q_gain=P + 4), dict(eps=-1.0),
                                 dict(eps=math.nan), dict(x=None), dict(x=P + 8), dict(ldx=767), dict(ldx=770), dict(out=None),
                                 dict(out=P + 4), dict(ldo=760), dict(ldo=1024), dict(pos=None), dict(steps=None),
                                 dict(steps=P + 4), dict(rows=(1 << 31) - 1)])
def test_rotate_refuses(L, bad):
    refused(L.cdb_rotate, rotate_args(**bad))


def prompt_args(draft, **kw):
    a = ops.PromptAttentionArgs(cache=cache_desc(), rows=3, n_heads=8, q=P, ldq=512, requests=2, row_start=P, lens=P, scale=0.125,
                                max_ctx=64, out=P, ldo=512, workspace=P, workspace_bytes=1 << 40)
    if draft:
        a.visible, a.mask_words = P, 1
    return filled(a, kw)


PROMPT_BAD = [dict(cache=cache_desc(**b)) for b in CACHE_BAD] + [
    dict(rows=-1), dict(requests=-1), dict(n_heads=0), dict(n_heads=6), dict(n_heads=4 * 129, ldq=1 << 16, ldo=1 << 16), dict(q=None),
    dict(q=P + 8), dict(ldq=504), dict(ldq=516), dict(out=None), dict(out=P + 2), dict(ldo=504), dict(ldo=518), dict(row_start=None),
    dict(lens=None), dict(slot=-1), dict(slot=2), dict(max_ctx=0), dict(max_ctx=65), dict(scale=math.nan), dict(scale=math.inf),
    dict(workspace=None), dict(workspace=P + 16), dict(workspace_bytes=0), dict(cache=cache_desc(kv_blocks=1 << 24)),
    dict(rows=(1 << 31) - 1, requests=1 << 20)]


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("bad", PROMPT_BAD)
def test_prompt_and_draft_attention_refuse(L, bad, draft):
    refused(L.cdb_draft_attention if draft else L.cdb_prompt_attention, prompt_args(draft, **bad))


@pytest.mark.parametrize("bad", [dict(visible=None), dict(visible=P + 4), dict(mask_words=0), dict(mask_words=5)])
def test_draft_attention_refuses_masks(L, bad):
    refused(L.cdb_draft_attention, prompt_args(True, **bad))


def test_a_prompt_has_no_mask(L):
    refused(L.cdb_prompt_attention, prompt_args(False, visible=P))


def keep_args(**kw):
    return filled(ops.KeepPathArgs(cache=cache_desc(), requests=2, base=P, path=P, ld_path=8, max_path=8, keep=P, seq=P), kw)


@pytest.mark.parametrize("bad", [dict(cache=cache_desc(**b)) for b in CACHE_BAD] +
                         [dict(requests=-1), dict(requests=65536), dict(max_path=0), dict(max_path=257, ld_path=257), dict(ld_path=7),
                          dict(base=None), dict(path=None), dict(keep=None)])
def test_keep_path_refuses(L, bad):
    refused(L.cdb_keep_path, keep_args(**bad))


def test_no_arguments_and_empty_calls(L):
    for f in (L.cdb_plan_pages, L.cdb_rotate, L.cdb_prompt_attention, L.cdb_draft_attention, L.cdb_keep_path):
        assert f(None, None) == ARG
    assert L.cdb_rotate(C.byref(rotate_args(rows=0, x=None, out=None)), None) == 0
    for draft, f in ((False, L.cdb_prompt_attention), (True, L.cdb_draft_attention)):
        assert f(C.byref(prompt_args(draft, rows=0, q=None)), None) == 0
        assert f(C.byref(prompt_args(draft, requests=0, workspace=None)), None) == 0
    assert L.cdb_keep_path(C.byref(keep_args(requests=0, base=None)), None) == 0


def test_workspace_holds_every_smaller_call(L):
    w = L.cdb_prompt_attention_workspace
    assert w(10, 2, 6, 4, 64, 100) == 0 and w(10, 2, 8, 4, 48, 100) == 0 and w(-1, 2, 8, 4, 64, 100) == 0
    for heads, kv, hd in ((16, 16, 128), (32, 8, 128), (7, 7, 32)):
        for rows in (1, 40, 1000, 8192):
            for requests in (1, 7, 64):
                most = w(rows, requests, heads, kv, hd, 8192)
                for r in sorted({1, rows // 3 + 1, rows - 1, rows} - {0}):
                    for n in sorted({1, requests // 2 + 1, requests}):
                        assert w(r, n, heads, kv, hd, 8192) <= most, (heads, rows, requests, r, n)


def test_draft_masks():
    m = ops.draft_mask([-1, 0, 0, 1, -1, 4], device="cpu")
    assert m[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10000, 0b110000]
    chain = ops.draft_mask(range(-1, 129), words=3, device="cpu").numpy().view(np.uint64)
    assert chain.shape == (130, 3)
    for u in (0, 63, 64, 127, 128, 129):
        bits = sum(int(chain[u, w]) << (64 * w) for w in range(3))
        assert bits == (1 << (u + 1)) - 1
    for wrong in ([0], [-1, 1], [-2], [-1] * 65):
        with pytest.raises(ValueError):
            ops.draft_mask(wrong, words=1, device="cpu")
    assert ops.draft_mask([], words=2, device="cpu").shape == (0, 2)


def test_rope_steps():
    steps, f = ops.rope_steps(64, theta=10000.0, device="cpu")
    assert f == 1.0 and steps.dtype == torch.int64
    turns = steps.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    want = 10000.0 ** (-np.arange(0, 64, 2) / 64) / (2 * math.pi)
    assert np.max(np.abs(turns / want - 1)) < 1e-15
    linear = ops.rope_steps(64, scaling="linear", factor=4.0, device="cpu")[0]
    # both are rounded to whole numbers of at least 5e14 (1e-15 each), from a handful of float64 roundings (2^-53 each)
    assert np.max(np.abs(linear.numpy() / (steps.numpy() / 4) - 1)) < 4e-15
    base = ops.rope_steps(64, scaling="base", factor=4.0, device="cpu")[0]
    assert base[0] == steps[0] and abs(float(steps[-1]) / float(base[-1]) - 4) < 1e-9
    parts, f = ops.rope_steps(64, scaling="parts", factor=4.0, trained=4096, device="cpu")
    assert abs(f - (0.1 * math.log(4) + 1)) < 1e-12
    assert parts[0] == steps[0] and abs(float(steps[-1]) / float(parts[-1]) - 4) < 1e-9
    ratio = steps.numpy() / parts.numpy()
    assert np.all(np.diff(ratio) >= -1e-12) and np.any((ratio > 1.01) & (ratio < 3.99))
    for wrong in (dict(rot_dim=7), dict(rot_dim=64, scaling="other"), dict(rot_dim=64, scaling="parts"),
                  dict(rot_dim=64, factor=0.5), dict(rot_dim=64, scaling="parts", trained=4096, low=3.0, high=2.0)):
        with pytest.raises(ValueError):
            ops.rope_steps(device="cpu", **wrong)
