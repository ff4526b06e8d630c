"""Cases for the operators of the decode step: the cache write, attention over the paged
cache, the same attention with a shared prefix, and sampling.

Where `own` is false, `run` computes each operator from elementary torch operations; where it
is true, it makes the calls a program makes of the package's operators.

Every cache is a pool [blocks, slots, 2, kv_heads, 16, head_dim]: 16-token pages, one slot per
loop step of a looped model, K then V, each head's 16 positions contiguous; `block_table` row s
names the blocks of sequence s.  An e4m3 pool holds codes and, per (position, head), a float32
scale.  A row with a negative sequence number is padding: nothing of it is read or written.
"""

import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
PAGE = 16
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One token of one sequence: the latency of a step's first kernel.
        dict(name="write one token", op="write", rows=1, heads=16, kv_heads=16, head_dim=128, src="fp32",
             norm=True, cache="e4m3", slots=4, pad=0),
        # A decode batch whose rows sit at different loop steps, grouped heads, padded to its bucket.
        dict(name="write a decode batch", op="write", rows=128, heads=32, kv_heads=8, head_dim=128, src="bf16",
             norm=True, cache="e4m3", slots=4, pad=9),
        # A full prefill chunk of 8192 prompt tokens.
        dict(name="write a prefill chunk", op="write", rows=8192, heads=16, kv_heads=16, head_dim=128, src="fp32",
             norm=True, cache="e4m3", slots=1, pad=0),
        # One sequence decoding alone.
        dict(name="attend one row", op="attend", rows=1, heads=16, kv_heads=16, head_dim=128, cache="e4m3",
             slots=4, ctx_lo=1000, ctx_hi=1001, pad=0),
        # The 64-slot decode batch of the default workload, rows at mixed loop steps.
        dict(name="attend a decode batch", op="attend", rows=64, heads=16, kv_heads=16, head_dim=128, cache="e4m3",
             slots=4, ctx_lo=128, ctx_hi=1280, pad=0),
        # Grouped heads over long, ragged contexts.
        dict(name="attend long contexts", op="attend", rows=128, heads=32, kv_heads=8, head_dim=128, cache="bf16",
             slots=1, ctx_lo=17, ctx_hi=8192, pad=3),
        # A few requests behind one system prompt.
        dict(name="shared short prompt", op="shared", rows=8, heads=16, kv_heads=16, head_dim=128, cache="bf16",
             slots=1, prefix=512, ctx_lo=1, ctx_hi=64, pad=0),
        # A decode batch behind one long document.
        dict(name="shared long document", op="shared", rows=64, heads=16, kv_heads=16, head_dim=128, cache="bf16",
             slots=1, prefix=8192, ctx_lo=1, ctx_hi=512, pad=0),
        # Many samples of one prompt, grouped heads, quantised cache.
        dict(name="shared many samples", op="shared", rows=256, heads=32, kv_heads=8, head_dim=128, cache="e4m3",
             slots=1, prefix=4096, ctx_lo=1, ctx_hi=256, pad=5),
        # One row of logits: the tail of a single-sequence step.
        dict(name="sample one row", op="sample", rows=1, vocab=49152, kind="fp32", flat=2.5, mix=True),
        # The decode batch, each request with its own settings.
        dict(name="sample a decode batch", op="sample", rows=64, vocab=49152, kind="fp32", flat=2.5, mix=True),
        # A wide batch over the larger vocabulary, bf16 logits (many equal values).
        dict(name="sample a wide batch", op="sample", rows=512, vocab=65536, kind="bf16", flat=1.5, mix=True),
    ]


HEADS = [(16, 16, 128), (32, 8, 128), (55, 55, 96), (14, 2, 64), (20, 4, 96), (16, 2, 128), (7, 7, 32), (24, 3, 64),
         (8, 1, 128), (40, 8, 128)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "attend", "shared", "sample"])
    h, hk, hd = rng.choice(HEADS)
    if op == "write":
        rows = _log(rng, 1, min(8192, 8192 * 6144 // ((h + 2 * hk) * hd)))
        return dict(op=op, rows=rows, heads=h, kv_heads=hk, head_dim=hd, src=rng.choice(["fp32", "bf16"]),
                    norm=rng.random() < 0.7, cache=rng.choice(["e4m3", "bf16"]), slots=rng.choice([1, 2, 4]),
                    pad=rng.randrange(0, max(1, rows // 8)))
    if op == "attend":
        hi = _log(rng, 1, 16384)
        room = 128 * 8192 * 8 * 128 // (hi * hk * hd)  # the plain form's gathered keys
        rows = _log(rng, 1, max(1, min(512, room)))
        return dict(op=op, rows=rows, heads=h, kv_heads=hk, head_dim=hd, cache=rng.choice(["e4m3", "bf16"]),
                    slots=rng.choice([1, 2, 4]), ctx_lo=rng.randint(1, hi), ctx_hi=hi + 1,
                    pad=rng.randrange(0, max(1, rows // 8)))
    if op == "shared":
        hi = _log(rng, 1, 1024)
        rows = _log(rng, 2, max(2, min(512, 64 * 1024 * 2048 // (hi * hk * hd))))
        prefix = PAGE * _log(rng, 1, max(1, min(1024, 256 * 32 * 4096 // (rows * h * PAGE))))
        return dict(op=op, rows=rows, heads=h, kv_heads=hk, head_dim=hd, cache=rng.choice(["e4m3", "bf16"]),
                    slots=1, prefix=prefix, ctx_lo=rng.randint(1, hi), ctx_hi=hi + 1,
                    pad=rng.randrange(0, max(1, rows // 8)))
    vocab = _log(rng, 300, 200000)
    rows = _log(rng, 1, max(1, min(1024, 512 * 65536 // vocab)))
    return dict(op=op, rows=rows, vocab=vocab, kind=rng.choice(["fp32", "bf16"]), flat=round(rng.uniform(0.5, 6.0), 2),
                mix=rng.random() < 0.8)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed) & 0x7FFFFFFF)


def _lengths(case, seed):
    """Keys of each row's own part (host), from the seed."""
    r = np.random.RandomState((int(seed) * 7919 + 11) & 0x7FFFFFFF)
    return r.randint(case["ctx_lo"], max(case["ctx_hi"], case["ctx_lo"] + 1), size=case["rows"])


def _rope_table(positions, rot, theta=10000.0):
    inv = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEVICE) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=DEVICE)[:, None] * inv
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _cache(case, blocks, g, fill):
    """An empty (zero) or filled pool: keys with a few loud channels, as attention keys have."""
    shape = (blocks, case["slots"], 2, case["kv_heads"], PAGE, case["head_dim"])
    e4m3 = case["cache"] == "e4m3"
    if not fill:
        pool = torch.zeros(shape, device=DEVICE, dtype=torch.uint8).view(torch.float8_e4m3fn) if e4m3 else \
            torch.zeros(shape, device=DEVICE, dtype=torch.bfloat16)
        return pool, torch.zeros(shape[:-1], device=DEVICE) if e4m3 else None
    x = torch.empty(shape, device=DEVICE, dtype=torch.bfloat16).normal_(generator=g)
    loud = 1 + 3 * (torch.rand(case["kv_heads"], 1, case["head_dim"], generator=g, device=DEVICE) > 0.95)
    x *= loud.to(torch.bfloat16)
    if not e4m3:
        return x, None
    scales = torch.empty(shape[:-1], device=DEVICE)
    codes = torch.empty(shape, device=DEVICE, dtype=torch.uint8)
    step = max(1, (1 << 26) // max(1, x[0].numel()))
    for b in range(0, blocks, step):
        y = x[b:b + step].float()
        s = (y.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN)
        scales[b:b + step] = s
        codes[b:b + step] = (y / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(torch.float8_e4m3fn), scales


def prepare(case, seed):
    g = _gen(seed)
    op, rows = case["op"], case["rows"]
    if op == "sample":
        x = torch.randn(rows, case["vocab"], generator=g, device=DEVICE) * case["flat"]
        peaks = torch.randint(0, case["vocab"], (rows, 6), generator=g, device=DEVICE)
        x.scatter_add_(1, peaks, 4 + 6 * torch.rand(rows, 6, generator=g, device=DEVICE))
        if case["kind"] == "bf16":
            x = x.bfloat16()
        u = torch.rand(rows, generator=g, device=DEVICE)
        t = torch.full((rows,), 0.8, device=DEVICE)
        k = torch.full((rows,), 50, device=DEVICE, dtype=torch.int32)
        p = torch.full((rows,), 0.95, device=DEVICE)
        mp = torch.zeros(rows, device=DEVICE)
        if case["mix"]:  # requests with settings of their own: greedy, plain, top-k, top-p, min-p, all of them
            pick = torch.randint(0, 8, (rows,), generator=g, device=DEVICE)
            t = torch.where(pick == 0, torch.zeros_like(t), 0.3 + 1.2 * torch.rand(rows, generator=g, device=DEVICE))
            k = torch.where((pick == 2) | (pick >= 6), torch.randint(1, 400, (rows,), generator=g, device=DEVICE), 0)
            k = k.to(torch.int32)
            p = torch.where((pick == 3) | (pick == 4) | (pick >= 6),
                            0.5 + 0.5 * torch.rand(rows, generator=g, device=DEVICE), torch.ones_like(p))
            mp = torch.where((pick == 5) | (pick == 7), 0.2 * torch.rand(rows, generator=g, device=DEVICE), mp)
        s = dict(case=case, logits=x, u=u, temperature=t, top_k=k, top_p=p, min_p=mp)
        if own:
            from continuous_depth_batching_gb300 import ops
            s["plan"] = ops.Sampler(rows, case["vocab"])
        return s

    h, hk, hd = case["heads"], case["kv_heads"], case["head_dim"]
    n = rows - case["pad"]
    seq = torch.full((rows,), -1, dtype=torch.int32, device=DEVICE)
    depth = torch.randint(0, case["slots"], (rows,), generator=g, device=DEVICE).to(torch.int32)
    if op == "write":
        # Rows of a decode batch: one row of each of n sequences; a long chunk: consecutive positions of a few.
        per = 1 if n <= 512 else 1024
        nseq = (n + per - 1) // per
        maxb = (4096 + per) // PAGE
        start = torch.randint(0, 4096, (nseq,), generator=g, device=DEVICE)
        i = torch.arange(n, device=DEVICE)
        pos = torch.zeros(rows, dtype=torch.int32, device=DEVICE)
        seq[:n] = (i // per).to(torch.int32)
        pos[:n] = (start[i // per] + i % per).to(torch.int32)
        # Only the pages that are written exist; every other block table entry is empty.
        most = (per + PAGE - 2) // PAGE + 1  # pages that `per` consecutive positions can touch
        blocks = nseq * most
        table = torch.full((nseq, maxb + 1), -1, dtype=torch.int32, device=DEVICE)
        perm = torch.randperm(blocks, generator=g, device=DEVICE).to(torch.int32).view(nseq, most)
        table.scatter_(1, start[:, None] // PAGE + torch.arange(most, device=DEVICE), perm)
        maxb += 1
        pool, scales = _cache(case, blocks, g, False)
        qkv = torch.randn(rows, (h + 2 * hk) * hd, generator=g, device=DEVICE)
        qkv *= 0.5 + 3 * torch.rand(rows, 1, generator=g, device=DEVICE)
        if case["src"] == "bf16":
            qkv = qkv.bfloat16()
        gain = [1 + 0.2 * torch.randn(hd, generator=g, device=DEVICE) for _ in range(2)] if case["norm"] else [None] * 2
        s = dict(case=case, qkv=qkv, seq=seq, pos=pos, depth=depth, table=table, pool=pool, scales=scales,
                 q_gain=gain[0], k_gain=gain[1], rope=_rope_table(maxb * PAGE, hd),
                 q=torch.zeros(rows, h * hd, dtype=torch.bfloat16, device=DEVICE))
        if own:
            from continuous_depth_batching_gb300 import ops
            s["plan"] = ops.CacheWriter(ops.PagedCache(pool, table, scales), h, s["rope"], q_gain=s["q_gain"],
                                        k_gain=s["k_gain"], eps=1e-6)
        return s

    lens = _lengths(case, seed)
    shared = case["prefix"] if op == "shared" else 0
    ppages = shared // PAGE
    need = (lens + PAGE - 1) // PAGE
    maxb = int(ppages + need.max())
    first = np.concatenate([[0], np.cumsum(need[:n])])
    blocks = int(ppages + first[n])
    perm = torch.randperm(blocks, generator=g, device=DEVICE).to(torch.int32)
    table = torch.full((n, maxb), -1, dtype=torch.int32, device=DEVICE)
    table[:, :ppages] = perm[:ppages]
    own_page = torch.arange(maxb - ppages, device=DEVICE)[None]
    fd = torch.from_numpy(first[:n].astype(np.int64)).to(DEVICE)[:, None]
    nd = torch.from_numpy(need[:n].astype(np.int64)).to(DEVICE)[:, None]
    idx = (ppages + fd + own_page).clamp(max=max(blocks - 1, 0))
    table[:, ppages:] = torch.where(own_page < nd, perm[idx], -1)
    seq[:n] = torch.randperm(n, generator=g, device=DEVICE).to(torch.int32)
    pos = torch.zeros(rows, dtype=torch.int32, device=DEVICE)
    own_len = torch.from_numpy(lens.astype(np.int32)).to(DEVICE)
    pos[:n] = shared + own_len[:n][seq[:n].long()] - 1
    pool, scales = _cache(case, blocks, g, True)
    q = (1.3 * torch.randn(rows, h * hd, generator=g, device=DEVICE)).bfloat16()
    s = dict(case=case, q=q, seq=seq, pos=pos, depth=depth, table=table, pool=pool, scales=scales, shared=shared,
             longest=shared + int(lens.max()), out=torch.zeros(rows, h * hd, dtype=torch.bfloat16, device=DEVICE))
    if own:
        from continuous_depth_batching_gb300 import ops
        s["plan"] = ops.DecodeAttention(ops.PagedCache(pool, table, scales), h, rows, s["longest"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        plan = state["plan"]
        if op == "sample":
            token, logprob = plan(state["logits"], state["u"], temperature=state["temperature"], top_k=state["top_k"],
                                  top_p=state["top_p"], min_p=state["min_p"])
            return {"token": token, "logprob": logprob}
        if op == "write":
            plan(state["qkv"], state["seq"], state["pos"], depth=state["depth"], q_out=state["q"])
            return _written(state)
        if op == "attend":
            return {"out": plan(state["q"], state["seq"], state["pos"], depth=state["depth"], out=state["out"])}
        return {"out": plan(state["q"], state["seq"], state["pos"], shared_len=state["shared"], out=state["out"])}
    if op == "sample":
        return _plain_sample(state)
    if op == "write":
        return _plain_write(state)
    return _plain_attend(state)


def _written(state):
    r = {"q": state["q"], "cache": state["pool"]}
    if state["scales"] is not None:
        r["scales"] = state["scales"]
    return r


def _plain_write(s):
    c = s["case"]
    h, hk, hd, n = c["heads"], c["kv_heads"], c["head_dim"], c["rows"] - c["pad"]
    x = s["qkv"][:n].float().view(n, h + 2 * hk, hd)
    q, k, v = x[:, :h], x[:, h:h + hk], x[:, h + hk:]
    if s["q_gain"] is not None:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6) * s["q_gain"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + 1e-6) * s["k_gain"]
    cs = s["rope"][s["pos"][:n].long()]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]

    def rotate(y):
        a, b = y[..., :hd // 2], y[..., hd // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    s["q"][:n] = rotate(q).reshape(n, h * hd).to(torch.bfloat16)
    kv = torch.stack([rotate(k), v], 1)  # [n, 2, kv_heads, head_dim]
    pos = s["pos"][:n].long()
    block = s["table"][s["seq"][:n].long(), pos // PAGE].long()
    slot, off = s["depth"][:n].long(), pos % PAGE
    if s["scales"] is None:
        s["pool"][block, slot, :, :, off] = kv.to(torch.bfloat16)
    else:
        scale = (kv.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN)
        code = (kv / scale[..., None]).to(torch.float8_e4m3fn)
        s["pool"].view(torch.uint8)[block, slot, :, :, off] = code.view(torch.uint8)
        s["scales"][block, slot, :, :, off] = scale
    return _written(s)


def _keys(s, block, slot, off):
    """K and V [..., kv_heads, head_dim] in 32 bits at (block, slot, off)."""
    if s["scales"] is None:
        x = s["pool"][block, slot, :, :, off].float()
    else:
        x = s["pool"].view(torch.uint8)[block, slot, :, :, off].view(torch.float8_e4m3fn).float()
        x = x * s["scales"][block, slot, :, :, off][..., None]
    return x.unbind(-3)


def _plain_attend(s):
    c = s["case"]
    h, hk, hd, n, p = c["heads"], c["kv_heads"], c["head_dim"], c["rows"] - c["pad"], s["shared"]
    q = s["q"][:n].float().view(n, hk, h // hk, hd)
    seq, pos = s["seq"][:n].long(), s["pos"][:n].long()
    slot = s["depth"][:n].long() if c["op"] == "attend" else torch.zeros_like(seq)
    j = torch.arange(p, s["longest"], device=q.device)
    block = s["table"][seq][:, j // PAGE].long().clamp_min(0)
    k, v = _keys(s, block, slot[:, None], (j % PAGE)[None])
    x = torch.einsum("rkgd,rlkd->rkgl", q, k) / math.sqrt(hd)
    x = x.masked_fill(j[None, None, None, :] > pos[:, None, None, None], -math.inf)
    if p:
        i = torch.arange(p, device=q.device)
        ks, vs = _keys(s, s["table"][0][i // PAGE].long(), torch.zeros_like(i), i % PAGE)
        x = torch.cat([torch.einsum("rkgd,lkd->rkgl", q, ks) / math.sqrt(hd), x], -1)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.einsum("rkgl,rlkd->rkgd", e[..., p:], v)
    if p:
        o = o + torch.einsum("rkgl,lkd->rkgd", e[..., :p], vs)
    s["out"][:n] = (o / e.sum(-1, keepdim=True)).reshape(n, h * hd).to(torch.bfloat16)
    return {"out": s["out"]}


def _plain_sample(s):
    # 64 bits: a token is chosen where a running sum crosses a border.
    x = s["logits"].double()
    vocab = x.shape[1]
    t = s["temperature"].double()[:, None]
    greedy = ~(t > 0)
    top = x.amax(1, keepdim=True)
    y, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((y - top) / torch.where(greedy, torch.ones_like(t), t))
    rank = torch.arange(vocab, device=x.device)[None]
    k = s["top_k"].long()[:, None]
    k = torch.where((k <= 0) | (k > vocab), vocab, k)
    k = torch.where(greedy, 1, k)
    w = w * (rank < k)
    run_sum = torch.cumsum(w, 1)
    p = s["top_p"].double()[:, None]
    keep = ((run_sum - w < p * run_sum[:, -1:]) | (p >= 1) | (rank == 0)) & (rank < k)
    keep &= w >= s["min_p"].double()[:, None].clamp(max=1)
    w = torch.zeros_like(w).scatter(1, order, w * keep)
    run_sum = torch.cumsum(w, 1)
    total = run_sum[:, -1:]
    token = (run_sum <= s["u"].double()[:, None] * total).sum(1).clamp(max=vocab - 1)
    logprob = torch.log(w.gather(1, token[:, None]) / total)[:, 0]
    return {"token": token.to(torch.int32), "logprob": logprob.float()}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _cell(case):
    return case["head_dim"] * 2 if case["cache"] == "bf16" else case["head_dim"] + 4


def work(case):
    rows = case["rows"]
    if case["op"] == "sample":
        es = 4 if case["kind"] == "fp32" else 2
        return {"bytes": rows * (case["vocab"] * es + 28), "flops": 4 * rows * case["vocab"]}
    h, hk, hd, n = case["heads"], case["kv_heads"], case["head_dim"], case["rows"] - case["pad"]
    if case["op"] == "write":
        es = 4 if case["src"] == "fp32" else 2
        moved = n * ((h + 2 * hk) * hd * es + h * hd * 2 + 2 * hk * _cell(case) + hd * 4 + 16)
        return {"bytes": moved, "flops": n * (h + 2 * hk) * hd * 8}
    mean = (case["ctx_lo"] + max(case["ctx_hi"], case["ctx_lo"] + 1) - 1) / 2
    shared = case.get("prefix", 0)
    keys = shared + n * mean
    return {"bytes": keys * 2 * hk * _cell(case) + n * (2 * h * hd * 2 + 12) + keys / PAGE * 4,
            "flops": 4 * n * (mean + shared) * h * hd}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    if case["op"] == "write":
        return _exact_write(s)
    return _exact_attend(s)


def _exact_sample(s):
    x = s["logits"].double().cpu().numpy()
    u, t, k, p, mp = (s[n].double().cpu().numpy() for n in ("u", "temperature", "top_k", "top_p", "min_p"))
    rows, vocab = x.shape
    if rows * vocab > 1 << 26:
        return None
    out = np.zeros(rows)
    for r in range(rows):
        if not t[r] > 0:
            continue  # the whole mass is on the argmax
        z = (x[r] - x[r].max()) / t[r]
        by = np.lexsort((np.arange(vocab), -x[r]))
        kept = by[:int(k[r])] if 0 < k[r] < vocab else by
        mass = np.exp(z[kept])
        if p[r] < 1:
            upto = np.searchsorted(np.cumsum(mass), p[r] * mass.sum(), side="left") + 1
            kept = kept[:upto]
        kept = np.sort(kept[z[kept] >= (math.log(min(mp[r], 1.0)) if mp[r] > 0 else -math.inf)])
        mass = np.exp(z[kept])
        at = min(np.searchsorted(np.cumsum(mass), u[r] * mass.sum(), side="right"), len(kept) - 1)
        out[r] = z[kept[at]] - math.log(mass.sum())
    return {"token": None, "logprob": out}


def _exact_write(s):
    c = s["case"]
    h, hk, hd, n = c["heads"], c["kv_heads"], c["head_dim"], c["rows"] - c["pad"]
    heads = list(s["qkv"][:n].double().view(n, h + 2 * hk, hd).unbind(1))
    at = s["pos"][:n].long()
    turn = torch.view_as_complex(s["rope"].double().contiguous())[at]
    q = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    pool = torch.zeros(s["pool"].shape, dtype=torch.float64, device=q.device)
    scales = None if s["scales"] is None else torch.zeros(s["scales"].shape, dtype=torch.float64, device=q.device)
    block = s["table"][s["seq"][:n].long(), torch.div(at, PAGE, rounding_mode="floor")].long()
    slot, off = s["depth"][:n].long(), at % PAGE
    for i, y in enumerate(heads):
        if i < h + hk:
            gain = s["q_gain"] if i < h else s["k_gain"]
            if gain is not None:
                y = y / torch.sqrt((y * y).sum(1, keepdim=True) / hd + 1e-6) * gain.double()
            z = torch.complex(y[:, :hd // 2].contiguous(), y[:, hd // 2:].contiguous()) * turn
            y = torch.cat([z.real, z.imag], 1)
        if i < h:
            q[:n, i * hd:(i + 1) * hd] = y
            continue
        kv, j = divmod(i - h, hk)
        if scales is None:
            pool[block, slot, kv, j, off] = y
            continue
        sc = torch.clamp(y.abs().max(1).values / E4M3_MAX, min=SCALE_MIN)
        z = y / sc[:, None]
        # e4m3: three bits behind the leading one, steps of 2^-9 below 2^-6
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(z.abs().clamp_min(1e-30))), min=-6) - 3)
        pool[block, slot, kv, j, off] = torch.round(z / step) * step
        scales[block, slot, kv, j, off] = sc
    r = {"q": q, "cache": pool}
    if scales is not None:
        r["scales"] = scales
    return r


def _exact_attend(s):
    c = s["case"]
    h, hk, hd, n = c["heads"], c["kv_heads"], c["head_dim"], c["rows"] - c["pad"]
    if n * s["longest"] * h * hd > 1 << 33:
        return None
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    seq, pos, depth = s["seq"].tolist(), s["pos"].tolist(), s["depth"].tolist()
    for r in range(n):
        length, slot = pos[r] + 1, depth[r] if c["op"] == "attend" else 0
        b = s["table"][seq[r], :(length + PAGE - 1) // PAGE].long()
        kv = s["pool"][b, slot].to(torch.float64)  # [pages, 2, kv_heads, 16, head_dim]
        if s["scales"] is not None:
            kv = kv * s["scales"][b, slot].double()[..., None]
        kv = kv.permute(1, 2, 0, 3, 4).reshape(2, hk, -1, hd)[:, :, :length]
        x = s["q"][r].double().view(hk, h // hk, hd) @ kv[0].transpose(1, 2) * hd ** -0.5
        out[r] = (torch.softmax(x, -1) @ kv[1]).reshape(-1)
    return {"out": out}
