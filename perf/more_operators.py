"""Cases for the operators that take prompts and drafts to the paged cache: pages and rows from request
lengths, rotary positions, attention of packed prompts, attention of drafted tokens, and keeping the
accepted ones.

Where `own` is false, `run` computes each operator from elementary torch operations; where it is true, it
makes the calls a program makes of the package's operators.

Every cache is a pool [blocks, slots, 2, kv_heads, 16, head_dim]: 16-token pages, one slot per loop step and
layer, K then V, each head's 16 positions contiguous; `table` row s names the blocks of sequence s.  An e4m3
pool holds codes and, per (position, head), a float32 scale.  Rows of a call are packed: request i has rows
row_start[i] .. row_start[i + 1] - 1; rows behind the last request are padding and left as they were.
"""

import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
PAGE = 16
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # A decode step's pages: every request grows by one token.
        dict(name="pages of a decode step", op="pages", requests=64, lo=1, hi=2, drop=0.0, ctx=2048),
        # A busy step: prompt chunks and drafts of many requests, rejected drafts given back.
        dict(name="pages of a mixed step", op="pages", requests=1000, lo=0, hi=64, drop=0.3, ctx=4096),
        # One token of one sequence: latency alone.
        dict(name="rotate one token", op="rotate", rows=1, heads=16, kv_heads=16, head_dim=128, rot=128,
             interleaved=False, src="fp32", norm=True, scaling="none", far=4096),
        # The rows of a batch of drafts, half of each head rotated, neighbours paired.
        dict(name="rotate a batch of drafts", op="rotate", rows=500, heads=32, kv_heads=8, head_dim=128, rot=64,
             interleaved=True, src="bf16", norm=False, scaling="linear", far=32768),
        # A full prefill chunk far inside a long context.
        dict(name="rotate a prompt chunk", op="rotate", rows=8192, heads=32, kv_heads=8, head_dim=128, rot=128,
             interleaved=False, src="bf16", norm=True, scaling="parts", far=1000000),
        # A short question.
        dict(name="one short prompt", op="prompt", requests=1, lo=37, hi=38, ctx_lo=0, ctx_hi=1, heads=16, kv_heads=16,
             head_dim=128, cache="bf16", slots=4, pad=0),
        # Chunks of prompts of which a part is cached already, grouped heads, quantised cache.
        dict(name="chunks behind cached tokens", op="prompt", requests=5, lo=100, hi=1100, ctx_lo=0, ctx_hi=3000, heads=32,
             kv_heads=8, head_dim=128, cache="e4m3", slots=1, pad=19),
        # A prompt that fills a whole prefill chunk.
        dict(name="one long prompt", op="prompt", requests=1, lo=8192, hi=8193, ctx_lo=0, ctx_hi=1, heads=32, kv_heads=8,
             head_dim=128, cache="bf16", slots=1, pad=0),
        # One request's draft, alone on the machine.
        dict(name="one draft", op="tree", requests=1, lo=8, hi=9, ctx_lo=1000, ctx_hi=1001, heads=16, kv_heads=16,
             head_dim=128, cache="bf16", slots=4, pad=0),
        # A decode batch with a draft of its own size for each request.
        dict(name="drafts of a batch", op="tree", requests=32, lo=1, hi=33, ctx_lo=500, ctx_hi=8000, heads=32, kv_heads=8,
             head_dim=128, cache="e4m3", slots=1, pad=7),
        # The accepted path of one draft in one layer's slots.
        dict(name="keep one path", op="keep", requests=1, nodes=8, keep=4, kv_heads=16, head_dim=128, cache="bf16",
             slots=4, ctx=500),
        # The accepted paths of a batch in all layers and loop steps of a model.
        dict(name="keep paths of a batch", op="keep", requests=16, nodes=32, keep=8, kv_heads=16, head_dim=128,
             cache="bf16", slots=96, ctx=600),
    ]


HEADS = [(16, 16, 128), (32, 8, 128), (55, 55, 96), (14, 2, 64), (20, 4, 96), (16, 2, 128), (7, 7, 32), (24, 3, 64),
         (8, 1, 128), (40, 8, 128)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "rotate", "prompt", "prompt", "tree", "tree", "keep"])
    h, hk, hd = rng.choice(HEADS)
    cache = rng.choice(["e4m3", "bf16"])
    if op == "pages":
        n = _log(rng, 1, 1000)
        lo = rng.randint(0, 8)
        return dict(op=op, requests=n, lo=lo, hi=lo + _log(rng, 1, max(1, min(2000, 56000 // n))),
                    drop=rng.choice([0.0, 0.1, 0.3, 0.6]), ctx=_log(rng, 1, 4096))
    if op == "rotate":
        return dict(op=op, rows=_log(rng, 1, min(8192, 8192 * 5120 // ((h + hk) * hd) // 2)), heads=h, kv_heads=hk,
                    head_dim=hd, rot=16 * rng.randint(1, hd // 16), interleaved=rng.random() < 0.5,
                    src=rng.choice(["fp32", "bf16"]), norm=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "base", "parts"]), far=_log(rng, 100, 1000000))
    if op == "keep":
        t = rng.randint(2, 64)
        k = rng.randint(1, min(t, 12))
        slots = rng.choice([1, 4, 24, 96])
        room = 16 * 3 * 96 * 16 * 128 // ((t // PAGE + 2) * slots * hk * hd)
        return dict(op=op, requests=_log(rng, 1, max(1, min(64, room))), nodes=t, keep=k, kv_heads=hk, head_dim=hd,
                    cache=cache, slots=slots, ctx=_log(rng, 1, 4096))
    if op == "tree":
        hi = _log(rng, 1, 64)
        ctx = _log(rng, 1, 16384)
        room = min(32 * 8000 * 8 * 128 // (ctx * hk * hd), 32 * 32 * 8000 * 32 // (hi * (ctx + hi) * h))
        n = _log(rng, 1, max(1, min(128, room)))
        return dict(op=op, requests=n, lo=rng.randint(1, hi), hi=hi + 1, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx + 1,
                    heads=h, kv_heads=hk, head_dim=hd, cache=cache, slots=rng.choice([1, 2]), pad=rng.randint(0, 9))
    hi = _log(rng, 1, 4096)
    ctx = _log(rng, 1, 8192) if rng.random() < 0.6 else 1
    room = min(32 * 8192 * 4096 // (h * hi * (ctx + hi)), 8192 * 8 * 128 * 2 // ((ctx + hi) * hk * hd))
    n = _log(rng, 1, max(1, min(64, room)))
    return dict(op=op, requests=n, lo=rng.randint(1, hi), hi=hi + 1, ctx_lo=rng.randint(0, ctx - 1), ctx_hi=ctx,
                heads=h, kv_heads=hk, head_dim=hd, cache=cache, slots=rng.choice([1, 2]), pad=rng.randint(0, 40))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed) & 0x7FFFFFFF)


def _host(seed):
    return np.random.RandomState((int(seed) * 7919 + 11) & 0x7FFFFFFF)


def _int(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(DEVICE)


def _spread(r, lo, hi, n):
    """n numbers evenly from lo to hi - 1 in an order of the seed's: their sum is the case's."""
    return r.permutation(np.linspace(lo if n > 1 else max(lo, hi - 1), max(lo, hi - 1), n).astype(np.int64))


def _lengths(case, seed):
    """Rows and cached tokens of each request (host), from the seed."""
    r = _host(seed)
    n = case["requests"]
    return _spread(r, case["lo"], case["hi"], n), _spread(r, case["ctx_lo"], case["ctx_hi"], n)


def _filled(case, blocks, g):
    """A filled pool: keys with a few loud channels, as attention keys have."""
    shape = (blocks, case["slots"], 2, case["kv_heads"], PAGE, case["head_dim"])
    x = torch.empty(shape, device=DEVICE, dtype=torch.bfloat16).normal_(generator=g)
    x *= (1 + 3 * (torch.rand(case["kv_heads"], 1, case["head_dim"], generator=g, device=DEVICE) > 0.95)).to(x.dtype)
    if case["cache"] == "bf16":
        return x, None
    scales = torch.empty(shape[:-1], device=DEVICE)
    codes = torch.empty(shape, device=DEVICE, dtype=torch.uint8)
    step = max(1, (1 << 26) // max(1, x[0].numel()))
    for b in range(0, blocks, step):
        y = x[b:b + step].float()
        s = (y.abs().amax(-1) / E4M3_MAX).clamp_min(2.0 ** -126)
        scales[b:b + step] = s
        codes[b:b + step] = (y / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(torch.float8_e4m3fn), scales


def _inverse(rot, scaling):
    """Radians per position of each pair, and what cos and sin are multiplied by.  linear: positions divided by 8;
    base: the base grows so that the slowest pair turns 8 times slower; parts: pairs of few turns over the 4096
    positions that were trained turn 8 times slower, those of many as before, a ramp between them."""
    theta, factor, trained, low, high = 10000.0, 8.0, 4096, 1.0, 32.0
    j = np.arange(rot // 2, dtype=np.float64)
    if scaling == "base":
        theta *= factor ** (rot / max(rot - 2, 1))
    inv = theta ** (-2 * j / rot)
    if scaling == "linear":
        inv = inv / factor
    if scaling == "parts":
        keep = np.clip((trained * inv / (2 * math.pi) - low) / (high - low), 0, 1)
        return inv * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1
    return inv, 1.0


def _trees(r, counts, words):
    """A random draft for each request: visible[t] has the bits of node t and of what it follows."""
    n, most = len(counts), int(max(counts.max(), 1))
    seen = np.zeros((n, most, words), dtype=np.uint64)
    for t in range(most):
        # a node follows one of the last few, or the last committed token (-1)
        parent = np.maximum(t - 1 - r.randint(0, 4, size=n), -1)
        if t:
            seen[:, t] = np.where((parent >= 0)[:, None], seen[np.arange(n), np.maximum(parent, 0)], 0)
        seen[:, t, t // 64] |= np.uint64(1 << (t % 64))
    return np.concatenate([seen[i, :counts[i]] for i in range(n)]).view(np.int64)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "pages":
        return _prepare_pages(case, seed)
    if op == "rotate":
        rows, heads, hd = case["rows"], case["heads"] + case["kv_heads"], case["head_dim"]
        wide = (heads + case["kv_heads"]) * hd  # a row of the projection: queries, keys, values
        qkv = torch.randn(rows, wide, generator=g, device=DEVICE) * (0.5 + 3 * torch.rand(rows, 1, generator=g, device=DEVICE))
        x = qkv.to(torch.float32 if case["src"] == "fp32" else torch.bfloat16)[:, :heads * hd]
        start = torch.randint(0, case["far"], (1,), generator=g, device=DEVICE)
        pos = ((start + torch.arange(rows, device=DEVICE)) % (case["far"] + rows)).to(torch.int32)
        gain = [1 + 0.2 * torch.randn(hd, generator=g, device=DEVICE) for _ in range(2)] if case["norm"] else [None] * 2
        inv, factor = _inverse(case["rot"], case["scaling"])
        s = dict(case=case, x=x, pos=pos, q_gain=gain[0], k_gain=gain[1], inv=torch.from_numpy(inv).to(DEVICE),
                 factor=factor, out=torch.zeros(rows, heads * hd, dtype=x.dtype, device=DEVICE))
        if own:
            from continuous_depth_batching_gb300 import ops
            steps, f = ops.rope_steps(case["rot"], theta=10000.0, scaling=case["scaling"], factor=8.0, trained=4096)
            s["plan"] = ops.Rotary(case["heads"], case["kv_heads"], hd, steps, interleaved=case["interleaved"],
                                   factor=f, q_gain=s["q_gain"], k_gain=s["k_gain"], eps=1e-6)
        return s

    n, hk, hd = case["requests"], case["kv_heads"], case["head_dim"]
    if op == "keep":
        r = _host(seed)
        base = r.randint(max(0, case["ctx"] - 32), case["ctx"] + 1, size=n)
        keep = np.full(n, case["keep"])
        if n > 1:
            keep = r.randint(0, case["keep"] + 1, size=n)
        path = np.full((n, case["keep"]), -1)
        for i in range(n):  # nodes that are in place, then later ones
            same = r.randint(0, keep[i] + 1)
            if case["nodes"] - keep[i] < keep[i] - same:
                same = keep[i]
            path[i, :same] = np.arange(same)
            path[i, same:keep[i]] = np.sort(r.permutation(np.arange(keep[i], case["nodes"]))[:keep[i] - same])
        first, last = base // PAGE, (base + case["nodes"] - 1) // PAGE
        per = (case["nodes"] + PAGE - 2) // PAGE + 1  # pages that so many positions can touch
        # Only the pages of the draft exist; every other block table entry is empty.
        table = np.full((n, int(last.max()) + 1), -1)
        ids = r.permutation(n * per).reshape(n, per)
        for i in range(n):
            table[i, first[i]:last[i] + 1] = ids[i, :last[i] - first[i] + 1]
        pool, scales = _filled(case, n * per, g)
        s = dict(case=case, pool=pool, scales=scales, table=_int(table), base=_int(base), keep=_int(keep), path=_int(path))
        if own:
            from continuous_depth_batching_gb300 import ops
            s["plan"] = ops.PathKeeper(ops.PagedCache(pool, s["table"], scales))
        return s

    counts, ctx = _lengths(case, seed)
    rows = int(counts.sum()) + case["pad"]
    lens = ctx + counts
    need = (lens + PAGE - 1) // PAGE
    first = np.concatenate([[0], np.cumsum(need)])
    table = np.full((n, int(need.max())), -1)
    perm = _host(seed + 1).permutation(int(first[-1]))
    for i in range(n):
        table[i, :need[i]] = perm[first[i]:first[i + 1]]
    order = _host(seed + 2).permutation(n)  # request i is sequence order[i]
    by_seq = np.empty_like(table)
    by_seq[order] = table
    pool, scales = _filled(case, int(first[-1]), g)
    h = case["heads"]
    start = np.concatenate([[0], np.cumsum(counts)])
    s = dict(case=case, pool=pool, scales=scales, table=_int(by_seq), seq=_int(order), lens=_int(lens), row_start=_int(start),
             q=(1.3 * torch.randn(rows, h * hd, generator=g, device=DEVICE)).bfloat16(), slot=case["slots"] - 1,
             out=torch.zeros(rows, h * hd, dtype=torch.bfloat16, device=DEVICE), rows=int(counts.sum()),
             most=int(counts.max()), longest=int(lens.max()))
    if op == "tree":
        s["visible"] = torch.from_numpy(_trees(_host(seed + 3), counts, (case["hi"] - 1 + 63) // 64)).to(DEVICE)
        pad = torch.zeros(case["pad"], s["visible"].shape[1], dtype=torch.int64, device=DEVICE)
        s["visible"] = torch.cat([s["visible"], pad])
    if own:
        from continuous_depth_batching_gb300 import ops
        cache = ops.PagedCache(pool, s["table"], scales)
        if op == "tree":
            s["plan"] = ops.DraftAttention(cache, h, rows, n, case["hi"] - 1, s["longest"])
        else:
            s["plan"] = ops.PromptAttention(cache, h, rows, n, s["longest"])
    return s


def _dropped(case):
    return int(case["requests"] * case["drop"])


def _prepare_pages(case, seed):
    r = _host(seed)
    n = case["requests"]
    lens = r.randint(0, case["ctx"] + 1, size=n)
    new = _spread(r, case["lo"], case["hi"], n - _dropped(case))
    rows = int(new.sum()) + 13
    back = -np.minimum(r.randint(1, 40, size=_dropped(case)), lens[:_dropped(case)])
    new = np.concatenate([back, new])
    mix = r.permutation(n)
    lens, new = lens[mix], new[mix]
    have, want = (lens + PAGE - 1) // PAGE, (np.maximum(lens, lens + new) + PAGE - 1) // PAGE
    most = (case["ctx"] + max(case["hi"], case["lo"] + 1) + PAGE) // PAGE
    blocks = n * most + 100
    ids = r.permutation(blocks)
    table = np.full((n, most), -1)
    at = np.concatenate([[0], np.cumsum(have)])
    order = r.permutation(n)
    for i in range(n):
        table[order[i], :have[i]] = ids[at[i]:at[i + 1]]
    head = int(r.randint(0, 5 * blocks))
    ring = np.full(blocks, -1)
    free = ids[at[n]:]
    ring[(head + np.arange(len(free))) % blocks] = free
    s = dict(case=case, lens=_int(lens), new=_int(new), seq=_int(order), table=_int(table), free=_int(ring), rows=rows,
             state=torch.tensor([head, head + len(free)], device=DEVICE),
             lens_out=torch.zeros(n, dtype=torch.int32, device=DEVICE),
             state_out=torch.zeros(2, dtype=torch.int64, device=DEVICE))
    if own:
        from continuous_depth_batching_gb300 import ops
        s["plan"] = ops.PagePlanner(s["table"], s["free"], n, rows)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if not own:
        return {"pages": _plain_pages, "rotate": _plain_rotate, "prompt": _plain_attend, "tree": _plain_attend,
                "keep": _plain_keep}[op](state)
    plan = state["plan"]
    if op == "pages":
        p = plan(state["state"], state["lens"], state["new"], seq=state["seq"], state_out=state["state_out"],
                 lens_out=state["lens_out"])
        return {"row_start": p.row_start, "seq": p.seq, "pos": p.pos, "slot": p.slot, "lens": state["lens_out"],
                "state": state["state_out"], "table": state["table"], "free": state["free"]}
    if op == "rotate":
        return {"out": plan(state["x"], state["pos"], out=state["out"])}
    if op == "keep":
        plan(state["base"], state["path"], state["keep"])
        return _cache(state)
    if op == "tree":
        return {"out": plan(state["q"], state["row_start"], state["lens"], state["visible"], seq=state["seq"],
                            slot=state["slot"], out=state["out"])}
    return {"out": plan(state["q"], state["row_start"], state["lens"], seq=state["seq"], slot=state["slot"],
                        out=state["out"])}


def _cache(s):
    return {"cache": s["pool"]} if s["scales"] is None else {"cache": s["pool"], "scales": s["scales"]}


def _plain_pages(s):
    lens, new, seq, table, free, rows = s["lens"].long(), s["new"].long(), s["seq"].long(), s["table"], s["free"], s["rows"]
    head, tail = s["state"].unbind()
    after = (lens + new).clamp_min(0)
    grow = new.clamp_min(0)
    end = torch.cumsum(grow, 0)
    start = end - grow
    have, want = (lens + PAGE - 1) // PAGE, (after + PAGE - 1) // PAGE
    most = table.shape[1]
    page = torch.arange(most, device=lens.device)[None]
    taken, given = (want - have).clamp_min(0), (have - want).clamp_min(0)
    t0, g0 = torch.cumsum(taken, 0) - taken, torch.cumsum(given, 0) - given
    mine = table[seq].long()
    take = (page >= have[:, None]) & (page < want[:, None])
    mine = torch.where(take, free.long()[(head + t0[:, None] + page - have[:, None]) % free.shape[0]], mine)
    table[seq] = mine.to(torch.int32)
    give = (page >= want[:, None]) & (page < have[:, None])
    # what is not given goes to a place behind the ring
    to = torch.where(give, (tail + g0[:, None] + page - want[:, None]) % free.shape[0], free.shape[0])
    longer = torch.cat([free, free[:1]])
    longer[to.reshape(-1)] = mine.reshape(-1).to(torch.int32)
    free.copy_(longer[:-1])
    row = torch.arange(rows, device=lens.device)
    i = torch.searchsorted(end, row, right=True).clamp(max=lens.shape[0] - 1)
    on = row < end[-1]
    pos = lens[i] + row - start[i]
    slot = mine[i, (pos // PAGE).clamp(0, most - 1)] * PAGE + pos % PAGE
    s["state_out"].copy_(torch.stack([head + taken.sum(), tail + given.sum()]))
    s["lens_out"].copy_(after)
    return {"row_start": torch.cat([start, end[-1:]]).to(torch.int32), "seq": torch.where(on, seq[i], -1).to(torch.int32),
            "pos": torch.where(on, pos, -1).to(torch.int32), "slot": torch.where(on, slot, -1), "lens": s["lens_out"],
            "state": s["state_out"], "table": table, "free": free}


def _plain_rotate(s):
    c = s["case"]
    h, hd, rot, rows = c["heads"], c["head_dim"], c["rot"], c["rows"]
    x = s["x"].float().view(rows, -1, hd)
    if s["q_gain"] is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        x = torch.cat([x[:, :h] * s["q_gain"], x[:, h:] * s["k_gain"]], 1)
    a = s["pos"].double()[:, None] * s["inv"]
    cos, sin = (a.cos() * s["factor"]).float()[:, None], (a.sin() * s["factor"]).float()[:, None]
    if c["interleaved"]:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
    else:
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
    s["out"].copy_(torch.cat([y, x[..., rot:]], -1).reshape(rows, -1))
    return {"out": s["out"]}


def _plain_attend(s):
    c = s["case"]
    h, hk, hd, t, length = c["heads"], c["kv_heads"], c["head_dim"], s["most"], s["longest"]
    start, lens = s["row_start"].long(), s["lens"].long()
    counts = start[1:] - start[:-1]
    i = torch.arange(t, device=lens.device)
    row = (start[:-1, None] + i).clamp(max=s["rows"] - 1)  # [requests, most]
    q = s["q"][row].float().view(-1, t, hk, h // hk, hd)
    j = torch.arange(length, device=lens.device)
    block = s["table"][s["seq"].long()][:, j // PAGE].long().clamp_min(0)
    if s["scales"] is None:
        kv = s["pool"][block, s["slot"], :, :, j % PAGE].float()
    else:
        kv = s["pool"].view(torch.uint8)[block, s["slot"], :, :, j % PAGE].view(torch.float8_e4m3fn).float()
        kv = kv * s["scales"][block, s["slot"], :, :, j % PAGE][..., None]
    k, v = kv.unbind(2)  # [requests, length, kv_heads, head_dim]
    before = lens - counts
    if c["op"] == "tree":
        node = j[None] - before[:, None]  # [requests, length]
        word = (node // 64).clamp(0, s["visible"].shape[1] - 1)
        bits = s["visible"][row].gather(2, word[:, None].expand(-1, t, -1))
        see = (node[:, None] < 0) | (((bits >> (node % 64)[:, None]) & 1) == 1) & (node < counts[:, None])[:, None]
    else:
        see = j[None, None] <= before[:, None, None] + i[None, :, None]
    x = torch.einsum("ntkgd,nlkd->nkgtl", q, k) / math.sqrt(hd)
    x = x.masked_fill_(~see[:, None, None], -math.inf)
    x = torch.exp(x.sub_(x.amax(-1, keepdim=True)))
    o = torch.einsum("nkgtl,nlkd->nkgtd", x, v) / x.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(-1, h * hd)
    r = torch.arange(s["rows"], device=lens.device)
    of = torch.searchsorted(start[1:], r, right=True)
    s["out"][:s["rows"]] = o[of * t + r - start[of]].to(torch.bfloat16)
    return {"out": s["out"]}


def _plain_keep(s):
    base, path, keep = s["base"].long(), s["path"].long(), s["keep"].long()
    k = torch.arange(path.shape[1], device=path.device)[None]
    move = (k < keep[:, None]) & (path != k)
    i = torch.arange(path.shape[0], device=path.device)[:, None].expand_as(path)[move]
    old, new = (base[:, None] + path)[move], (base[:, None] + k)[move]
    a, b = s["table"][i, old // PAGE].long(), s["table"][i, new // PAGE].long()
    pool = s["pool"].view(torch.uint8) if s["scales"] is not None else s["pool"]
    pool[b, :, :, :, new % PAGE] = pool[a, :, :, :, old % PAGE]
    if s["scales"] is not None:
        s["scales"][b, :, :, :, new % PAGE] = s["scales"][a, :, :, :, old % PAGE]
    return _cache(s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _mean(case, lo, hi, n):
    a, b = case[lo], max(case[lo], case[hi] - 1)
    return (a + b) / 2 if n > 1 else b


def _cell(case):
    return case["head_dim"] * 2 if case["cache"] == "bf16" else case["head_dim"] + 4


def work(case):
    op = case["op"]
    if op == "pages":
        n = case["requests"]
        rows = (n - _dropped(case)) * _mean(case, "lo", "hi", n)
        return {"bytes": n * 20 + rows * 16 + rows / PAGE * 8 + _dropped(case) * 10, "flops": n + rows}
    if op == "rotate":
        each = (case["heads"] + case["kv_heads"]) * case["head_dim"]
        return {"bytes": case["rows"] * (2 * each * (4 if case["src"] == "fp32" else 2) + 4),
                "flops": case["rows"] * each * (8 if case["norm"] else 4)}
    hk, hd, n = case["kv_heads"], case["head_dim"], case["requests"]
    if op == "keep":
        moved = n * case["keep"] / (2 if n > 1 else 1) / 2
        return {"bytes": 2 * moved * case["slots"] * 2 * hk * _cell(case) + n * (8 + 4 * case["keep"]), "flops": moved}
    h = case["heads"]
    t, ctx = _mean(case, "lo", "hi", n), _mean(case, "ctx_lo", "ctx_hi", n)
    rows = n * t
    seen = ctx + (t + 1) / 2
    return {"bytes": n * (ctx + t) * 2 * hk * _cell(case) + 2 * rows * h * hd * 2, "flops": 4 * rows * seen * h * hd}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op == "pages":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "rotate":
        return _exact_rotate(s)
    if op == "keep":
        return _exact_keep(s)
    return _exact_attend(s)


def _exact_rotate(s):
    c = s["case"]
    hd, rot = c["head_dim"], c["rot"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEVICE)
    turn = s["factor"] * torch.exp(1j * (s["pos"].double()[:, None] * s["inv"][None, :]))
    for i in range(c["heads"] + c["kv_heads"]):
        y = s["x"][:, i * hd:(i + 1) * hd].double()
        gain = s["q_gain"] if i < c["heads"] else s["k_gain"]
        if gain is not None:
            y = y / torch.sqrt((y * y).sum(1, keepdim=True) / hd + 1e-6) * gain.double()
        to = out[:, i * hd:(i + 1) * hd]
        to[:] = y
        if c["interleaved"]:
            z = torch.view_as_complex(y[:, :rot].reshape(-1, rot // 2, 2).contiguous()) * turn
            to[:, :rot] = torch.view_as_real(z).reshape(-1, rot)
        else:
            z = torch.complex(y[:, :rot // 2].contiguous(), y[:, rot // 2:rot].contiguous()) * turn
            to[:, :rot // 2], to[:, rot // 2:rot] = z.real, z.imag
    return {"out": out}


def _exact_keep(s):
    r = {"cache": s["pool"].to(torch.float64)}
    if s["scales"] is not None:
        r["scales"] = s["scales"].double()
    base, keep, path, table = s["base"].tolist(), s["keep"].tolist(), s["path"].tolist(), s["table"].tolist()
    for i in range(len(base)):
        for k in range(keep[i]):
            a, b = base[i] + path[i][k], base[i] + k
            for of in r.values():
                of[table[i][b // PAGE], :, :, :, b % PAGE] = of[table[i][a // PAGE], :, :, :, a % PAGE]
    return r


def _exact_attend(s):
    c = s["case"]
    h, hk, hd = c["heads"], c["kv_heads"], c["head_dim"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEVICE)
    start, lens, seq = s["row_start"].tolist(), s["lens"].tolist(), s["seq"].tolist()
    if sum((start[i + 1] - start[i]) * lens[i] for i in range(len(lens))) * h * hd > 1 << 40:
        return None
    for i in range(len(lens)):
        t, length = start[i + 1] - start[i], lens[i]
        b = s["table"][seq[i], :(length + PAGE - 1) // PAGE].long()
        kv = s["pool"][b, s["slot"]].to(torch.float64)  # [pages, 2, kv_heads, 16, head_dim]
        if s["scales"] is not None:
            kv = kv * s["scales"][b, s["slot"]].double()[..., None]
        kv = kv.permute(1, 2, 0, 3, 4).reshape(2, hk, -1, hd)[:, :, :length]
        hidden = torch.ones(t, length, dtype=torch.bool, device=DEVICE).triu(length - t + 1)
        if c["op"] == "tree":
            seen = s["visible"][start[i]:start[i + 1]].cpu().numpy().view(np.uint64)
            u = np.arange(t)
            bits = (seen[:, u // 64] >> (u % 64).astype(np.uint64)) & np.uint64(1)
            hidden = torch.zeros(t, length, dtype=torch.bool, device=DEVICE)
            hidden[:, length - t:] = torch.from_numpy(bits == 0).to(DEVICE)
        q = s["q"][start[i]:start[i + 1]].double().view(t, h, hd)
        for head in range(h):
            x = q[:, head] @ kv[0, head * hk // h].T * hd ** -0.5
            x[hidden] = -math.inf
            out[start[i]:start[i + 1], head * hd:(head + 1) * hd] = torch.softmax(x, -1) @ kv[1, head * hk // h]
    return {"out": out}
