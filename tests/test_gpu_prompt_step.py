"""The operators for prompts and drafts together, as a program uses them: pages planned, queries and keys rotated, the
cache written, prompts and a drafted tree attended to, the accepted path kept and the rest given back, the next token
decoded.  Against float64 over the text so far.

Tolerances: those of tests/test_gpu_prompt_attention.py; queries and keys are read back from the cache writer's outputs
and the cache, so that each step is held to its own error."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

H, HK, HD = 8, 2, 64
WIDTH = (H + 2 * HK) * HD


def i32(v):
    import torch
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def read(cache, seq, positions):
    """float64 keys and values [positions, kv_heads, head_dim] as the cache holds them."""
    import torch
    j = torch.as_tensor(np.asarray(positions), device="cuda").long()
    blk = cache.block_table[seq, j // 16].long()
    kv = cache.pool[blk, 0, :, :, j % 16].double()
    if cache.scales is not None:
        kv = kv * cache.scales[blk, 0, :, :, j % 16].double()[..., None]
    return kv[:, 0], kv[:, 1]


def close(got, q, k, v, see, e4m3):
    import torch
    q = q.double().view(-1, HK, H // HK, HD)
    x = torch.einsum("tkgd,lkd->tkgl", q, k) * HD ** -0.5
    x = torch.where(see[:, None, None], x, -torch.inf)
    o = torch.einsum("tkgl,lkd->tkgd", torch.softmax(x, -1), v)
    S = torch.einsum("tkgd,lkd->tkgl", q.abs(), k.abs()).amax() * HD ** -0.5
    top = q.abs().amax(-1, keepdim=True)
    small = torch.einsum("tkgd,lkd->tkgl", (q.abs() < 2.0 ** -8 * top).double() * top, k.abs()).amax() * HD ** -0.5
    w = 2.0 ** -11 + len(k) * 2.0 ** -33 + 2.0 ** -17 * small if e4m3 else 2.0 ** -17
    tol = 2.0 ** -8 * o.abs() + v.abs().max() * (2 * (HD * 2.0 ** -23 * S + 2.0 ** -20 + w) + (16 + len(k) / 8) * 2.0 ** -23)
    err = (got.double().view(o.shape) - o).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("graphs", [False, True])
def test_prompts_a_draft_and_the_next_token(dtype, graphs):
    import torch
    from continuous_depth_batching_gb300 import ops
    rng = np.random.default_rng(4)
    n, blocks, max_rows = 3, 64, 300
    e4m3 = dtype == "e4m3"
    shape = (blocks, 1, 2, HK, 16, HD)
    pool = torch.full(shape, 0xFF, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) if e4m3 else \
        torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    scales = torch.full(shape[:-1], float("nan"), device="cuda") if e4m3 else None
    table = torch.full((n, 20), -1, dtype=torch.int32, device="cuda")
    cache = ops.PagedCache(pool, table, scales)
    planner = ops.PagePlanner(table, i32(rng.permutation(blocks)), n, max_rows)
    state, lens = torch.tensor([0, blocks], device="cuda"), i32([0, 0, 0])
    steps, factor = ops.rope_steps(HD, scaling="parts", factor=4.0, trained=64)
    rotary = ops.Rotary(H, HK, HD, steps, interleaved=True, factor=factor)
    writer = ops.CacheWriter(cache, H)
    prompt, draft = ops.PromptAttention(cache, H, max_rows, n), ops.DraftAttention(cache, H, max_rows, n, 64)
    keeper, decode = ops.PathKeeper(cache), ops.DecodeAttention(cache, H, n)
    qkv = torch.zeros(max_rows, WIDTH, device="cuda")
    turn = torch.zeros(max_rows, dtype=torch.int32, device="cuda")  # positions of the rotation
    new, q, out = i32([0, 0, 0]), torch.zeros(max_rows, H * HD, dtype=torch.bfloat16, device="cuda"), \
        torch.zeros(max_rows, H * HD, dtype=torch.bfloat16, device="cuda")
    visible = torch.zeros(max_rows, 1, dtype=torch.int64, device="cuda")
    plan = planner._out

    def forward(attend):
        rotary(qkv, turn)
        writer(qkv, plan.seq, plan.pos, q_out=q)
        attend()

    attends = {"prompt": lambda: prompt(q, plan.row_start, lens, out=out), "draft": lambda: draft(q, plan.row_start, lens, visible, out=out)}
    held = {}
    if graphs:  # one graph for each, replayed at other lengths than they were captured with
        turn.fill_(-1)
        planner(state, lens, new)
        for name, a in attends.items():
            forward(a)
            torch.cuda.synchronize()
            held[name] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(held[name]):
                forward(a)

    def step(name, counts, depth=None):
        """Rows for `counts` new tokens of each request; their results."""
        new.copy_(i32(counts))
        planner(state, lens, new)
        rows = int(sum(counts))
        qkv.normal_()
        turn.copy_(plan.pos)
        if depth is not None:
            turn[:rows] = depth
        if graphs:
            held[name].replay()
        else:
            forward(attends[name])
        for op in (planner, writer, prompt, draft):
            op.check()
        return rows

    counts = [37, 5, 130]
    text = np.zeros(n, dtype=int)
    for counts in ([37, 5, 130], [20, 1, 3]):  # prompts, in two chunks
        rows = step("prompt", counts)
        assert lens.tolist() == (text + counts).tolist()
        at = 0
        for i, c in enumerate(counts):
            k, v = read(cache, i, np.arange(text[i] + c))
            see = torch.ones(c, text[i] + c, dtype=torch.bool, device="cuda").tril(int(text[i]))
            close(out[at:at + c], q[at:at + c], k, v, see, e4m3)
            at += c
        text += counts
        assert at == rows

    # a tree of drafted tokens for each request
    parents = [[-1, 0, 0, 1, 3], [-1], [-1, -1, 0, 1, 1, 2, 5, 4, 6]]
    counts = [len(p) for p in parents]
    depths = [[] for _ in parents]
    for d, p in zip(depths, parents):
        for u in p:
            d.append(0 if u < 0 else d[u] + 1)
    visible[:sum(counts)] = torch.cat([ops.draft_mask(p, words=1) for p in parents])
    rows = step("draft", counts, i32(np.concatenate([text[i] + np.array(d) for i, d in enumerate(depths)])))
    at = 0
    for i, c in enumerate(counts):
        k, v = read(cache, i, np.arange(text[i] + c))
        see = torch.zeros(c, text[i] + c, dtype=torch.bool, device="cuda")
        see[:, :text[i]] = True
        for u in range(c):
            w = u
            while w >= 0:
                see[u, text[i] + w] = True
                w = parents[i][w]
        close(out[at:at + c], q[at:at + c], k, v, see, e4m3)
        at += c

    # what is accepted goes to its place, the rest is given back
    paths = [[0, 1, 3], [], [0, 2, 5, 6, 8]]
    kept = [read(cache, i, text[i] + np.array(p, dtype=int)) for i, p in enumerate(paths)]
    path = np.full((n, 6), 63)
    for i, p in enumerate(paths):
        path[i, :len(p)] = p
    keeper(i32(text), i32(path), i32([len(p) for p in paths]))
    keeper.check()
    new.copy_(i32([len(p) - c for p, c in zip(paths, counts)]))
    planner(state, lens, new)
    planner.check()
    text += [len(p) for p in paths]
    assert lens.tolist() == text.tolist()
    assert int(state[1] - state[0]) == blocks - sum(-(-int(t) // 16) for t in text)
    for i, p in enumerate(paths):
        k, v = read(cache, i, np.arange(text[i] - len(p), text[i]))
        assert torch.equal(k, kept[i][0]) and torch.equal(v, kept[i][1])

    # the next token of each, by the decode operator and as a prompt of one row
    step("prompt", [1, 1, 1])
    text += 1
    one = decode(q[:n], plan.seq[:n], plan.pos[:n])
    for i in range(n):
        k, v = read(cache, i, np.arange(text[i]))
        see = torch.ones(1, text[i], dtype=torch.bool, device="cuda")
        close(one[i:i + 1], q[i:i + 1], k, v, see, e4m3)
        close(out[i:i + 1], q[i:i + 1], k, v, see, e4m3)


@pytest.mark.parametrize("draft", [False, True])
def test_blocks_behind_32_bits_of_elements(draft):
    """Pages at the end of a pool of more than 2^32 elements."""
    import torch
    from continuous_depth_batching_gb300 import ops
    from tests.test_gpu_prompt_attention import check, make, tree
    heads, hk, hd = 16, 16, 128
    cs = make("bf16", heads, hk, hd, [40, 7], [300, 20], slots=1, slot=0, seed=2, **(dict(mask=tree) if draft else {}))
    old = cs["cache"]
    blocks = (1 << 32) // (2 * hk * 16 * hd) + 64
    pool = torch.empty(blocks, 1, 2, hk, 16, hd, dtype=torch.bfloat16, device="cuda")
    shift = blocks - old.pool.shape[0]
    pool[shift:] = old.pool
    table = torch.where(old.block_table >= 0, old.block_table + shift, -1).to(torch.int32)
    cs["cache"] = ops.PagedCache(pool, table)
    check(cs)
    keeper = ops.PathKeeper(cs["cache"])
    s = cs["s"][0]
    before = pool[shift:].clone()
    keeper(i32([300]), i32([[3, 9, 30]]), i32([3]), seq=i32([s]))
    keeper.check()
    t = cs["table"][s]
    for k, p in enumerate((3, 9, 30)):
        a, b = 300 + p, 300 + k
        assert torch.equal(pool[shift + t[b // 16], :, :, :, b % 16], before[t[a // 16], :, :, :, a % 16])


def test_objects_on_other_streams_keep_their_memory():
    """A dropped object's memory waits for every stream that called it; torch.cuda._sleep holds the stream up."""
    import gc

    import torch
    from continuous_depth_batching_gb300 import ops
    from tests.test_gpu_operator_streams import freed_for
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    cache = ops.PagedCache(torch.randn(8, 1, 2, HK, 16, HD, device="cuda").bfloat16(), table)
    side = torch.cuda.Stream()
    q, out = torch.randn(6, H * HD, device="cuda").bfloat16(), torch.zeros(6, H * HD, dtype=torch.bfloat16, device="cuda")
    start, lens, visible = i32([0, 2, 6]), i32([40, 50]), torch.full((6, 1), -1, dtype=torch.int64, device="cuda")
    path = i32([[0], [0]])  # made before: a copy from the host would wait for the stream
    ring, state, new, seq = i32([9] * 8), torch.tensor([0, 0], device="cuda"), i32([0, 0]), i32([0, 1])
    for held in (0, 1_000_000_000):  # the first calls load the kernels
        objects = [ops.PromptAttention(cache, H, 6, 2), ops.DraftAttention(cache, H, 6, 2, 64), ops.PagePlanner(table, ring, 2, 50),
                   ops.PathKeeper(cache)]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(held)
            objects[0](q, start, lens, out=out)
            objects[1](q, start, lens, visible, out=out)
            objects[2](state, lens, new, seq=seq)
            objects[3](lens, path, new)
    mine = [objects[0].workspace, objects[1].workspace, objects[2].slot] + [o.status for o in objects]
    old, sizes, types = {m.data_ptr() for m in mine}, [m.numel() for m in mine], [m.dtype for m in mine]
    del objects, mine
    gc.collect()
    new_ones = freed_for(sizes, types)
    assert not side.query(), "the calls were done too early to show anything"
    assert not old & new_ones
    torch.cuda.synchronize()
