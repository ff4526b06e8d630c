"""How exact queries meet an e4m3 cache in prompt and draft attention, with channels of q far louder than the others,
against float64.

The loud channels of the keys are 0, so that scores are sums of the quiet ones; those of a key have one sign, so that what is
lost of equal elements of a query adds up.  Tolerance: the query's elements are exact
down to 2^-14 of the head's largest, and within 2^-21 of that below; a score is then off by that times sum |k|, and
by head_dim fp32 steps of 2^-23 of S = |scale| * sum |q k|; a weight by 2^-11 of itself or 2^-33 of the largest, 2^-20 for the
exponential; both enter twice (numerator, sum).  The weighted sum adds 2^-23 of max |v| for every 16 keys and joined range, the
output's rounding 2^-8 of its value."""

import pytest

from tests.test_gpu_prompt_attention import make, run, tree, visible

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("loud", [100, 1000, 8000])
@pytest.mark.parametrize("heads,hk,hd", [(8, 2, 128), (4, 4, 96), (6, 2, 64), (3, 1, 32)])
@pytest.mark.parametrize("counts,cached", [([20], [300]), ([200], [64]), ([7, 150], [3000, 10])])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("equal", [False, True])
def test_a_loud_channel_of_q_leaves_the_others_their_bits(loud, heads, hk, hd, counts, cached, draft, equal):
    import torch
    cs = make("e4m3", heads, hk, hd, counts, cached, seed=loud + hd, **(dict(mask=tree, words=4) if draft else {}))
    channel = hd // 2 + 5
    k8 = cs["cache"].pool.view(torch.uint8)[:, :, 0]
    sign = torch.randint(0, 2, k8.shape[:-1], device="cuda", dtype=torch.uint8)[..., None]
    k8.copy_((k8 & 0x7F) | sign << 7)
    k8[..., channel] = 0
    cs["vals"][:, :, 0] = cs["vals"][:, :, 0].abs() * (1 - 2 * sign.double())
    cs["vals"][:, :, 0, :, :, channel] = 0
    q = cs["q"].view(-1, heads, hd)
    if equal:
        q.fill_(0.75 + 2.0 ** -7)
    q[:, :, channel] = loud * 1.5 * torch.where(torch.rand(q.shape[:2], device="cuda") < 0.5, -1.0, 1.0).bfloat16()
    got = run(cs)
    scale = hd ** -0.5
    for i, c in enumerate(counts):
        length, r0 = int(cs["L"][i]), int(cs["start"][i])
        j = torch.arange(length)
        blk = torch.from_numpy(cs["table"][cs["s"][i], (j // 16).numpy()]).long().cuda()
        kv = cs["vals"][blk, cs["slot"], :, :, (j % 16).cuda()]
        k, v = kv[:, 0], kv[:, 1]
        x = q[r0:r0 + c].double().view(c, hk, heads // hk, hd)
        see = torch.from_numpy(visible(cs, i)).cuda()[:, None, None]
        s = torch.einsum("tkgd,lkd->tkgl", x, k) * scale
        p = torch.softmax(torch.where(see, s, -torch.inf), -1)
        o = torch.einsum("tkgl,lkd->tkgd", p, v)
        size = torch.einsum("tkgd,lkd->tkgl", x.abs(), k.abs()).amax() * scale
        top = x.abs().amax(-1, keepdim=True)
        small = torch.einsum("tkgd,lkd->tkgl", (x.abs() < 2.0 ** -14 * top).double() * top, k.abs()).amax() * scale
        w = 2.0 ** -11 + length * 2.0 ** -33 + 2.0 ** -21 * small + hd * 2.0 ** -23 * size + 2.0 ** -20
        tol = 2.0 ** -8 * o.abs() + v.abs().amax() * (2 * w + (16 + length / 8) * 2.0 ** -23)
        err = (got[r0:r0 + c, :heads * hd].double().view(o.shape) - o).abs()
        assert (err <= tol).all(), (i, float((err / tol).max()))
