"""Decode over shared prefixes where scores are large, on the GPU: outputs are those of the keys with the largest score.

A query holds 2^a in its first dimension and zeros, a key n 2^e with |n| < 128, so that a score is one product, exact in
f32, and two keys of different n differ by far more than the 2^-24 of a score that f32 arithmetic may lose.  In 64 bits the
weights are then 0 and 1 / count, and the output is the mean of the values of the keys with the largest n."""
import pytest
import torch

from gpu_util import binding
from shared_util import BF16, HALF, PAGE, Case

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def far_case(D, exponent, sign, seed, groups, own):
    """n of the shared keys is in [-120, 120] but for a few of 125; own keys lie below, at and above it.  With sign -1 the
    queries are negative, and so are the largest scores where every key's n is positive."""
    c = Case(groups, own, 8, 2, D, theta=0.0, seed=seed, poison=False)
    g = torch.Generator().manual_seed(seed)
    half = exponent // 2
    c.q.zero_(), c.k_pool.zero_(), c.k.zero_()
    c.q[..., 0] = sign * 2.0 ** half
    low = 1 if sign < 0 else -120
    n = torch.randint(low, 121, (c.num_pages, 2, PAGE), generator=g).float()
    for r, (page, pos) in enumerate(zip(c.table.tolist(), c.positions.tolist())):
        shared = int(c.pages[sum(1 for s in c.start[1:-1].tolist() if s <= r)])
        best = 125.0 if sign > 0 else 0.5
        n[page[0], :, 5] = n[page[shared - 1], :, 63] = n[page[shared // 2], 0, 17] = best
        if pos // PAGE > shared:                       # a row with whole pages of its own
            n[page[shared], 1, 9] = best if r % 2 else 2 * best
    c.k_pool[..., 0] = (n * 2.0 ** (exponent - half)).to(BF16)
    new = torch.tensor([[3.0, 125.0], [125.0, 126.0], [7.0, 1.0]]) if sign > 0 else torch.tensor([[3.0, 0.5], [0.5, 0.25], [7.0, 1.0]])
    c.k[..., 0] = (new[torch.arange(c.rows) % 3] * 2.0 ** (exponent - half)).to(BF16)
    return c


def means(c):
    """(outputs, bounds): a weight is 2^x with |x| <= 8 and x the same for equal scores of one piece, by 2^-22 apart
    between pieces, rounded to bf16; the sum that divides it is of such weights."""
    out = torch.zeros(c.rows, c.heads, c.D, dtype=torch.float64)
    size = torch.zeros_like(out)
    for r, pos in enumerate(c.positions.tolist()):
        t = torch.arange(pos + 1)
        page = c.table[r].long()[t // PAGE]
        k, v = (pool[page, :, t % PAGE].double().transpose(0, 1) for pool in (c.k_pool, c.v_pool))
        score = c.q[r].double().view(c.kv_heads, -1, c.D) @ k.transpose(1, 2)
        w = (score == score.amax(-1, keepdim=True)).double()
        w = w / w.sum(-1, keepdim=True)
        out[r], size[r] = (w @ v).reshape(c.heads, -1), (w @ v.abs()).reshape(c.heads, -1)
    bound = (2 * HALF + 2 * 2.0 ** -22) * size
    return out, bound + HALF * (out.abs() + bound)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("exponent", [20, 24, 27, 30, 33, 40, 64, 100])
@pytest.mark.parametrize("groups,own", [([(20, 12), (9, 7)], [3, 70]), ([(65, 9)], [1, 130, 64])])
def test_far_scores(D, sign, exponent, groups, own):
    c = far_case(D, exponent, sign, D + exponent, groups, own)
    b = binding()
    up = lambda t: t.cuda()
    q, k, v, pos, table, start, pages, kp, vp = map(up, (c.q, c.k, c.v, c.positions, c.table, c.start, c.pages, c.k_pool, c.v_pool))
    p = b.make_params(c.rows, c.heads, c.kv_heads, D, c.width, c.num_pages, BF16)
    ws, out = b.new_shared_workspace(p, len(groups)), torch.full_like(q, 7.0)
    b.decode_shared(p, q, k, v, pos, table, start, pages, kp, vp, out, ws)
    b.check_status(ws)
    c.write()
    want, bound = means(c)
    err = (out.cpu().double() - want).abs()
    assert (err <= bound).all(), (int((~(err <= bound)).sum()), int((~torch.isfinite(out)).sum()))
