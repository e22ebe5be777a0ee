"""The operators for many continuations of one prompt as they are used together, against what each sample has seen, kept
on the host: pages forked and copied, keys rotated, prompt pages attended once for all samples."""
import pytest
import torch

from gpu_util import binding
from pages_util import PAGE, State
from shared_util import BF16, HALF
from test_gpu_rotary import hold, turned

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


class History:
    """Keys and values [n, kv_heads, D] of every row, position by position."""

    def __init__(self, rows):
        self.k, self.v = [[None] * rows for _ in range(2)]

    def fork(self, parents, keep):
        self.k, self.v = ([None if p < 0 else x[p][:n].clone() for p, n in zip(parents, keep)] for x in (self.k, self.v))

    def append(self, k, v):
        self.k, self.v = ([torch.cat([a, b[r:r + 1]]) for r, a in enumerate(x)] for x, b in ((self.k, k), (self.v, v)))

    def want(self, q):
        """(outputs, bounds) as in tests/shared_util.py, from the history alone."""
        D = q.shape[-1]
        scale, out, bound = float(torch.tensor(D ** -0.5)), torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
        for r in range(q.shape[0]):
            k, v = (x[r].double().transpose(0, 1) for x in (self.k, self.v))
            qr = q[r].double().view(k.shape[0], -1, D)
            score = (qr @ k.transpose(1, 2)) * scale
            w = torch.softmax(score, -1)
            size = (qr.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True) * scale
            off = 2 * HALF + 2 * (D * 2.0 ** -24 * size + 2.0 ** -22)
            out[r], bound[r] = (w @ v).reshape(-1, D), (off * (w @ v.abs())).reshape(-1, D)
        return out, bound + HALF * (out.abs() + bound)


def same_bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("inter,D,heads,kv", [(True, 64, 8, 2), (False, 128, 6, 3)])
def test_samples_against_what_they_have_seen(inter, D, heads, kv):
    b = binding()
    rows, width, N = 6, 12, 60
    g = torch.Generator(device="cuda").manual_seed(3)
    rot = b.make_rotary(D, 10000.0, rot_dim=32, interleaved=inter, scaling="ramp", factor=4.0, low=1.0, high=32.0,
                        original_len=256)
    p = b.make_params(rows, heads, kv, D, width, N, BF16)
    kp, vp = (torch.randn(N, kv, PAGE, D, generator=g, device="cuda").to(BF16) for _ in range(2))
    prompt = 7 * PAGE + 20
    s = State(rows, width, N, [prompt] + [0] * (rows - 1), seed=1)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table, lengths, refs = ints(s.table), ints(s.lengths), ints(s.refs)
    cache, pws, rws = b.make_pages(p, [kp, vp]), b.new_pages_workspace(p), b.new_status()
    sws = b.new_shared_workspace(p, 2)
    start, count = ints([0, rows, rows]), ints([7, 0])

    def seen(pool, r, n):
        t = torch.arange(n, device="cuda")
        return pool[table[r].long()[t // PAGE], :, t % PAGE].cpu()

    past = History(rows)
    past.k[0], past.v[0] = seen(kp, 0, prompt), seen(vp, 0, prompt)
    held = [prompt] + [0] * (rows - 1)
    for step in range(60):
        parents = [0] * rows if step == 0 else [2, 2, 2, 4, 4, 5] if step in (30, 31) else list(range(rows))
        back = [9 if step == 40 and r % 2 else 0 for r in range(rows)]          # some rows give positions back
        keep = [held[x] - d for x, d in zip(parents, back)]
        if any(back):
            b.pages_update(p, cache, table, lengths, refs, ints(parents), ints(keep), pws)
            lengths = ints(keep)
            past.fork(parents, keep)
            parents = list(range(rows))
        new = ints([n + 1 for n in keep])
        b.pages_update(p, cache, table, lengths, refs, ints(parents), new, pws)
        b.check_status(pws)
        if not any(back):
            past.fork(parents, keep)
        lengths, held = new, [n + 1 for n in keep]
        positions = lengths - 1
        q, k, v = (torch.randn(rows, h, D, generator=g, device="cuda").to(BF16) for h in (heads, kv, kv))
        qr, kr, out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
        b.rotary_apply(rot, q, k, positions, qr, kr, rws)
        b.decode_shared(p, qr, kr, v, positions, table, start, count, kp, vp, out, sws)
        for ws in (rws, sws):
            b.check_status(ws)
        hold(qr, *turned(rot, q, positions, False), BF16)
        hold(kr, *turned(rot, k, positions, False), BF16)
        past.append(kr.cpu(), v.cpu())
        for r, n in enumerate(held):
            assert same_bits(seen(kp, r, n), past.k[r]) and same_bits(seen(vp, r, n), past.v[r]), (step, r)
        want, bound = past.want(qr.cpu())
        err = (out.cpu().double() - want).abs()
        assert (err <= bound).all(), (step, float((err / bound).max()))
    b.pages_compact(p, cache, table, lengths, refs, torch.empty_like(refs), pws)
    b.check_status(pws)
    assert int(table.max()) < int((refs > 0).sum())
    for r, n in enumerate(held):
        assert same_bits(seen(kp, r, n), past.k[r]) and same_bits(seen(vp, r, n), past.v[r]), r
