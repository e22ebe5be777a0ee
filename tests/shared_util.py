"""Decode over shared prefixes: cases, a plain computation in 64 bits with the bound its kernels have to keep, and the
planner's arithmetic in Python."""
import math
import random

import torch

PAGE = 64
BF16 = torch.bfloat16
HALF = 2.0 ** -8          # half a step of bf16, relative


class Case:
    """groups: (rows, shared pages) of each; own: lengths of the rows' own positions (the new one last), cycled."""

    def __init__(self, groups, own, heads, kv_heads, D, window=0, sinks=False, theta=10000.0, seed=0, spare=3, poison=True):
        g = torch.Generator().manual_seed(seed)
        rng = random.Random(seed)
        self.heads, self.kv_heads, self.D, self.window = heads, kv_heads, D, window
        self.groups = groups
        rows = [(i, p) for i, (n, p) in enumerate(groups) for _ in range(n)]
        self.rows = len(rows)
        own = [own[r % len(own)] for r in range(self.rows)]
        self.positions = torch.tensor([p * PAGE + n - 1 for (_, p), n in zip(rows, own)], dtype=torch.int32)
        self.width = max([(int(p) + PAGE) // PAGE for p in self.positions] + [1]) + 1
        need = sum(p for _, p in groups) + sum(-(-n // PAGE) for n in own)
        self.num_pages = need + spare
        ids = list(range(self.num_pages))
        rng.shuffle(ids)
        common = []
        for _, p in groups:
            common.append([ids.pop() for _ in range(p)])
        table = []
        for (i, p), n in zip(rows, own):
            mine = common[i] + [ids.pop() for _ in range(-(-n // PAGE))]
            table.append(mine + [-1] * (self.width - len(mine)))
        self.table = torch.tensor(table, dtype=torch.int32).view(self.rows, self.width)
        self.start = torch.tensor([sum(n for n, _ in groups[:i]) for i in range(len(groups) + 1)], dtype=torch.int32)
        self.pages = torch.tensor([p for _, p in groups], dtype=torch.int32)

        def normal(*shape):
            return torch.randn(*shape, generator=g).to(BF16)

        self.q, self.k, self.v = (normal(self.rows, h, D) for h in (heads, kv_heads, kv_heads))
        self.k_pool, self.v_pool = (normal(self.num_pages, kv_heads, PAGE, D) for _ in range(2))
        self.sinks = normal(heads) if sinks else None
        self.cos = self.sin = None
        if theta > 0:
            f = torch.exp(torch.arange(D // 2, dtype=torch.float64) * (-2.0 / D * math.log(theta)))
            angle = torch.arange(self.width * PAGE, dtype=torch.float64)[:, None] * f
            angle = torch.cat([angle, angle], -1)
            self.cos, self.sin = torch.cos(angle).to(BF16), torch.sin(angle).to(BF16)
        if poison:
            self._poison()

    def _poison(self):
        """Every slot that no row sees holds a NaN."""
        seen = torch.zeros(self.num_pages, PAGE, dtype=torch.bool)
        for r, pos in enumerate(self.positions.tolist()):
            t = torch.arange(self.low(pos), pos + 1)
            seen[self.table[r].long()[t // PAGE], t % PAGE] = True
        for pool in (self.k_pool, self.v_pool):
            pool[(~seen)[:, None].expand(-1, self.kv_heads, -1)] = float("nan")

    def low(self, pos):
        return max(0, pos - self.window + 1) if self.window > 0 else 0

    def rope(self, x, r):
        """Row r's vectors rotated as the kernels do: f32 products and sum, one rounding."""
        if self.cos is None:
            return x[r]
        c, s = (t[int(self.positions[r])].float() for t in (self.cos, self.sin))
        y, h = x[r].float(), self.D // 2
        return (y * c + torch.cat([-y[..., h:], y[..., :h]], -1) * s).to(BF16)

    def write(self, skip=()):
        """New keys and values put into the pools."""
        for r, pos in enumerate(self.positions.tolist()):
            if r not in skip:
                page = int(self.table[r, pos // PAGE])
                self.k_pool[page, :, pos % PAGE], self.v_pool[page, :, pos % PAGE] = self.rope(self.k, r), self.v[r]

    def want(self, skip=()):
        """(outputs, bounds) in 64 bits, from the pools as they are.

        A weight is rounded to bf16 (HALF of it) where it meets its value, and the sum that divides it is of rounded or
        unrounded weights: 2 HALF of sum w |v|.  A score is a sum of D products in f32, off by less than D 2^-24 of
        sum |q k|, and 2^x by 2^-22, which moves a weight and its sum by twice as much.  The output rounds once more."""
        out = torch.zeros(self.rows, self.heads, self.D, dtype=torch.float64)
        bound = torch.zeros_like(out)
        scale = float(torch.tensor(1.0 / math.sqrt(self.D)))
        for r, pos in enumerate(self.positions.tolist()):
            if r in skip:
                continue
            t = torch.arange(self.low(pos), pos + 1)
            page = self.table[r].long()[t // PAGE]
            k, v = (pool[page, :, t % PAGE].double().transpose(0, 1) for pool in (self.k_pool, self.v_pool))   # [Hk, t, D]
            q = self.rope(self.q, r).double().view(self.kv_heads, -1, self.D)
            score = (q @ k.transpose(1, 2)) * scale
            norm = torch.logsumexp(score, -1, keepdim=True)
            if self.sinks is not None:
                norm = torch.logaddexp(norm, self.sinks.double().view(self.kv_heads, -1, 1))
            w = torch.exp(score - norm)
            size = (q.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True) * scale
            off = 2 * HALF + 2 * (self.D * 2.0 ** -24 * size + 2.0 ** -22)
            out[r], bound[r] = ((w @ v).reshape(self.heads, -1), (off * (w @ v.abs())).reshape(self.heads, -1))
        return out, bound + HALF * (out.abs() + bound) + 1e-30


def shared_slots(groups, group_size, kv_heads, ctas, min_pages=6, min_saved=24):
    """The partial slots that the pieces of every (tile, kv head) take, as the kernels place them, checked for being
    each piece's own; returns (units, units per CTA, one past the last slot)."""
    per = 2 * (128 // group_size)
    shared = [(i, n, (p + 1) // 2) for i, (n, p) in enumerate(groups) if p >= min_pages and (n - 1) * p >= min_saved]
    total = sum(-(-n // per) * nb * kv_heads for _, n, nb in shared)
    share = max(-(-total // ctas), 1)
    unit, s1, s2, end = 0, 0, 0, 0
    for i, n, nb in shared:
        slot0 = s1 // share + 2 * s2 + i
        assert slot0 >= end
        most = (nb + share - 2) // share + 1
        for t in range(-(-n // per)):
            for h in range(kv_heads):
                u = unit + (t * kv_heads + h) * nb
                assert 1 <= (u + nb - 1) // share - u // share + 1 <= most and (u + nb - 1) // share < ctas
        end = slot0 + n * kv_heads * most
        unit += -(-n // per) * nb * kv_heads
        s1 += n * kv_heads * nb
        s2 += n * kv_heads
    assert unit == total
    return total, share, end


def own_runs(units, ctas, start=3):
    """(long, short) runs of the rows' own pages: how many, and their number in all."""
    share = -(-units // ctas)
    even = share <= 6 * (start + 1)
    big = max(share, start + 1) if even else share // 4 * 3
    small = big if even else max((share + 15) // 16, 5 * (start + 1))
    x = min(units, big * ctas)
    assert -(-x // big) <= ctas
    return -(-x // big) + -(-(units - x) // small)
