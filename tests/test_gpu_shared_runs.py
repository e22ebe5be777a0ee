"""Decode over shared prefixes with work for many runs of the rows' own pages: a long run for each CTA, short ones from a
cursor, and rows that span several of them.  Outputs within the bound of tests/shared_util.py, and the same bits each time
whatever CTA takes which run."""
import random

import pytest
import torch

from gpu_util import binding
from shared_util import BF16, PAGE, Case, own_runs

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

START = 3                       # what a pair's start counts, in pages


def pairs(c):
    """(first unit, one past the last) of the pages of every (row, kv head) with its own pages, in order; units in all."""
    out, x = [], 0
    for pos, shared in zip(c.positions.tolist(), c.row_pages):
        n = pos // PAGE - shared + 1
        for _ in range(c.kv_heads):
            out.append((x + START, x + START + n))
            x += START + n
    return out, x


def whole_short_runs(c, ctas):
    """Short runs (taken from the cursor) that lie inside one pair, for each number of CTAs that may take own pages."""
    where, units = pairs(c)
    share = -(-units // ctas)
    assert share > 6 * (START + 1) and own_runs(units, ctas) > ctas
    long_, short = share // 4 * 3, max((share + 15) // 16, 5 * (START + 1))
    at = long_ * ctas
    return sum(max(0, (e - at) // short - max(0, -(-(s - at) // short))) for s, e in where if e > at)


def many_runs(D, heads, kv_heads, seed, sinks=False):
    """256 rows in three groups, own lengths of 1 to 1500; the first and the last rows hold more than 100 own pages."""
    rng = random.Random(seed)
    own = [rng.choice([1, 63, 64, 65, rng.randint(1, 1500), rng.randint(700, 1500)]) for _ in range(256)]
    own[0], own[128], own[254], own[255] = 110 * PAGE + 1, 75 * PAGE, 130 * PAGE + 5, 101 * PAGE
    groups = [(90, 8), (150, 12), (16, 6)]
    c = Case(groups, own, heads, kv_heads, D, sinks=sinks, seed=seed, poison=False)
    c.row_pages = [p for n, p in groups for _ in range(n)]
    return c


class Run:
    def __init__(self, c):
        self.b, self.c = binding(), c
        up = lambda t: None if t is None else t.cuda()
        self.t = [up(t) for t in (c.q, c.k, c.v, c.positions, c.table, c.start, c.pages, c.k_pool, c.v_pool)]
        self.p = self.b.make_params(c.rows, c.heads, c.kv_heads, c.D, c.width, c.num_pages, BF16, rope_cos=up(c.cos),
                                    rope_sin=up(c.sin), sinks=up(c.sinks))
        self.ws = self.b.new_shared_workspace(self.p, len(c.groups))
        self.out = torch.full_like(self.t[0], 7.0)

    def call(self):
        self.b.decode_shared(self.p, *self.t, self.out, self.ws)


@pytest.mark.parametrize("D,heads,kv_heads,sinks", [(64, 16, 8, True), (128, 8, 4, False), (128, 24, 8, False)])
def test_rows_over_many_runs(D, heads, kv_heads, sinks):
    c = many_runs(D, heads, kv_heads, D + heads, sinks)
    # whatever number of the CTAs takes own pages (most of the work here), some pair covers whole runs of the cursor
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    assert all(whole_short_runs(c, n) > 0 for n in range(ctas // 4, ctas + 1))
    r = Run(c)
    r.call()
    r.b.check_status(r.ws)
    first = r.out.clone()
    for _ in range(8):
        r.out.fill_(0)
        r.call()
        assert torch.equal(r.out.view(torch.int16), first.view(torch.int16))
    r.b.check_status(r.ws)
    c.write()
    for got, want in ((r.t[7], c.k_pool), (r.t[8], c.v_pool)):
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))
    want, bound = c.want()
    err = (first.cpu().double() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())
