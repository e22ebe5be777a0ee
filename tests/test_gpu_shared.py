"""Decode over shared prefixes on the GPU against tests/shared_util.py: keys and values bit for bit, outputs within the
bound derived there."""
import random

import pytest
import torch

from gpu_util import binding
from pages_util import State, pages
from shared_util import BF16, PAGE, Case

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


class Run:
    """A case's tensors on the GPU and the call on them."""

    def __init__(self, c):
        self.b, self.c = binding(), c
        up = lambda t: None if t is None else t.cuda()
        self.q, self.k, self.v, self.pos, self.table = map(up, (c.q, c.k, c.v, c.positions, c.table))
        self.start, self.pages, self.kp, self.vp = map(up, (c.start, c.pages, c.k_pool, c.v_pool))
        self.p = self.b.make_params(c.rows, c.heads, c.kv_heads, c.D, c.width, c.num_pages, BF16, window=c.window,
                                    rope_cos=up(c.cos), rope_sin=up(c.sin), sinks=up(c.sinks))
        self.ws = self.b.new_shared_workspace(self.p, len(c.groups))
        self.out = torch.full_like(self.q, 7.0)

    def call(self, stream=None):
        self.b.decode_shared(self.p, self.q, self.k, self.v, self.pos, self.table, self.start, self.pages, self.kp,
                             self.vp, self.out, self.ws, stream=stream)

    def hold(self, skip=()):
        self.c.write(skip)
        for got, want in ((self.kp, self.c.k_pool), (self.vp, self.c.v_pool)):
            assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))
        want, bound = self.c.want(skip)
        got = self.out.cpu()
        err = (got.double() - want).abs()
        for r in range(self.c.rows):
            if r in skip:
                assert (got[r] == 7).all()
            else:
                assert (err[r] <= bound[r]).all(), (r, float((err[r] / bound[r]).max()))

    def check(self, skip=()):
        self.call()
        self.b.check_status(self.ws)
        assert self.b.last_launch_count() == 3
        self.hold(skip)


CASES = {
    # name: (groups of (rows, shared pages), own lengths, heads, kv heads, D, kwargs)
    "one row": ([(1, 9)], [5], 4, 1, 64, {}),
    "two rows": ([(2, 24)], [1, 64], 8, 1, 128, {}),
    "five samples": ([(5, 7)], [1, 100, 63, 64, 65], 64, 8, 64, dict(sinks=True)),
    "odd pages": ([(6, 7)], [3], 4, 4, 128, {}),
    "full half": ([(32, 6)], [10, 70], 8, 2, 128, {}),
    "half and one": ([(33, 6)], [10, 70], 8, 2, 128, {}),
    "tile and one": ([(65, 6)], [1, 130], 8, 2, 64, dict(sinks=True)),
    "groups of three heads": ([(50, 9)], [20, 200], 6, 2, 64, {}),
    "groups of five heads": ([(30, 8)], [20, 200], 10, 2, 128, {}),
    "seven heads, two tiles": ([(37, 11)], [1, 2, 3], 7, 1, 64, {}),
    "one head": ([(300, 7)], [1, 65], 2, 2, 64, {}),
    "several groups": ([(3, 12), (1, 8), (0, 4), (20, 6), (2, 11), (9, 31), (4, 0), (2, 25)], [1, 63, 64, 65, 300], 8, 2, 64, {}),
    "nothing shared": ([(4, 0), (3, 5), (2, 12)], [10, 100], 8, 8, 64, {}),
    "long prefix, one kv head": ([(3, 333)], [7], 2, 1, 128, {}),
    "long prefix": ([(40, 120)], [7, 90], 8, 2, 64, {}),
    "many kv heads": ([(2, 24)], [9], 48, 48, 64, {}),
    "many groups": ([(2, 24)] * 70, [1, 66], 2, 1, 64, {}),
    "no rotation": ([(7, 10)], [30], 8, 2, 128, dict(theta=0.0)),
    "wide window": ([(7, 10)], [30, 5], 8, 2, 64, dict(window=100000)),
    "window hides": ([(7, 10), (3, 13)], [30, 5, 400], 8, 2, 64, dict(window=500, sinks=True)),
    "window inside own": ([(7, 10)], [300], 8, 2, 128, dict(window=77)),
}


@pytest.mark.parametrize("name", CASES)
def test_decode_shared(name):
    groups, own, heads, kv, D, kw = CASES[name]
    Run(Case(groups, own, heads, kv, D, seed=len(name), **kw)).check()


def test_own_pages_past_one_queue_slot():
    """Rows with more than 64 own pages, whose items are handed over in pieces."""
    Run(Case([(3, 13), (2, 4)], [70 * PAGE + 1, 30, 140 * PAGE], 2, 1, 64, seed=5)).check()


def test_more_rows_and_groups_than_the_planner_holds_at_once():
    rng = random.Random(3)
    groups = [(rng.choice([1, 2, 3]), rng.choice([0, 6, 13, 24])) for _ in range(1300)]
    c = Case(groups, [1, 2, 65], 1, 1, 64, seed=3)
    assert c.rows > 2048 and len(groups) > 1024
    Run(c).check()


@pytest.mark.parametrize("seed", range(6))
def test_drawn(seed):
    rng = random.Random(100 + seed)
    kv = rng.choice([1, 2, 4])
    groups = [(rng.choice([0, 1, 2, 5, 17, 40]), rng.randint(0, 40)) for _ in range(rng.randint(1, 5))] + [(1, 0)]
    own = [rng.randint(1, 400) for _ in range(11)]
    Run(Case(groups, own, kv * rng.choice([1, 2, 3, 4, 6, 8]), kv, rng.choice([64, 128]), sinks=rng.random() < 0.5,
             window=rng.choice([0, 0, 700]), seed=seed)).check()


def test_large_scores_and_one_key_that_takes_all():
    """Scores that grow along the prefix raise the running maximum block after block; the last key wins by far."""
    c = Case([(20, 12)], [3], 4, 2, 64, seed=2, theta=0.0)
    ramp = torch.linspace(0.5, 12.0, 12 * PAGE)
    for i, x in enumerate(c.table[0, :12].tolist()):
        c.k_pool[x] = (c.k_pool[x].float() * ramp[i * PAGE:(i + 1) * PAGE, None]).to(BF16)
    Run(c).check()


def test_infinite_and_undefined_values_reach_only_those_that_see_them():
    c = Case([(5, 7), (4, 9)], [10, 70], 8, 2, 64, seed=9)
    x = int(c.table[0, 2])
    c.v_pool[x, 1, 5, 7] = float("nan")            # seen by group 0, kv head 1
    r = Run(c)
    r.call()
    r.b.check_status(r.ws)
    bad = ~torch.isfinite(r.out.cpu())
    want = torch.zeros_like(bad)
    want[:5, 4:, 7] = True
    assert torch.equal(bad, want)


def test_the_same_call_gives_the_same_bits():
    c = Case([(30, 30), (7, 9)], [1, 64, 500], 8, 2, 128, seed=4)
    r = Run(c)
    r.call()
    first = r.out.clone()
    for _ in range(5):
        r.out.fill_(0)
        r.call()
        assert torch.equal(r.out.view(torch.int16), first.view(torch.int16))
    r.b.check_status(r.ws)


def test_rows_that_are_skipped():
    """Positions outside the table, negative, or inside the shared pages: those rows are skipped and write nothing."""
    c = Case([(6, 7), (3, 12)], [40, 2], 8, 2, 64, seed=6)
    c.positions[1], c.positions[3], c.positions[7] = -1, c.width * PAGE, 12 * PAGE - 1
    skip = (1, 3, 7)
    r = Run(c)
    r.call()
    with pytest.raises(r.b.PdattnError) as e:
        r.b.check_status(r.ws)
    assert e.value.status == r.b.EBADPOS
    r.hold(skip)
    c2 = Case([(6, 7), (3, 12)], [40, 2], 8, 2, 64, seed=7)       # the workspace stays usable
    r2 = Run(c2)
    r2.ws = r.ws
    r2.check()


@pytest.mark.parametrize("case", ["first", "last", "falls", "negative pages", "negative start", "past"])
def test_groups_that_are_no_partition(case):
    c = Case([(3, 12), (2, 25), (4, 8)], [10], 8, 2, 64, seed=8)
    r = Run(c)
    if case == "first":
        r.start[0] = 1
    elif case == "last":
        r.start[3] = 8
    elif case == "falls":
        r.start[1], r.start[2] = 5, 3
    elif case == "negative pages":
        r.pages[1] = -1
    elif case == "negative start":
        r.start[1] = -3
    else:
        r.start[3] = 1 << 30
    r.call()
    with pytest.raises(r.b.PdattnError) as e:
        r.b.check_status(r.ws)
    assert e.value.status == r.b.EBADPOS and (r.out == 7).all()


def test_shared_pages_past_the_table():
    c = Case([(3, 12), (2, 25)], [10], 8, 2, 64, seed=8)
    r = Run(c)
    r.pages[1] = 1 << 30
    r.call()
    with pytest.raises(r.b.PdattnError) as e:
        r.b.check_status(r.ws)
    assert e.value.status == r.b.EBADPOS
    r.hold(skip=(3, 4))


@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_bad_shared_page(bad):
    c = Case([(3, 13), (2, 25)], [10], 8, 2, 64, seed=8)
    r = Run(c)
    r.table[:3, 2] = bad
    r.call()
    with pytest.raises(r.b.PdattnError) as e:
        r.b.check_status(r.ws)
    assert e.value.status == r.b.EBADPAGE
    # the other group's rows are right
    c.write()
    want, bound = c.want()
    assert ((r.out.cpu().double() - want).abs() <= bound)[3:].all()


def test_in_graphs_that_share_a_workspace_with_groups_that_change():
    c = [Case([(6, 8), (5, 7)], [30, 100], 8, 2, 64, seed=1), Case([(3, 13), (8, 6)], [77, 3], 8, 2, 64, seed=2)]
    c[1].width = c[0].width = max(x.width for x in c)
    for x in c:
        pad = torch.full((x.rows, x.width - x.table.shape[1]), -1, dtype=torch.int32)
        x.table = torch.cat([x.table, pad], 1)
    runs = [Run(x) for x in c]
    ws = max((r.ws for r in runs), key=lambda t: t.numel())
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(stream):
        for r in runs:
            r.ws = ws
            r.call()
        stream.synchronize()
        for r in runs:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=stream):
                r.call()
        for r, x in zip(runs, c):
            r.kp.copy_(x.k_pool), r.vp.copy_(x.v_pool), r.out.fill_(7.0)
        for i in (0, 1, 1, 0):
            graphs[i].replay()
            runs[i].b.check_status(ws, stream)
        for r in runs:
            r.hold()
        # the same rows, grouped otherwise, through the first graph: only its device arrays change
        runs[0].start.copy_(torch.tensor([0, 6, 11], dtype=torch.int32))
        runs[0].pages.copy_(torch.tensor([7, 0], dtype=torch.int32))
        runs[0].out.fill_(7.0)
        graphs[0].replay()
        runs[0].b.check_status(ws, stream)
        runs[0].hold()
    torch.cuda.current_stream().wait_stream(stream)


def test_two_calls_at_once_on_two_streams():
    runs = [Run(Case([(20, 20), (3, 14)], [30, 100], 8, 2, 128, seed=s)) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(3):
        for r, s in zip(runs, streams):
            with torch.cuda.stream(s):
                r.call()
    for r, s in zip(runs, streams):
        r.b.check_status(r.ws, s)
        r.hold()


def test_no_other_call_runs_its_plan():
    c = Case([(6, 8)], [30], 8, 2, 64, seed=1)
    r = Run(c)
    r.check()
    big = torch.zeros(max(r.ws.numel(), r.b.workspace_size(r.p)), dtype=torch.uint8, device="cuda")
    r.ws = big
    r.call()
    r.b.attend(r.p, r.q, r.pos, r.table, r.kp, r.vp, torch.empty_like(r.out), big)
    with pytest.raises(r.b.PdattnError) as e:
        r.b.check_status(big)
    assert e.value.status == r.b.EINVAL
    r.call()                                       # and the other way round
    r.b.check_status(big)
    r.hold()


def test_a_wait_that_runs_out_is_reported():
    """The test hook of the decode kernel: its first stage is never filled, the bounded waits run out and the call
    reports it; the next call on the workspace is right."""
    c = Case([(6, 8)], [30], 8, 2, 64, seed=1)
    r = Run(c)
    r.ws[52] = 1
    r.call()
    with pytest.raises(r.b.PdattnError) as e:
        r.b.check_status(r.ws)
    assert e.value.status == r.b.ETIMEOUT
    r.ws[52] = 0
    r.kp.copy_(c.k_pool), r.vp.copy_(c.v_pool), r.out.fill_(7.0)
    r.check()


def test_f32_is_refused():
    b = binding()
    p = b.make_params(2, 4, 4, 64, 8, 16, torch.float32)
    with pytest.raises(b.PdattnError):
        b.new_shared_workspace(p, 1)


def test_samples_of_one_prompt_step_by_step():
    """The operators as they are used together: a prompt's pages are forked to several samples, whose tables grow and
    whose tails are copied on the way; queries and keys are rotated with frequencies scaled for a long context; each
    step attends the shared pages once.  Every step against decode_fused over the same tables, and at the end the
    samples' caches are compacted and a last step gives the same output."""
    b = binding()
    heads, kv, D, rows, width, N = 8, 2, 64, 6, 12, 60
    gen = torch.Generator(device="cuda").manual_seed(3)
    rot = b.make_rotary(D, 10000.0, rot_dim=32, interleaved=True, scaling="ramp", factor=4.0, low=1.0, high=32.0,
                        original_len=256)
    p = b.make_params(rows, heads, kv, D, width, N, BF16)
    kp, vp = (torch.randn(N, kv, PAGE, D, generator=gen, device="cuda").to(BF16) for _ in range(2))
    s = State(rows, width, N, [7 * PAGE + 20] + [0] * (rows - 1), seed=1)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table, lengths, refs = ints(s.table), ints(s.lengths), ints(s.refs)
    cache, pws, rws = b.make_pages(p, [kp, vp]), b.new_pages_workspace(p), b.new_status()
    sws, dws = b.new_shared_workspace(p, 2), b.new_workspace(p)
    parents = ints([0] * rows)
    start, count = ints([0, rows, rows]), ints([7, 0])
    for step in range(50):
        if step == 30:
            parents = ints([2, 2, 2, 4, 4, 5])       # beams continue one another
        new = lengths[parents.long()] + 1
        b.pages_update(p, cache, table, lengths, refs, parents, new, pws)
        b.check_status(pws)
        lengths, parents = new, ints(range(rows))
        positions = lengths - 1
        q, k, v = (torch.randn(rows, h, D, generator=gen, device="cuda").to(BF16) for h in (heads, kv, kv))
        qr, kr = torch.empty_like(q), torch.empty_like(k)
        b.rotary_apply(rot, q, k, positions, qr, kr, rws)
        outs = [torch.empty_like(q) for _ in range(2)]
        b.decode_shared(p, qr, kr, v, positions, table, start, count, kp, vp, outs[0], sws)
        b.decode_fused(p, qr, kr, v, positions, table, kp, vp, outs[1], dws)
        for ws in (rws, sws, dws):
            b.check_status(ws)
        # both are within 2^-7 of sum w |v| (below 4) and a rounding of what they stand for
        assert (outs[0].float() - outs[1].float()).abs().max() <= 4 * 2.0 ** -6
        assert torch.isfinite(outs[0].float()).all()
    held = sum(int(x) > 0 for x in refs)
    page_map = torch.empty_like(refs)
    b.pages_compact(p, cache, table, lengths, refs, page_map, pws)
    b.check_status(pws)
    assert int((refs > 0).sum()) == held and int(table.max()) < held
    again = torch.empty_like(q)
    b.decode_shared(p, qr, kr, v, positions, table, start, count, kp, vp, again, sws)
    b.check_status(sws)
    assert torch.equal(again, outs[0])


def test_calls_that_follow_one_another_on_a_stream():
    """Each call's launches start while those before them end: inputs that the work just before writes (positions, the
    table, pages, groups, queries) are read only afterwards, and a step's outputs are whole for what comes next."""
    c = Case([(20, 20), (9, 12)], [1, 64, 130], 8, 2, 64, seed=11)
    r = Run(c)
    clean = [t.clone() for t in (r.q, r.k, r.v, r.pos, r.table, r.start, r.pages, r.kp, r.vp)]
    mine = (r.q, r.k, r.v, r.pos, r.table, r.start, r.pages, r.kp, r.vp)
    rot, rws = r.b.make_rotary(64, 1e4), r.b.new_status()
    big = torch.zeros(200000, 8, 64, device="cuda", dtype=BF16)
    at = torch.zeros(200000, dtype=torch.int32, device="cuda")
    outs = []
    for i in range(6):
        for t in mine:
            t.zero_()
        if i % 2:
            r.b.rotary_apply(rot, big, None, at, big, None, rws)      # a long kernel just before
        for t, good in zip(mine, clean):
            t.copy_(good)
        r.call()
        outs.append(r.out.clone())
        r.out.fill_(7.0)
    r.b.check_status(r.ws)
    assert all(torch.equal(o.view(torch.int16), outs[0].view(torch.int16)) for o in outs)
    r.out.copy_(outs[0])
    r.hold()
