"""Page bookkeeping on the GPU against tests/pages_util.py: tables, counts and pools have to be equal, bit for bit."""
import random

import pytest
import torch

from gpu_util import binding
from pages_util import PAGE, State, pages

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF16, F32, INT8 = torch.bfloat16, torch.float32, torch.int8


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Cache:
    """A state on the GPU, with pools of several types and head counts."""

    def __init__(self, state, kinds=((BF16, 2, 64), (F32, 0, 1)), seed=0):
        self.b, self.s = binding(), state
        rows = len(state.table)
        self.p = self.b.make_params(rows, 8, 8, 64, state.width, state.num_pages, BF16)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.pools = []
        for dtype, dim, heads in kinds:
            shape = (state.num_pages, heads, PAGE) + ((dim,) if dim else ())
            self.pools.append(torch.randint(-100, 100, shape, generator=g, device="cuda").to(dtype))
        self.before = [t.clone() for t in self.pools]
        self.pages = self.b.make_pages(self.p, self.pools)
        self.ws = self.b.new_pages_workspace(self.p)
        self.load()

    def load(self):
        s = self.s
        self.table, self.lengths, self.refs = ints(s.table).view(len(s.table), s.width), ints(s.lengths), ints(s.refs)

    def update(self, parents, new, **kw):
        self.b.pages_update(self.p, self.pages, self.table, self.lengths, self.refs, ints(parents), ints(new), self.ws, **kw)

    def compact(self, page_map, **kw):
        self.b.pages_compact(self.p, self.pages, self.table, self.lengths, self.refs, page_map, self.ws, **kw)

    def check(self):
        self.b.check_status(self.ws)

    def want_pools(self, copies):
        want = [t.clone() for t in self.before]
        for src, dst, n in copies:
            for t, old in zip(want, self.before):
                t[dst, :, :n] = old[src, :, :n]
        return want

    def same(self, table, refs, copies):
        assert torch.equal(self.table, ints(table)) and torch.equal(self.refs, ints(refs))
        for got, want in zip(self.pools, self.want_pools(copies)):
            assert torch.equal(got, want)


KINDS = ((BF16, 2, 64), (F32, 0, 3))     # (type, dimensions (0: a scale), heads)
ALL = ((BF16, 128, 2), (F32, 64, 3), (INT8, 64, 5), (F32, 0, 5), (INT8, 3, 1))


def drawn(seed, rows, hi, grow, share):
    rng = random.Random(seed)
    lengths = [rng.choice([0, 1, PAGE - 1, PAGE, PAGE + 1, rng.randint(0, hi)]) for _ in range(rows)]
    if share > 1:
        lengths = [lengths[r - r % share] for r in range(rows)]
    parents, new = [], []
    for r in range(rows):
        kind = rng.randrange(6)
        p = r if kind < 2 else rng.randrange(rows) if kind < 5 else -1
        held = lengths[p] if p >= 0 else 0
        parents.append(p)
        new.append(rng.choice([held, held + rng.randint(0, grow), rng.randint(0, held), held + 1]))
    return lengths, parents, new


@pytest.mark.parametrize("seed,rows,hi,grow,share", [(1, 1, 50, 3, 1), (2, 2, 200, 100, 1), (3, 7, 300, 1, 1),
                                                     (4, 33, 500, 200, 3), (5, 64, 130, 64, 64), (6, 150, 900, 5, 5),
                                                     (7, 40, 64, 1, 4), (8, 1100, 90, 30, 1), (9, 2500, 130, 2, 10),
                                                     (10, 900, 3000, 40, 2), (11, 3000, 800, 9, 3)])
def test_update(seed, rows, hi, grow, share):
    lengths, parents, new = drawn(seed, rows, hi, grow, share)
    width = max(pages(n) for n in lengths + new) + 1
    need = sum(pages(n) for n in lengths) + sum(pages(n) for n in new) + 5
    s = State(rows, width, need, lengths, seed, share, pins=(0, 0, need - 1))
    c = Cache(s, KINDS if rows > 200 else ALL)
    table, refs, copies = s.update(parents, new)
    c.update(parents, new)
    c.check()
    c.same(table, refs, copies)


@pytest.mark.parametrize("inplace", [False, True])
def test_update_uses_the_pages_it_frees_and_needs_no_more(inplace):
    # three rows hold every page; two are freed and the third grows into all that is left
    for extra, ok in ((0, True), (1, False)):
        s2 = State(3, 11, 10, [3 * PAGE, 2 * PAGE + 5, 4 * PAGE - 1])
        c = Cache(s2)
        out = {} if inplace else dict(table_out=torch.full_like(c.table, 5), refs_out=torch.full_like(c.refs, 5))
        before = [t.clone() for t in (c.table, c.refs)]
        parents, want = [0, -1, -1], [10 * PAGE + extra, 0, 0]
        c.update(parents, want, **out)
        if ok:
            c.check()
            table, refs, copies = s2.update(parents, want)
            if not inplace:
                assert all(torch.equal(a, b) for a, b in zip(before, (c.table, c.refs)))
                c.table, c.refs = out["table_out"], out["refs_out"]
            c.same(table, refs, copies)
        else:
            assert s2.update(parents, want) == "no pages"
            with pytest.raises(c.b.PdattnError) as e:
                c.check()
            assert e.value.status == c.b.ENOPAGES
            assert all(torch.equal(a, b) for a, b in zip(before, (c.table, c.refs)))
            assert all((t == 5).all() for t in out.values())
            assert all(torch.equal(a, b) for a, b in zip(c.pools, c.before))
            c.update([0, 1, 2], s2.lengths)      # the workspace stays usable
            c.check()


@pytest.mark.parametrize("case", ["parent high", "parent low", "new negative", "new long", "length negative", "length long",
                                  "page high", "page negative", "few refs", "negative refs"])
def test_update_changes_nothing_on_bad_data(case):
    s = State(4, 5, 24, [70, 130, 64, 300], seed=3)
    c = Cache(s)
    parents, new, status = [0, 1, 1, 3], [71, 131, 140, 300], c.b.EBADPOS
    if case == "parent high":
        parents[2] = 4
    elif case == "parent low":
        parents[2] = -2
    elif case == "new negative":
        new[1] = -1
    elif case == "new long":
        new[3] = 5 * PAGE + 1
    elif case == "length negative":
        c.lengths[2] = -1
    elif case == "length long":
        c.lengths[2] = 5 * PAGE + 1
    elif case.startswith("page"):
        c.table[3, 4] = 24 if case == "page high" else -1
        status = c.b.EBADPAGE
    else:
        c.refs[s.table[1][0] if case == "few refs" else s.free[0]] -= 1
        status = c.b.EBADPAGE
    before = [t.clone() for t in (c.table, c.refs)]
    c.update(parents, new)
    with pytest.raises(c.b.PdattnError) as e:
        c.check()
    assert e.value.status == status
    assert all(torch.equal(a, b) for a, b in zip(before, (c.table, c.refs)))
    assert all(torch.equal(a, b) for a, b in zip(c.pools, c.before))


@pytest.mark.parametrize("parents", [[1, 0, 2], [1, 2, 0], [2, 2, 2], [-1, 0, 0]])
def test_rows_swap_and_fork_in_place(parents):
    s = State(3, 6, 40, [100, 200, 300], seed=5)
    new = [(s.lengths[p] if p >= 0 else 0) + 1 for p in parents]
    c = Cache(s)
    table, refs, copies = s.update(parents, new)
    c.update(parents, new)
    c.check()
    c.same(table, refs, copies)


def test_many_steps_keep_every_count():
    """Forks, growth, truncations and freed rows, one step after another, each against the plain one; at the end every
    row is freed and every page but the pinned one is free."""
    rng = random.Random(11)
    rows, width, N = 20, 12, 300
    s = State(rows, width, N, [rng.randint(0, 300) for _ in range(rows)], seed=1, pins=(N - 1,))
    c = Cache(s)
    for step in range(12):
        parents = [rng.choice([r, r, r, rng.randrange(rows), -1]) for r in range(rows)]
        new = []
        for p in parents:
            held = s.lengths[p] if p >= 0 else 0
            new.append(min(width * PAGE, rng.choice([held, held + 1, held + rng.randint(0, 90), rng.randint(0, held)])))
        if step == 11:
            parents, new = [-1] * rows, [0] * rows
        table, refs, copies = s.update(parents, new)
        c.update(parents, new)
        c.check()
        c.same(table, refs, copies)
        c.before = [t.clone() for t in c.pools]
        s.table, s.refs, s.lengths = table, refs, new
        c.lengths = ints(new)
    assert sum(s.refs) == 1


@pytest.mark.parametrize("seed,rows,hi,share,spare,low", [(1, 1, 10, 1, 0, False), (2, 3, 300, 1, 7, False),
                                                          (3, 9, 200, 3, 0, False), (4, 30, 900, 1, 250, False),
                                                          (5, 5, 400, 1, 40, True), (6, 0, 0, 1, 5, False),
                                                          (7, 1500, 90, 2, 20000, False)])
def test_compact(seed, rows, hi, share, spare, low):
    rng = random.Random(seed)
    lengths = [rng.randint(0, hi) for _ in range(max(rows, 1))]
    lengths = [lengths[r - r % share] for r in range(len(lengths))]
    if rows == 0:
        lengths = [0]       # one row that holds nothing
    need = max(1, sum(pages(n) for n in lengths))
    pins = (need + spare - 1, 0) if spare else ()
    s = State(len(lengths), max(pages(n) for n in lengths) + 2, need + spare, lengths, seed, share, pins, low)
    c = Cache(s, KINDS if rows > 200 else ALL)
    table, refs, to = s.compact()
    page_map = torch.full((s.num_pages,), 99, dtype=torch.int32, device="cuda")
    out = dict(table_out=torch.empty_like(c.table), refs_out=torch.empty_like(c.refs))
    copies = [(x, y, PAGE) for x, y in enumerate(to) if y >= 0 and y != x]
    c.compact(page_map, **out)
    c.check()
    assert torch.equal(page_map, ints(to))
    first = (c.table, c.refs)
    assert torch.equal(c.table, ints(s.table)) and torch.equal(c.refs, ints(s.refs))
    c.table, c.refs = out["table_out"], out["refs_out"]
    c.same(table, refs, copies)
    c.table, c.refs = first
    page_map.fill_(99)
    c.compact(page_map)      # in place; the sources still hold their pages
    c.check()
    assert torch.equal(page_map, ints(to))
    c.same(table, refs, copies)
    n = sum(x > 0 for x in refs)
    assert (c.refs[:n] > 0).all() and (c.refs[n:] == 0).all()


@pytest.mark.parametrize("num_pages", [1, 40, 6000])
@pytest.mark.parametrize("inplace", [False, True])
def test_pages_without_rows(num_pages, inplace):
    # no row, but holders outside the table: counts are passed on, pages still move
    pins = tuple(range(0, num_pages, 3)) + (0,)
    s = State(0, 4, num_pages, [], seed=2, pins=pins)
    c = Cache(s)
    out = {} if inplace else dict(refs_out=torch.full_like(c.refs, 5))
    c.update([], [], **out)
    c.check()
    assert torch.equal(out.get("refs_out", c.refs), ints(s.refs)) and torch.equal(c.refs, ints(s.refs))
    _, refs, to = s.compact()
    page_map = torch.full((num_pages,), 99, dtype=torch.int32, device="cuda")
    c.compact(page_map, **out)
    c.check()
    assert torch.equal(page_map, ints(to)) and torch.equal(out.get("refs_out", c.refs), ints(refs))
    for got, want in zip(c.pools, c.want_pools([(x, y, PAGE) for x, y in enumerate(to) if y >= 0 and y != x])):
        assert torch.equal(got, want)


@pytest.mark.parametrize("case", ["page high", "page free", "negative refs", "length long"])
def test_compact_changes_nothing_on_bad_data(case):
    s = State(4, 6, 30, [70, 130, 64, 300], seed=3)
    c = Cache(s)
    status = c.b.EBADPAGE
    if case == "page high":
        c.table[1, 0] = 30
    elif case == "page free":
        c.table[1, 0] = s.free[0]
    elif case == "negative refs":
        c.refs[s.free[0]] = -1
    else:
        c.lengths[0] = 6 * PAGE + 1
        status = c.b.EBADPOS
    page_map = torch.full((30,), 99, dtype=torch.int32, device="cuda")
    before = [t.clone() for t in (c.table, c.refs)]
    c.compact(page_map)
    with pytest.raises(c.b.PdattnError) as e:
        c.check()
    assert e.value.status == status
    assert all(torch.equal(a, b) for a, b in zip(before, (c.table, c.refs))) and (page_map == 99).all()
    assert all(torch.equal(a, b) for a, b in zip(c.pools, c.before))


def test_more_pools_than_one_launch_takes():
    s = State(3, 4, 16, [100, 30, 129], seed=2)
    c = Cache(s, ((INT8, 16, 1),) * 131)
    parents, new = [0, 0, 2], [101, 120, 130]
    table, refs, copies = s.update(parents, new)
    c.update(parents, new)
    assert c.b.last_launch_count() == 3
    c.check()
    c.same(table, refs, copies)


def test_update_in_a_graph_on_another_stream():
    """A captured growth step: its lengths live in one buffer, so that every replay takes one more position."""
    s = State(5, 4, 32, [60, 63, 64, 1, 0], seed=4)
    c = Cache(s)
    lengths, new, parents = c.lengths, torch.empty_like(c.lengths), ints([0, 1, 2, 3, 3])

    def step():
        torch.add(lengths[parents.long()], 1, out=new)
        c.b.pages_update(c.p, c.pages, c.table, lengths, c.refs, parents, new, c.ws)
        lengths.copy_(new)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        for got, start in zip((c.table, c.lengths, c.refs), (s.table, s.lengths, s.refs)):
            got.copy_(ints(start))
        for t, old in zip(c.pools, c.before):
            t.copy_(old)
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for _ in range(6):
            graph.replay()
            c.b.check_status(c.ws, stream)
            want = [s.lengths[p] + 1 for p in (0, 1, 2, 3, 3)]
            table, refs, copies = s.update([0, 1, 2, 3, 3], want)
            c.same(table, refs, copies)
            c.before = [t.clone() for t in c.pools]
            s.table, s.refs, s.lengths = table, refs, want
    torch.cuda.current_stream().wait_stream(stream)


def test_pages_past_32_bit_offsets():
    """A pool of more than 4 GiB: pages at its far end are copied to its start and back."""
    N, heads, D = 1100, 64, 512      # 8 MiB a page: f32 rows of 2 KiB
    if torch.cuda.mem_get_info()[0] < 3 * N * heads * PAGE * D * 4:
        pytest.skip("not enough memory")
    b = binding()
    pool = torch.empty(N, heads, PAGE, D, dtype=F32, device="cuda")
    p = b.make_params(2, 8, 8, 64, 3, N, BF16)
    for x in (0, 1, N - 2, N - 1):
        pool[x] = torch.randn(heads, PAGE, D, device="cuda")
    far = pool[N - 2:].clone()
    table, lengths = ints([[N - 2, N - 1, -1], [-1, -1, -1]]), ints([100, 0])
    refs = torch.zeros(N, dtype=torch.int32, device="cuda")
    refs[N - 2:] = 1
    pages_, ws = b.make_pages(p, [pool]), b.new_pages_workspace(p)
    b.pages_update(p, pages_, table, lengths, refs, ints([0, 0]), ints([101, 101]), ws)
    b.check_status(ws)
    assert table.tolist() == [[N - 2, N - 1, -1], [N - 2, 0, -1]] and torch.equal(pool[0, :, :36], far[1, :, :36])
    page_map = torch.empty_like(refs)
    b.pages_compact(p, pages_, table, ints([101, 101]), refs, page_map, ws)
    b.check_status(ws)
    assert table.tolist() == [[1, 2, -1], [1, 0, -1]]
    assert torch.equal(pool[1], far[0]) and torch.equal(pool[2], far[1])
