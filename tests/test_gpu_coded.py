"""The coded (8-bit) cache on the GPU against the CPU references of coded_util.py: codes and scales bit for bit,
attention within the bounds derived there."""
import math

import pytest
import torch

import coded_util as cu
from gpu_util import binding

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

E4M3, INT8, BF16, F32 = torch.float8_e4m3fn, torch.int8, torch.bfloat16, torch.float32
EBADPAGE, ETIMEOUT, EBADPOS = 4, 5, 6


def gpu(*ts):
    return [None if t is None else t.cuda() for t in ts]


class Run:
    """A case's tensors on the GPU and the calls on them."""

    def __init__(self, c, **kw):
        self.b, self.c = binding(), c
        self.p = c.params(self.b, **kw)
        self.tensors = c.cache.gpu()
        self.cache = self.b.make_coded_cache(self.p, *self.tensors)
        self.q, self.k, self.v, self.pos, self.rows, self.slots, self.table = gpu(
            c.q, c.k_new, c.v_new, c.positions, c.rows, c.slots, c.table)
        self.ws = self.b.new_coded_workspace(self.p, len(c.q))
        self.out = torch.full_like(self.q, 7.0)

    def decode(self, out=None):
        self.b.coded_decode(self.p, self.cache, self.q, self.k, self.v, self.pos, self.table,
                            self.out if out is None else out, self.ws)
        return self.out

    def prefill(self, out=None):
        self.b.coded_prefill(self.p, self.cache, self.q, self.k, self.v, self.pos, self.rows, self.slots, self.table,
                             self.out if out is None else out, self.ws)
        return self.out

    def check(self, kind, what=""):
        getattr(self, kind)()
        self.b.check_status(self.ws)
        self.c.write()
        self.c.cache.same(self.tensors)
        want, bound = self.c.want(kind)
        return cu.hold(self.out, want, bound, what)


# ---------------------------------------------------------------------------
# write and read
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("dtype,D,kv_heads,n,theta", [(BF16, 128, 8, 1, 1e4), (BF16, 64, 3, 130, 1e4), (F32, 64, 12, 37, 0.0),
                                                      (F32, 128, 1, 65, 5e5), (BF16, 128, 2, 700, 0.0)])
def test_write_gives_the_formulas_codes(kind, dtype, D, kv_heads, n, theta):
    r = Run(cu.Case(kv_heads, kv_heads, D, [3, 60], [n // 2, n - n // 2], dtype, kind, theta, seed=n))
    r.b.coded_write(r.p, r.cache, r.k, r.v, r.pos, r.slots, r.ws)
    assert r.b.last_launch_count() == 1
    r.b.check_status(r.ws)
    r.c.write()
    r.c.cache.same(r.tensors)           # the new slots and every other one


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_write_at_the_ends_of_the_range(kind, dtype):
    g = torch.Generator().manual_seed(3)
    n, D = 64, 64
    c = cu.Case(1, 1, D, [0], [n], dtype, kind, theta=0.0, seed=5)
    x = torch.randn(n, 1, D, generator=g)
    scales = [0.0, 2.0 ** -149, 2.0 ** -133, 2.0 ** -126, 2.0 ** -120, 2.0 ** -61, 2.0 ** -59, 1e-30, 1.0, 448.0, 127.0, 7.0,
              3.0, 2.0 ** 59, 2.0 ** 61, 1e30, 1e38]
    for i, s in enumerate(scales):
        x[i] = x[i].clamp(-3, 3) * s
    x[20], x[21, 0, 5], x[22, 0, 7], x[23, 0, 9] = 0.0, math.inf, -math.inf, math.nan
    # ties: multiples of half a step of the scale
    x[24, 0], x[24, 0, 0] = torch.arange(D) * 0.5, 127.0
    x[25, 0], x[25, 0, 0] = torch.arange(D) * 0.5 + 16.0, 448.0
    x[26, 0], x[26, 0, 0] = torch.arange(D) * 2.0 ** -11, 448.0
    c.k_new, c.v_new = x.to(dtype), x.flip(0).contiguous().to(dtype)
    r = Run(c)
    r.b.coded_write(r.p, r.cache, r.k, r.v, r.pos, r.slots, r.ws)
    r.b.check_status(r.ws)
    c.write()
    for mine, theirs in zip((c.cache.k, c.cache.v), r.tensors[:2]):
        assert torch.equal(mine, theirs.cpu().view(torch.uint8))
    for mine, theirs in zip((c.cache.ks, c.cache.vs), r.tensors[2:]):
        assert torch.equal(torch.nan_to_num(mine, 5.0), torch.nan_to_num(theirs.cpu(), 5.0))


@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_write_divides_as_the_formula_does_at_every_exponent(kind):
    g = torch.Generator().manual_seed(11)
    n, D = 2048, 64
    c = cu.Case(8, 8, D, [0], [n], F32, kind, theta=0.0, seed=6)
    # every mantissa bit random; a vector's exponents lie within 2^6, the vectors' anywhere an f32 has one
    low = torch.randint(1, 248, (n, 8, 1), generator=g, dtype=torch.int32)
    low[:, 0] = torch.randint(60, 74, (n, 1), generator=g, dtype=torch.int32)       # about 2^-60
    low[:, 1] = torch.randint(180, 194, (n, 1), generator=g, dtype=torch.int32)     # about 2^60
    exps = low + torch.randint(0, 7, (n, 8, D), generator=g, dtype=torch.int32)
    bits = (exps << 23) | torch.randint(0, 2 ** 23, (n, 8, D), generator=g, dtype=torch.int32)
    sign = torch.randint(0, 2, (n, 8, D), generator=g, dtype=torch.int32) << 31
    x = (bits | sign).view(torch.float32)
    c.k_new, c.v_new = x, x.flip(0).contiguous()
    r = Run(c)
    r.b.coded_write(r.p, r.cache, r.k, r.v, r.pos, r.slots, r.ws)
    r.b.check_status(r.ws)
    c.write()
    c.cache.same(r.tensors)


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("dtype,D,kv_heads,n", [(BF16, 128, 8, 1), (BF16, 64, 5, 333), (F32, 128, 2, 66), (F32, 64, 1, 31)])
def test_read_gives_what_the_codes_stand_for(kind, dtype, D, kv_heads, n):
    g = torch.Generator().manual_seed(n)
    r = Run(cu.Case(kv_heads, kv_heads, D, [400], [1], dtype, kind))
    slots = torch.randint(0, r.c.pages * 64, (n,), generator=g).to(torch.int32)   # some of them more than once
    k, v = (torch.empty(n, kv_heads, D, dtype=dtype, device="cuda") for _ in range(2))
    r.b.coded_read(r.p, r.cache, slots.cuda(), k, v, r.ws)
    r.b.check_status(r.ws)
    cache = r.c.cache
    for got, codes, scales in ((k, cache.k, cache.ks), (v, cache.v, cache.vs)):
        assert torch.equal(got.cpu(), cache.meant(codes, scales, slots, torch.float32).to(dtype))


def test_bad_slots_and_positions_are_skipped_and_reported():
    c = cu.Case(4, 2, 64, [0], [6], theta=1e4)
    r = Run(c)
    bad = c.slots.clone()
    bad[1], bad[4] = -1, c.pages * 64
    r.b.coded_write(r.p, r.cache, r.k, r.v, r.pos, bad.cuda(), r.ws)
    with pytest.raises(r.b.PdattnError) as e:
        r.b.check_status(r.ws)
    assert e.value.status == EBADPAGE
    r.b.check_status(r.ws)                       # cleared
    keep = torch.tensor([0, 2, 3, 5])
    c.cache.write(cu.rope(c.k_new.float(), c.cos, c.sin, c.positions)[keep], c.v_new.float()[keep], c.slots[keep])
    c.cache.same(r.tensors)
    pos = c.positions.clone()
    pos[2], pos[3] = -5, c.width * 64            # past the rope table
    r.b.coded_write(r.p, r.cache, r.k, r.v, pos.cuda(), r.slots, r.ws)
    with pytest.raises(r.b.PdattnError) as e:
        r.b.check_status(r.ws)
    assert e.value.status == EBADPOS
    k, v = (torch.full((6, 2, 64), 9.0, dtype=BF16, device="cuda") for _ in range(2))
    r.b.coded_read(r.p, r.cache, bad.cuda(), k, v, r.ws)
    with pytest.raises(r.b.PdattnError) as e:
        r.b.check_status(r.ws)
    assert e.value.status == EBADPAGE
    assert (k[[1, 4]] == 9).all() and (v[[1, 4]] == 9).all() and not (k[[0, 2, 3, 5]] == 9).all()


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,kind", [(BF16, E4M3), (BF16, INT8), (F32, E4M3), (F32, INT8)])
@pytest.mark.parametrize("heads,kv_heads,D", [(8, 8, 64), (8, 2, 128), (24, 3, 64), (5, 1, 128)])
def test_decode(dtype, kind, heads, kv_heads, D):
    ctx = [1, 2, 63, 64, 65, 127, 128, 129, 300, 700]
    r = Run(cu.Case(heads, kv_heads, D, [c - 1 for c in ctx], [1] * len(ctx), dtype, kind, seed=heads))
    r.check("decode")
    assert r.b.last_launch_count() == 2


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [1, 2, 64, 100, 5000])
def test_decode_windows_and_sinks(dtype, window):
    ctx = [1, 64, 65, 130, 513]
    Run(cu.Case(16, 2, 64, [c - 1 for c in ctx], [1] * len(ctx), dtype, INT8, 1.5e5, window, sinks=True)).check("decode")


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("heads,kv_heads,D", [(4, 4, 64), (6, 3, 128), (6, 2, 64), (8, 2, 64), (10, 2, 128)])
def test_f32_decode_of_small_groups(kind, heads, kv_heads, D):
    # groups of up to four heads hold both f16 parts of a head in one tile, larger ones take two passes
    ctx = [1, 17, 64, 129, 2500]
    Run(cu.Case(heads, kv_heads, D, [c - 1 for c in ctx], [1] * len(ctx), F32, kind, 1e4, 700, sinks=True)).check("decode")


@pytest.mark.parametrize("dtype,D,rows,ctx", [(BF16, 128, 1, 9000), (F32, 64, 1, 5001), (BF16, 64, 3, 4133)])
def test_decode_of_long_rows_shared_by_many_ctas(dtype, D, rows, ctx):
    Run(cu.Case(2, 1, D, [ctx - 1 - 7 * i for i in range(rows)], [1] * rows, dtype, E4M3, 0.0)).check("decode")


def test_decode_of_more_rows_than_a_block_holds():
    ctx = [1 + (37 * i) % 90 for i in range(700)]
    Run(cu.Case(2, 2, 64, [c - 1 for c in ctx], [1] * len(ctx), BF16, INT8)).check("decode")


def test_decode_scales_that_differ_by_powers():
    # keys and values of very different sizes, token by token
    c = cu.Case(4, 1, 128, [500], [1], F32, INT8, 0.0)
    g = torch.Generator().manual_seed(8)
    c.cache.ks *= 2.0 ** torch.randint(-6, 3, c.cache.ks.shape, generator=g)
    c.cache.vs *= 2.0 ** torch.randint(-12, 12, c.cache.vs.shape, generator=g)
    Run(c).check("decode")


# ---------------------------------------------------------------------------
# prefill
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("heads,kv_heads,D,prefix,chunk", [
    (8, 2, 128, [0], [1]),                                    # one token, one page
    (8, 2, 128, [0, 5, 64, 500], [3, 1, 64, 8]),              # drafted tokens: halves alternate
    (4, 4, 64, [0, 10], [129, 260]),                          # one head a group: tiles of 256
    (8, 1, 64, [0, 63, 65, 200], [33, 32, 17, 90]),           # groups of 8: tiles of 32
    (6, 2, 128, [100], [200]),                                # groups of 3: rows of the MMA left over
    (10, 2, 64, [0, 1], [52, 51]),                            # groups of 5
    (2, 2, 128, [3000], [2]),                                 # split along the keys
])
def test_prefill(kind, heads, kv_heads, D, prefix, chunk):
    r = Run(cu.Case(heads, kv_heads, D, prefix, chunk, kind=kind, seed=D))
    r.check("prefill")
    assert r.b.last_launch_count() in (3, 4)


@pytest.mark.parametrize("window", [1, 7, 64, 128, 1000])
def test_prefill_windows_and_sinks(window):
    Run(cu.Case(16, 2, 64, [0, 77, 400], [150, 3, 70], kind=INT8, window=window, sinks=True)).check("prefill")


@pytest.mark.parametrize("order", ["mixed", "reverse"])
def test_prefill_of_tokens_in_any_order(order):
    Run(cu.Case(4, 1, 128, [0, 30], [70, 40], order=order)).check("prefill")


def test_prefill_with_more_tiles_than_are_split():
    # enough tiles that none is split: three launches
    r = Run(cu.Case(64, 64, 64, [0, 40], [600, 900], kind=E4M3))
    r.check("prefill")
    assert r.b.last_launch_count() == 3


@pytest.mark.parametrize("rows,chunk", [(1100, 1), (1, 4200)])
def test_prefill_plans_of_many_tiles_and_many_tokens(rows, chunk):
    # more tiles, and more tokens, than the one-pass planner holds, in calls small enough to be split
    r = Run(cu.Case(1, 1, 64, [(5 * i) % 140 for i in range(rows)], [chunk] * rows, kind=INT8, theta=0.0))
    r.check("prefill")
    assert r.b.last_launch_count() == 4


def test_scale_and_chunk_pages():
    c = cu.Case(8, 2, 64, [300, 9], [1, 1])
    r = Run(c, scale=0.05, chunk_pages=3)        # decode takes any chunk_pages and does not use it
    r.decode()
    r.b.check_status(r.ws)
    c.write()
    want, bound = cu.attend(c.cache, cu.rope(c.q.float(), c.cos, c.sin, c.positions), c.positions, c.rows, c.table,
                            scale=0.05)
    cu.hold(r.out, want, bound)


def test_an_uncoded_plan_does_not_outlive_a_coded_step():
    r = Run(cu.Case(8, 2, 128, [130, 20], [1, 1]))
    b = r.b
    ws = torch.zeros(max(b.workspace_size(r.p), b.coded_workspace_size(r.p)), dtype=torch.uint8, device="cuda")
    b.plan(r.p, r.pos, ws)
    r.ws = ws
    r.decode()
    pools = [torch.zeros(r.c.pages, 2, 64, 128, dtype=BF16, device="cuda") for _ in range(2)]
    b.attend(r.p, r.q, r.pos, r.table, *pools, torch.empty_like(r.q), ws)
    with pytest.raises(b.PdattnError) as e:
        b.check_status(ws)
    assert e.value.status == b.EINVAL


@pytest.mark.parametrize("prefix,chunk", [([900, 30], [5, 3]), ([0] * 40, [300] * 40)])   # split tiles, and none
def test_a_coded_prefills_tiles_serve_no_other_call(prefix, chunk):
    c = cu.Case(8, 2, 64, prefix, chunk, BF16, E4M3, seed=8)
    r = Run(c)
    k_pool, v_pool = (torch.zeros(c.pages, 2, 64, 64, dtype=BF16, device="cuda") for _ in range(2))
    r.check("prefill")
    before = r.out.clone()
    r.b.prefill_attend(r.p, r.pos, r.table, k_pool, v_pool, r.out, r.ws)
    torch.cuda.synchronize()
    assert torch.equal(r.out, before)
    r.b.check_status(r.ws)
    r.check("prefill")


def test_prefill_writes_outputs_aligned_to_16_bytes_only():
    c = cu.Case(8, 2, 128, [0, 90], [70, 5])
    r = Run(c)
    wide = torch.zeros(c.q.numel() + 8, dtype=BF16, device="cuda")
    out = wide[8:].view(c.q.shape)
    assert out.data_ptr() % 32 == 16
    r.prefill(out)
    r.prefill()
    r.b.check_status(r.ws)
    assert torch.equal(out, r.out) and (wide[:8] == 0).all()


def test_prefill_scales_that_differ_by_powers():
    c = cu.Case(4, 1, 128, [300], [40], BF16, INT8, 0.0)
    g = torch.Generator().manual_seed(9)
    c.cache.ks *= 2.0 ** torch.randint(-6, 3, c.cache.ks.shape, generator=g)
    c.cache.vs *= 2.0 ** torch.randint(-6, 7, c.cache.vs.shape, generator=g)
    Run(c).check("prefill")


# ---------------------------------------------------------------------------
# what must not show in an output
# ---------------------------------------------------------------------------
def _poison(c, r):
    """NaN scales and e4m3 NaN codes in every slot that no token may see."""
    seen = torch.zeros(c.pages * 64, dtype=torch.bool)
    for row in range(c.n_rows):
        mine = c.positions[c.rows == row]
        if len(mine) == 0:
            continue
        lo = max(0, int(mine.min()) - c.window + 1) if c.window > 0 else 0
        t = torch.arange(lo, int(mine.max()) + 1)
        seen[c.table[row].long()[t // 64] * 64 + t % 64] = True
    hide = ~seen.view(c.pages, 64)
    page, off = hide.nonzero(as_tuple=True)
    for codes, scales in ((r.tensors[0], r.tensors[2]), (r.tensors[1], r.tensors[3])):
        codes.view(torch.uint8)[page, :, off] = 0x7f
        scales[page, :, off] = math.nan


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("window", [0, 50])
def test_unseen_slots_never_reach_an_output(kind, window):
    chunk = [1, 1, 1] if kind == "decode" else [20, 3, 90]
    clean, dirty = (Run(cu.Case(8, 2, 128, [5, 64, 200], chunk, window=window)) for _ in range(2))
    _poison(dirty.c, dirty)
    getattr(clean, kind)()
    getattr(dirty, kind)()
    dirty.b.check_status(dirty.ws)
    assert torch.isfinite(dirty.out).all()
    assert torch.equal(clean.out, dirty.out)


@pytest.mark.parametrize("which", ["k_new", "v_new"])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_a_non_finite_token_reaches_only_who_sees_it(which, value):
    # decode: row 1's own new token
    c = cu.Case(8, 2, 128, [70, 70, 70], [1, 1, 1])
    getattr(c, which)[1, 0, 17] = value
    r = Run(c)
    r.decode()
    r.b.check_status(r.ws)
    out = r.out.cpu()
    assert torch.isnan(out[1, :4]).all() and torch.isfinite(out[[0, 2]]).all() and torch.isfinite(out[1, 4:]).all()
    # prefill: token 9 of 30, whose kv head 1 is poisoned, in the same tile as its elders
    c = cu.Case(8, 2, 128, [70], [30])
    getattr(c, which)[9, 1, 3] = value
    r = Run(c)
    r.prefill()
    r.b.check_status(r.ws)
    out = r.out.cpu()
    assert torch.isfinite(out[:, :4]).all() and torch.isfinite(out[:9]).all() and torch.isnan(out[9:, 4:]).all()


def test_rows_with_bad_positions_or_pages_are_reported_and_the_others_right():
    c = cu.Case(8, 2, 128, [100, 5, 70, 200], [1, 1, 1, 1])
    r = Run(c)
    r.pos[1] = -1
    r.decode()
    with pytest.raises(r.b.PdattnError) as e:
        r.b.check_status(r.ws)
    assert e.value.status == EBADPOS
    assert (r.out[1] == 7).all()                         # left as it was
    keep = torch.tensor([0, 2, 3])
    c.cache.write(cu.rope(c.k_new.float(), c.cos, c.sin, c.positions)[keep], c.v_new.float()[keep], c.slots[keep])
    c.cache.same(r.tensors)
    want, bound = c.want("decode")
    cu.hold(r.out[keep.cuda()], want[keep], bound[keep])
    r.pos[1] = 5
    r.table[2, 0] = c.pages                               # an earlier page of row 2
    r.decode()
    with pytest.raises(r.b.PdattnError) as e:
        r.b.check_status(r.ws)
    assert e.value.status == EBADPAGE
    c.write()
    want, bound = c.want("decode")
    for row in (0, 1, 3):
        cu.hold(r.out[row], want[row], bound[row], f"row {row}")
    # prefill: a row index outside the table, and nothing is written to out
    c = cu.Case(8, 2, 128, [0], [5])
    r = Run(c)
    r.rows[3] = 1
    r.prefill()
    with pytest.raises(r.b.PdattnError) as e:
        r.b.check_status(r.ws)
    assert e.value.status == EBADPOS and (r.out == 7).all()


# ---------------------------------------------------------------------------
# a run of them, graphs, streams, workspaces
# ---------------------------------------------------------------------------
def test_prompt_then_steps_then_read_back():
    """A prompt in two chunks, six decode steps and the cache read back, on one workspace."""
    b = binding()
    heads, kv_heads, D, kind, lens = 8, 2, 128, E4M3, [150, 61]
    c = cu.Case(heads, kv_heads, D, [0, 0], [n + 6 for n in lens], kind=kind, seed=3)
    c.cache = cu.Cache(c.pages, kv_heads, D, kind)
    p = c.params(b)
    cache = b.new_coded_cache(p, kind)
    ws = b.new_coded_workspace(p, len(c.q))
    table = c.table.cuda()
    first = [40, 61]
    cut = [(c.positions < torch.tensor(first)[c.rows.long()]), None]
    cut[1] = ~cut[0] & (c.positions < torch.tensor(lens)[c.rows.long()])
    parts = [m.nonzero().squeeze(1) for m in cut]
    steps = [torch.tensor([(c.rows == r).nonzero()[n + t].item() for r, n in enumerate(lens)]) for t in range(6)]
    q_rot = cu.rope(c.q.float(), c.cos, c.sin, c.positions)
    k_rot = cu.rope(c.k_new.float(), c.cos, c.sin, c.positions)

    def check(at, out, kind_):
        c.cache.write(k_rot[at], c.v_new.float()[at], c.slots[at])
        want, bound = cu.attend(c.cache, q_rot[at], c.positions[at], c.rows[at], c.table, kind=kind_)
        cu.hold(out, want, bound, kind_)

    for at in parts:
        out = torch.empty_like(c.q[at]).cuda()
        b.coded_prefill(p, cache, *gpu(c.q[at], c.k_new[at], c.v_new[at], c.positions[at], c.rows[at], c.slots[at]),
                        table, out, ws)
        check(at, out, "prefill")
    for at in steps:
        out = torch.empty_like(c.q[at]).cuda()
        b.coded_decode(p, cache, *gpu(c.q[at], c.k_new[at], c.v_new[at], c.positions[at]), table, out, ws)
        check(at, out, "decode")
    b.check_status(ws)
    c.cache.same(cache._tensors)
    k, v = (torch.empty(len(c.q), kv_heads, D, dtype=BF16, device="cuda") for _ in range(2))
    b.coded_read(p, cache, c.slots.cuda(), k, v, ws)
    b.check_status(ws)
    assert torch.equal(k.cpu(), c.cache.meant(c.cache.k, c.cache.ks, c.slots, torch.float32).to(BF16))
    # within half an e4m3 step of the rotated keys, and the bf16 rounding
    err = (k.cpu().float() - k_rot).abs()
    assert (err <= k_rot.abs() * (2.0 ** -4 + 2.0 ** -8) * 1.01 + k_rot.abs().amax(-1, keepdim=True) * 2.0 ** -17).all()


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_calls_are_repeatable(kind):
    """The same call twice gives the same bits: shares and merges have a fixed order."""
    r = Run(cu.Case(8, 2, 128, [700, 2000, 63], [1, 1, 1] if kind == "decode" else [2, 5, 40]))
    getattr(r, kind)()
    first = r.out.clone()
    for _ in range(5):
        r.out.fill_(0)
        getattr(r, kind)()
        assert torch.equal(first, r.out)
    r.b.check_status(r.ws)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_captured_and_replayed_with_new_inputs(kind):
    r = Run(cu.Case(8, 2, 128, [64, 300, 10], [1, 1, 1] if kind == "decode" else [4, 33, 1]))
    getattr(r, kind)()                      # set-up outside the capture
    r.c.write()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        getattr(r, kind)()
    g = torch.Generator().manual_seed(1)
    c = r.c
    for it in range(3):
        c.q = torch.randn(c.q.shape, generator=g).to(BF16)
        c.k_new, c.v_new = (torch.randn(c.k_new.shape, generator=g).to(BF16) for _ in range(2))
        if kind == "decode":                # positions advance inside the rows' last pages
            c.positions = c.positions + 1
            c.slots = (c.table[c.rows.long(), c.positions.long() // 64] * 64 + c.positions % 64).to(torch.int32)
        for dst, src in ((r.q, c.q), (r.k, c.k_new), (r.v, c.v_new), (r.pos, c.positions), (r.slots, c.slots)):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        r.b.check_status(r.ws)
        c.write()
        c.cache.same(r.tensors)
        want, bound = c.want(kind)
        cu.hold(r.out, want, bound, f"replay {it}")


def test_calls_on_another_stream_and_two_at_once():
    runs = [Run(cu.Case(8, 2, 128, [900 + 100 * i], [1], seed=i)) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(3):
        for r, s in zip(runs, streams):
            with torch.cuda.stream(s):
                r.decode()
    for r, s in zip(runs, streams):
        r.b.coded_decode(r.p, r.cache, r.q, r.k, r.v, r.pos, r.table, r.out, r.ws, stream=s)
    torch.cuda.synchronize()
    for r in runs:
        r.b.check_status(r.ws)
        r.c.write()
        r.c.cache.same(r.tensors)
        want, bound = r.c.want("decode")
        cu.hold(r.out, want, bound)


def test_a_workspace_serves_every_call_in_turn():
    """Uncoded and coded calls in turn on one workspace: nothing one leaves there disturbs the next."""
    b = binding()
    c = cu.Case(8, 2, 128, [130, 20, 64], [1, 1, 1])
    pre = cu.Case(8, 2, 128, [130, 20, 64], [20, 1, 3], seed=4)
    r, rp = Run(c), Run(pre)
    size = max(b.workspace_size(r.p), b.coded_workspace_size(r.p, 24), b.prefill_workspace_size(r.p, 24))
    r.ws = rp.ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    pools = [torch.randn(c.pages, 2, 64, 128, device="cuda").to(BF16) for _ in range(2)]
    for _ in range(2):
        b.decode_fused(r.p, r.q, r.k, r.v, r.pos, r.table, *pools, torch.empty_like(r.q), r.ws)
        r.out.fill_(0)
        r.decode()
        rp.prefill()
    b.check_status(r.ws)
    for run, kind in ((r, "decode"), (rp, "prefill")):
        run.c.write()
        want, bound = run.c.want(kind)
        cu.hold(run.out, want, bound, kind)


def test_the_binding_refuses_wrong_tensors():
    r = Run(cu.Case(8, 2, 128, [10], [1]))
    b = r.b
    for bad in (r.q.float(), r.q[:, :4], r.q.cpu(), r.q.transpose(1, 2), torch.cat([r.q, r.q]), None):
        with pytest.raises((ValueError, TypeError)):
            b.coded_decode(r.p, r.cache, bad, r.k, r.v, r.pos, r.table, r.out, r.ws)
    with pytest.raises(ValueError):
        b.coded_decode(r.p, r.cache, r.q, r.k, r.v, r.pos.long(), r.table, r.out, r.ws)
    with pytest.raises(ValueError):
        b.coded_decode(r.p, r.cache, r.q, r.k, r.v, r.pos, r.table[:, :1], r.out, r.ws)
    with pytest.raises(TypeError):
        b.coded_decode(r.p, r.tensors, r.q, r.k, r.v, r.pos, r.table, r.out, r.ws)
    with pytest.raises(b.PdattnError):
        b.coded_decode(r.p, r.cache, r.q, r.k, r.v, r.pos, r.table, r.out, torch.zeros(512, dtype=torch.uint8, device="cuda"))
    other = b.make_params(1, 8, 2, 128, r.c.width, r.c.pages + 1, BF16)
    with pytest.raises(ValueError):
        b.coded_decode(other, r.cache, r.q, r.k, r.v, r.pos, r.table, r.out, r.ws)
    with pytest.raises(ValueError):
        b.make_coded_cache(r.p, r.tensors[0], r.tensors[1], r.tensors[2].half(), r.tensors[3])
    assert (r.out == 7).all()
    # no rows, no tokens: nothing to do
    empty = b.make_params(0, 8, 2, 128, r.c.width, r.c.pages, BF16)
    z = [t[:0] for t in (r.q, r.k, r.v, r.pos)]
    b.coded_decode(empty, r.cache, *z, r.table[:0], r.out[:0], r.ws)
    b.coded_prefill(r.p, r.cache, *z, r.rows[:0], r.slots[:0], r.table, r.out[:0], r.ws)
    b.coded_read(r.p, r.cache, r.slots[:0], r.k[:0], r.v[:0], r.ws)
    assert b.last_launch_count() == 0


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    r = Run(cu.Case(8, 2, 128, [300, 500], [1, 1]))
    hold = r.ws[13 * 4:14 * 4].view(torch.int32)       # the control block's test hook (test_gpu_timeout.py)
    hold.fill_(1)
    r.decode()
    with pytest.raises(r.b.PdattnError) as e:
        r.b.check_status(r.ws)
    assert e.value.status == ETIMEOUT
    hold.fill_(0)
    r.check("decode")


# ---------------------------------------------------------------------------
# keys that a token does not see
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("power", [10, 20, 24, 30, 60])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("heads,kv_heads,D,prefix,chunk,at,window,kind", [
    (4, 1, 128, 300, 40, 335, 0, E4M3),      # a later token of the chunk; tiles of 64, cut along the keys
    (8, 2, 64, 150, 20, 165, 0, INT8),       # tiles of one half: blocks alternate
    (2, 2, 64, 30, 230, 100, 50, E4M3),      # the window leaves it behind inside a tile of 256
    (16, 2, 128, 300, 30, 290, 20, INT8),    # a cached token that the last tokens' window excludes
])
def test_a_huge_key_or_value_leaves_the_tokens_that_do_not_see_it_alone(heads, kv_heads, D, prefix, chunk, at, window,
                                                                        kind, which, power):
    c = cu.Case(heads, kv_heads, D, [prefix], [chunk], BF16, kind, window=window, seed=power)
    if at >= prefix:
        getattr(c, which + "_new")[at - prefix] *= 2.0 ** power
    else:
        slot = int(c.table[0, at // 64]) * 64 + at % 64
        getattr(c.cache, which + "s")[slot // 64, :, slot % 64] *= 2.0 ** power
    r = Run(c)
    r.prefill()
    r.b.check_status(r.ws)
    c.write()
    c.cache.same(r.tensors)
    want, bound = c.want("prefill")
    # a token that sees a value 2^24 times the others' may lose the others
    sees = (c.positions >= at) & ((c.positions < at + window) if window else torch.tensor(True))
    held = torch.ones_like(sees) if which == "k" or power < 14 else ~sees
    assert held.any() and not held.all() or which == "k" or power < 14
    cu.hold(r.out[held.cuda()], want[held], bound[held])


def test_sizes_of_keys_and_values_all_over_the_range():
    # every token of another size; rows split, alternating and whole
    g = torch.Generator().manual_seed(12)
    for prefix, chunk, window in (([700], [9], 0), ([90, 0], [130, 70], 0), ([200], [150], 60)):
        c = cu.Case(8, 2, 128, prefix, chunk, BF16, E4M3, 0.0, window)
        c.cache.ks *= 2.0 ** torch.randint(-30, 2, c.cache.ks.shape, generator=g)
        c.cache.vs *= 2.0 ** torch.randint(-30, 30, c.cache.vs.shape, generator=g)
        c.k_new *= 2.0 ** torch.randint(-30, 2, c.k_new.shape[:2], generator=g)[..., None]
        c.v_new *= 2.0 ** torch.randint(-30, 30, c.v_new.shape[:2], generator=g)[..., None]
        c.k_new[3], c.v_new[5] = 0.0, 0.0
        Run(c).check("prefill")


def _garbage_where_nobody_looks(r):
    """Finite garbage in every slot that no single token sees: scales of 1e30, codes that are NaN in e4m3."""
    c = r.c
    seen = torch.zeros(c.pages * 64, dtype=torch.bool)
    for row, pos in zip(c.rows.tolist(), c.positions.tolist()):
        t = torch.arange(max(0, pos - c.window + 1) if c.window > 0 else 0, pos + 1)
        seen[c.table[row].long()[t // 64] * 64 + t % 64] = True
    page, off = (~seen.view(c.pages, 64)).nonzero(as_tuple=True)
    for codes, scales in ((r.tensors[0], r.tensors[2]), (r.tensors[1], r.tensors[3])):
        codes.view(torch.uint8)[page, :, off] = 0x7f
        scales[page, :, off] = 1e30


def _moved(c, positions):
    """The case with its tokens at other positions of their rows."""
    c.positions = positions.to(torch.int32)
    c.slots = (c.table[c.rows.long(), c.positions.long() // 64] * 64 + c.positions % 64).to(torch.int32)
    return c


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("heads,kv_heads,order", [(8, 2, "two runs"), (8, 2, "in turn"), (2, 2, "two runs"), (2, 2, "backwards"),
                                                  (16, 2, "three runs")])
def test_keys_between_the_windows_of_a_rows_tokens_reach_no_output(heads, kv_heads, order, kind):
    at = {"two runs": [*range(5, 15), *range(890, 900)], "in turn": [x for i in range(10) for x in (5 + i, 890 + i)],
          "backwards": [*range(899, 889, -1), *range(14, 4, -1)],
          "three runs": [*range(300, 308), *range(10, 14), *range(892, 900)]}[order]
    outs = []
    for dirty in (False, True):
        r = Run(_moved(cu.Case(heads, kv_heads, 128, [880], [20], kind=kind, window=50), torch.tensor(at)))
        if dirty:
            _garbage_where_nobody_looks(r)
        r.prefill()
        r.b.check_status(r.ws)
        outs.append(r.out)
    assert torch.equal(*outs)
    r.c.write()
    want, bound = r.c.want("prefill")
    cu.hold(r.out, want, bound)


@pytest.mark.parametrize("rows,chunk,kv_heads,launches", [(100, 42, 1, 4), (32, 40, 64, 3)])
def test_windows_that_leave_gaps_in_calls_of_many_tokens(rows, chunk, kv_heads, launches):
    # more tokens than the one-pass planner takes, and a call that is not cut along the keys
    at = torch.tensor([*range(3, 3 + chunk // 2), *range(300 - chunk // 2, 300)]).repeat(rows)
    outs = []
    for dirty in (False, True):
        c = cu.Case(kv_heads, kv_heads, 64, [300 - chunk] * rows, [chunk] * rows, theta=0.0, window=40)
        r = Run(_moved(c, at))
        if dirty:
            _garbage_where_nobody_looks(r)
        r.prefill()
        assert r.b.last_launch_count() == launches
        r.b.check_status(r.ws)
        outs.append(r.out)
    assert torch.isfinite(outs[0]).all() and torch.equal(*outs)
# ---------------------------------------------------------------------------
# positions past the rope table
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_row_past_the_rope_table_is_skipped(dtype):
    c = cu.Case(8, 2, 128, [100, 5, 200, 70], [1, 1, 1, 1], dtype)
    r = Run(c)
    r.check("decode")                                    # leaves every row's query in the workspace
    g = torch.Generator().manual_seed(2)
    c.q, c.k_new, c.v_new = (torch.randn(x.shape, generator=g).to(dtype) for x in (c.q, c.k_new, c.v_new))
    for dst, src in ((r.q, c.q), (r.k, c.k_new), (r.v, c.v_new)):
        dst.copy_(src)
    r.p.rope_len = 128                                   # rows 0, 1 and 3 lie in it
    r.out.fill_(7.0)
    r.decode()
    with pytest.raises(r.b.PdattnError) as e:
        r.b.check_status(r.ws)
    assert e.value.status == EBADPOS
    assert (r.out[2] == 7).all()
    keep = torch.tensor([0, 1, 3])
    c.cache.write(cu.rope(c.k_new.float(), c.cos, c.sin, c.positions)[keep], c.v_new.float()[keep], c.slots[keep])
    c.cache.same(r.tensors)
    want, bound = c.want("decode")
    cu.hold(r.out[keep.cuda()], want[keep], bound[keep])
# ---------------------------------------------------------------------------
# scores far beyond the exponential's precision
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("power", [20, 30, 40])
@pytest.mark.parametrize("what,dtype,kind", [("decode", BF16, E4M3), ("decode", F32, INT8), ("decode", F32, E4M3),
                                             ("prefill", BF16, INT8)])
def test_keys_of_any_size_pick_the_largest_score(what, dtype, kind, power):
    heads = 8 if kind == INT8 else 4                     # f32 groups of four and of eight
    c = cu.Case(heads, 1, 64, [100, 300], [1, 1] if what == "decode" else [9, 30], dtype, kind, 0.0, seed=power)
    c.cache.ks *= 2.0 ** power
    c.k_new = c.k_new * 2.0 ** power
    r = Run(c)
    getattr(r, what)()
    r.b.check_status(r.ws)
    c.write()
    out = r.out.cpu().double()
    assert torch.isfinite(out).all()
    sure = 0
    for i, (row, pos) in enumerate(zip(c.rows.tolist(), c.positions.tolist())):
        t = torch.arange(pos + 1)
        slots = c.table[row].long()[t // 64] * 64 + t % 64
        k, v = (c.cache.meant(a, s, slots)[:, 0] for a, s in ((c.cache.k, c.cache.ks), (c.cache.v, c.cache.vs)))
        s = c.q[i].double() @ k.T / 8.0
        # q, K's ratio and code * ratio in 11 bits, f32 sums: scores closer than this may change places
        off = 2 * (3 * 2.0 ** -11 + 72 * 2.0 ** -24) * (c.q[i].double().abs() @ k.abs().T / 8.0).amax(-1)
        top2 = s.topk(2, -1)
        for h in range(heads):
            if top2.values[h, 0] - top2.values[h, 1] > off[h] + 200:      # the others' weights are nothing
                sure += 1
                want = v[top2.indices[h, 0]]
                assert ((out[i, h] - want).abs() <= want.abs() * 2.0 ** -7 + 2.0 ** -20).all()
    assert sure >= len(c.q) * heads // 2
# ---------------------------------------------------------------------------
# more of what a call may be given
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("what,dtype", [("decode", BF16), ("decode", F32), ("prefill", BF16)])
def test_a_query_that_is_not_finite_spoils_its_own_head_only(what, dtype, value):
    c = cu.Case(8, 2, 64, [70, 300, 10], [1, 1, 1] if what == "decode" else [20, 3, 40], dtype)
    n = 1 if what == "decode" else 12
    c.q[n, 5, 17] = value
    r = Run(c)
    getattr(r, what)()
    r.b.check_status(r.ws)
    out = r.out.cpu()
    assert torch.isnan(out[n, 5]).all()
    out[n, 5] = 0
    assert torch.isfinite(out).all()


def test_workspaces_of_other_types_and_wrong_ones():
    c = cu.Case(8, 2, 128, [10], [1])
    r = Run(c)
    r.ws = torch.zeros(r.ws.numel() // 4, dtype=torch.int32, device="cuda")
    r.check("decode")
    b = r.b
    for bad in (None, r.ws.cpu(), r.ws[::2], 7):
        with pytest.raises((ValueError, TypeError)):
            b.coded_decode(r.p, r.cache, r.q, r.k, r.v, r.pos, r.table, r.out, bad)
        with pytest.raises((ValueError, TypeError)):
            b.coded_write(r.p, r.cache, r.k, r.v, r.pos, r.slots, bad)


@pytest.mark.parametrize("heads,kv_heads,D,prefix,chunk,split", [
    (8, 2, 128, [0], [1], False), (4, 4, 64, [0, 10], [129, 260], False), (2, 2, 128, [3000], [2], True),
    (8, 2, 64, [0, 2500], [40, 3], True)])
def test_which_calls_are_cut_along_the_keys(heads, kv_heads, D, prefix, chunk, split):
    r = Run(cu.Case(heads, kv_heads, D, prefix, chunk))
    r.prefill()
    assert r.b.last_launch_count() == 4                  # few tiles: they may be cut, and a merge follows
    last_cut = int(r.ws[9 * 4:10 * 4].view(torch.int32))  # the control block's count of tiles up to the last one cut
    r.b.check_status(r.ws)
    assert (last_cut > 0) == split


@pytest.mark.parametrize("spread", [9, 14, 19, 22])
@pytest.mark.parametrize("heads,kv_heads,D,prefix,chunk,window", [(4, 1, 128, [1500], [6], 0), (8, 1, 64, [700], [70], 0),
                                                                 (2, 2, 128, [200, 40], [300, 5], 90)])
def test_scales_that_lie_far_apart(heads, kv_heads, D, prefix, chunk, window, spread):
    # up to where ratios still hold them, at the border and past it; whole blocks of larger and smaller ones
    g = torch.Generator().manual_seed(spread)
    c = cu.Case(heads, kv_heads, D, prefix, chunk, BF16, INT8, 0.0, window)
    for scales in (c.cache.ks, c.cache.vs):
        scales *= 2.0 ** torch.randint(-spread, 1, scales.shape, generator=g)
    c.cache.vs *= 2.0 ** torch.randint(-8, 9, c.cache.vs.shape[:1], generator=g)[:, None, None]
    Run(c).check("prefill")


def test_a_write_without_rotation_takes_any_position():
    c = cu.Case(2, 2, 64, [0], [3], theta=0.0)
    r = Run(c)
    pos = torch.tensor([0, 10 ** 9, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    r.b.coded_write(r.p, r.cache, r.k, r.v, pos, r.slots, r.ws)
    r.b.check_status(r.ws)
    c.write()
    c.cache.same(r.tensors)


@pytest.mark.parametrize("what,prefix,chunk", [("prefill", [3000], [2]), ("prefill", [300], [40]), ("decode", [3000], [1])])
def test_values_near_the_end_of_the_range(what, prefix, chunk):
    # values of 2^124: outputs are averages of values, and no sum on the way may leave f32
    c = cu.Case(2, 2, 128, prefix, chunk, BF16, E4M3, 0.0, seed=1)
    c.cache.vs[:, :, ::7] = 2.0 ** 115
    Run(c).check(what)


@pytest.mark.parametrize("what,prefix,chunk", [("prefill", [8000], [2]), ("prefill", [9, 2000], [70, 130]), ("decode", [8000], [1])])
def test_values_near_the_lower_end_of_the_range(what, prefix, chunk):
    # values of about 2^-110: averages of many of them are still normal numbers
    c = cu.Case(2, 2, 64, prefix, chunk, BF16, E4M3, 0.0, seed=1)
    c.cache.vs.fill_(2.0 ** -118)
    c.v_new = c.v_new * 2.0 ** -112
    Run(c).check(what)


def test_prefills_on_two_streams_at_once():
    cases = [cu.Case(8, 2, 128, [900, 30], [5, 200], seed=i, window=(0, 70)[i]) for i in range(2)]
    runs = [Run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(4):
        for r, s in zip(runs, streams):
            with torch.cuda.stream(s):
                r.prefill()
    torch.cuda.synchronize()
    for r in runs:
        r.b.check_status(r.ws)
        r.c.write()
        r.c.cache.same(r.tensors)
        want, bound = r.c.want("prefill")
        cu.hold(r.out, want, bound)


def test_two_graphs_that_share_a_workspace():
    """Captured calls of both kinds on one workspace, replayed in turn in both orders."""
    pre, dec = cu.Case(8, 2, 128, [300, 20], [6, 90]), cu.Case(8, 2, 128, [700, 64], [1, 1], seed=2)
    runs = [(Run(pre), "prefill"), (Run(dec), "decode")]
    ws = max((r.ws for r, _ in runs), key=lambda t: t.numel())
    graphs = []
    for r, kind in runs:
        r.ws = ws
        getattr(r, kind)()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            getattr(r, kind)()
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for r, _ in runs:
            r.out.fill_(0)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for r, kind in runs:
            r.b.check_status(ws)
            r.c.write()
            want, bound = r.c.want(kind)
            cu.hold(r.out, want, bound, f"{kind} {order}")


@pytest.mark.parametrize("which", ["k_new", "v_new"])
def test_a_non_finite_token_beside_a_huge_one(which):
    c = cu.Case(8, 2, 128, [70], [30])
    getattr(c, which)[9, 1, 3] = math.nan
    c.v_new[20] *= 2.0 ** 60
    c.k_new[25] *= 2.0 ** 30
    r = Run(c)
    r.prefill()
    r.b.check_status(r.ws)
    out = r.out.cpu()
    assert torch.isfinite(out[:, :4]).all() and torch.isfinite(out[:9]).all() and torch.isnan(out[9:, 4:]).all()
    c.write()
    want, bound = c.want("prefill")
    cu.hold(out[:9], want[:9], bound[:9])
    cu.hold(out[:20, :4], want[:20, :4], bound[:20, :4])
