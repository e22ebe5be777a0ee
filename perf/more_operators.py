"""Cases of the operators for many continuations of one long prompt: rotary positions for long contexts, a paged cache
whose rows fork, grow and are moved together, and a decode step that attends a shared prefix once for all its rows.

  tables    cos and sin [length, D] of rotary frequencies that are scaled for long contexts
  rotary    q and k turned at their positions (or back: the gradient), half or interleaved pairs, part of the head
  update    the page table after a step: rows continue, fork, start anew, give room back or take more; a partly filled
            page that two rows hold is copied for the one that writes it
  compact   the pages in use moved to the lowest ids, with their tables
  shared    one new token per row, where groups of rows hold the same leading pages

`run` computes them in elementary torch operations, or, where `own` is true, by the framework's calls.
"""
import math
import random

import torch

own = False

PAGE = 64
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LLAMA = dict(heads=32, kv_heads=8, head_dim=128, dtype="bf16")
GPTOSS = dict(heads=64, kv_heads=8, head_dim=64, dtype="bf16")
GPT2 = dict(heads=12, kv_heads=12, head_dim=64, dtype="f32")
PLAIN = dict(scaling="none", factor=1.0, low=1.0, high=1.0, original=0)
WAVES = dict(scaling="wavelength", factor=8.0, low=1.0, high=4.0, original=8192)
RAMP = dict(scaling="ramp", factor=32.0, low=1.0, high=32.0, original=4096)


def listed():
    return [
        # the tables of a short model, built at start
        dict(name="tables_short", op="tables", length=4096, head_dim=64, dtype="bf16", theta=150000.0, **RAMP),
        # the tables of a context of 131072 positions
        dict(name="tables_long", op="tables", length=131072, head_dim=128, dtype="bf16", theta=500000.0, **WAVES),
        # one decode step's tokens
        dict(name="rotary_step", op="rotary", tokens=37, rot=64, interleaved=False, inverse=False, joined=False,
             top=1024, theta=10000.0, **GPT2, **PLAIN),
        # the gradient of a prompt batch's q and k inside the gradient of one joined projection, pairs interleaved, half
        # of the head
        dict(name="rotary_grad", op="rotary", tokens=8192, rot=64, interleaved=True, inverse=True, joined=True,
             top=131072, theta=500000.0, **LLAMA, **WAVES),
        # a decode step's bookkeeping: every row takes one more position, some start anew
        dict(name="update_step", op="update", rows=64, beams=1, prompt_lo=257, prompt_hi=4000, own_hi=96, grow=1,
             pools=2, kv_heads=8, head_dim=64, dtype="bf16"),
        # beams continue one another: tails are copied in four layers' caches
        dict(name="update_beams", op="update", rows=256, beams=4, prompt_lo=100, prompt_hi=600, own_hi=200, grow=1,
             pools=8, kv_heads=8, head_dim=128, dtype="bf16"),
        # a small int8 cache with its scales
        dict(name="compact_coded", op="compact", rows=9, beams=3, prompt_lo=65, prompt_hi=300, own_hi=70, live=0.55,
             pools=4, kv_heads=12, head_dim=64, dtype="int8"),
        # a fragmented cache of two layers
        dict(name="compact_large", op="compact", rows=96, beams=2, prompt_lo=300, prompt_hi=1300, own_hi=400, live=0.45,
             pools=4, kv_heads=8, head_dim=128, dtype="bf16"),
        # five samples of one short prompt
        dict(name="shared_samples", op="shared", rows=5, groups=1, prefix_lo=7, prefix_hi=7, own_lo=1, own_hi=100,
             window=0, sinks=True, theta=150000.0, **GPTOSS),
        # requests under one system prompt
        dict(name="shared_system", op="shared", rows=64, groups=1, prefix_lo=32, prefix_hi=32, own_lo=16, own_hi=2000,
             window=0, sinks=True, theta=150000.0, **GPTOSS),
        # questions about one long document
        dict(name="shared_document", op="shared", rows=24, groups=1, prefix_lo=1023, prefix_hi=1023, own_lo=5,
             own_hi=300, window=0, sinks=False, theta=500000.0, **LLAMA),
        # a serving batch of several prompts
        dict(name="shared_serving", op="shared", rows=256, groups=6, prefix_lo=8, prefix_hi=64, own_lo=1, own_hi=1500,
             window=0, sinks=False, theta=500000.0, **LLAMA),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["tables", "rotary", "rotary", "update", "update", "compact", "shared", "shared", "shared"])
    if op in ("tables", "rotary"):
        c = dict(op=op, head_dim=rng.choice([64, 128]), dtype=rng.choice(["bf16", "f32"]),
                 theta=rng.choice([10000.0, 150000.0, 500000.0]))
        c.update(rng.choice([PLAIN, dict(PLAIN, scaling="linear", factor=4.0), WAVES, RAMP]))
        if op == "tables":
            return dict(c, length=_log_int(rng, 1, 65536))
        kv_heads = rng.choice([1, 2, 4, 8, 12])
        return dict(c, tokens=_log_int(rng, 1, 4096), heads=kv_heads * rng.choice([1, 3, 4, 5]), kv_heads=kv_heads,
                    rot=rng.choice([c["head_dim"], c["head_dim"] // 2, 32, 48]), interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.4, joined=rng.random() < 0.5, top=_log_int(rng, 64, 1 << 20))
    if op in ("update", "compact"):
        beams = rng.choice([1, 1, 2, 3, 5])
        hi = _log_int(rng, 1, 1200)
        c = dict(op=op, rows=beams * _log_int(rng, 1, 160 // beams), beams=beams, prompt_lo=rng.randint(1, hi),
                 prompt_hi=hi, own_hi=_log_int(rng, 1, 200), pools=rng.choice([1, 2, 3, 4]),
                 kv_heads=rng.choice([1, 2, 5, 8]), head_dim=rng.choice([64, 128]),
                 dtype=rng.choice(["bf16", "f32", "int8"]))
        return dict(c, grow=_log_int(rng, 1, 150)) if op == "update" else dict(c, live=rng.uniform(0.2, 0.95))
    kv_heads = rng.choice([1, 2, 4, 8])
    rows = _log_int(rng, 1, 192)
    hi = min(_log_int(rng, 1, 400), 6000 // rows + 8)
    own_hi = min(_log_int(rng, 1, 3000), 300000 // rows)
    return dict(op=op, heads=kv_heads * rng.choice([1, 2, 3, 4, 5, 8]), kv_heads=kv_heads,
                head_dim=rng.choice([64, 128]), dtype="bf16", rows=rows, groups=rng.randint(1, min(rows, 7)),
                prefix_lo=rng.randint(0, hi), prefix_hi=hi, own_lo=rng.randint(1, own_hi), own_hi=own_hi,
                window=rng.choice([0, 0, 0, _log_int(rng, 1, 4000)]), sinks=rng.random() < 0.3,
                theta=rng.choice([0.0, 10000.0, 500000.0]))


def _spaced(lo, hi, n):
    """n whole numbers over [lo, hi], the ends among them where n > 1."""
    return [int(round(lo + (hi - lo) * (i / (n - 1) if n > 1 else 1.0))) for i in range(n)]


# ---- rotary -----------------------------------------------------------------------------------------------------------

def _frequencies(case, rot):
    """Radians per position of every pair, in 64 bits, and the factor of cos and sin."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    f = torch.exp(i * (-2.0 / rot * math.log(case["theta"])))
    slow = f / case["factor"]
    if case["scaling"] == "linear":
        return slow, 1.0
    if case["scaling"] == "wavelength":
        # turns of the pair over the original context: under `low` slowed down, over `high` left as they are
        turns = case["original"] * f / (2 * math.pi)
        keep = ((turns - case["low"]) / (case["high"] - case["low"])).clamp(0.0, 1.0)
        return slow * (1 - keep) + f * keep, 1.0
    if case["scaling"] == "ramp":
        # pairs between those of `high` and of `low` turns over the original context, by their index
        at = [rot / 2 * math.log(case["original"] / (2 * math.pi * t)) / math.log(case["theta"])
              for t in (case["high"], case["low"])]
        keep = 1 - ((i - at[0]) / max(at[1] - at[0], 1e-3)).clamp(0.0, 1.0)
        return slow * (1 - keep) + f * keep, 0.1 * math.log(case["factor"]) + 1.0
    return f, 1.0


def _cos_sin(case, rot, positions):
    f, gain = _frequencies(case, rot)
    angle = positions.double()[:, None] * f
    return torch.cos(angle) * gain, torch.sin(angle) * gain


def _turned(x, s):
    """x [n, heads, D] in f32, its pairs turned by their angles (back, where the case is the gradient)."""
    rot = s["rot"]
    c, sn = (t.float()[:, None] for t in _cos_sin(s, rot, s["positions"]))
    sn = -sn if s["inverse"] else sn
    x = x.float()
    if s["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([y, x[..., rot:]], -1).to(TYPES[s["dtype"]])


# ---- pages ------------------------------------------------------------------------------------------------------------

def _page_rows(case):
    """(length, prompt pages shared by the row's beams, the row's beam group) of every row, from the case alone."""
    rng = random.Random(case["rows"] * 7919 + case["prompt_hi"])
    rows = []
    for b, prompt in enumerate(_spaced(case["prompt_lo"], case["prompt_hi"], case["rows"] // case["beams"])):
        length = prompt + rng.randint(0, case["own_hi"])
        rows += [(length, prompt // PAGE if case["beams"] > 1 else 0, b)] * case["beams"]
    return rows


def _asked(case):
    """(parents, new lengths) of an update: beams continue one another; one row in 16 starts anew, one in 16 gives
    positions back."""
    rng = random.Random(case["rows"] * 104729 + case["own_hi"])
    rows, parents, lengths = _page_rows(case), [], []
    for r, (length, _, b) in enumerate(rows):
        parents.append(b * case["beams"] + rng.randrange(case["beams"]))
        lengths.append(length + case["grow"])
        kind = rng.randrange(16)
        if kind == 0:
            parents[r], lengths[r] = -1, rng.randint(0, case["prompt_hi"])
        elif kind == 1:
            lengths[r] = rng.randint(0, length)
    return parents, lengths


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _page_counts(case):
    """(pages of the pool, table width)."""
    rows = _page_rows(case)
    used = 3
    for r, (length, common, b) in enumerate(rows):
        used += _pages(length) - (common if r % case["beams"] else 0)
    longest = max(n for n, _, _ in rows)
    if case["op"] == "compact":
        return int(used / case["live"]) + 1, _pages(longest) + 2
    fresh = sum(_pages(n) for n in _asked(case)[1])
    return used + min(fresh, 3 * case["rows"] + 40 * _pages(case["prompt_hi"])), _pages(max([longest] + _asked(case)[1])) + 1


def _page_state(case, seed):
    """Table, lengths and reference counts of a cache whose pages lie anywhere; three pages are held by no row, and the
    first group's first page once more (a kept prefix)."""
    rng = random.Random(seed)
    rows = _page_rows(case)
    pages, width = _page_counts(case)
    ids = list(range(pages))
    rng.shuffle(ids)
    table, refs, at = [], [0] * pages, 0
    for r, (length, common, b) in enumerate(rows):
        mine = table[-1][:common] if r % case["beams"] else []
        k = _pages(length) - len(mine)
        mine = mine + ids[at:at + k]
        at += k
        for x in mine:
            refs[x] += 1
        table.append(mine + [-1] * (width - len(mine)))
    for x in ids[at:at + 3]:
        refs[x] = 1
    if rows[0][0] > 0:
        refs[table[0][0]] += 1
    return table, [n for n, _, _ in rows], refs


def _update_plan(s):
    """The new table and counts, and which rows copy a tail: from where, to where, how many positions."""
    table, lengths, refs = s["table"].long(), s["lengths"].long(), s["refs"].long()
    parents, new = s["parents"].long(), s["new_lengths"].long()
    R, W = table.shape
    N = refs.numel()
    col, row = torch.arange(W, device="cuda"), torch.arange(R, device="cuda")

    def counted(mask, pages):
        return torch.zeros(N + 1, dtype=torch.int64, device="cuda").scatter_add_(
            0, torch.where(mask, pages, N).flatten(), torch.ones(R * W, dtype=torch.int64, device="cuda"))[:N]

    pins = refs - counted(col < ((lengths + PAGE - 1) // PAGE)[:, None], table)
    src = table[parents.clamp(min=0)]
    keep = torch.where(parents >= 0, torch.minimum(lengths[parents.clamp(min=0)], new), 0)
    full, part, writes = keep // PAGE, keep % PAGE > 0, new > keep
    shared = (col < full[:, None]) | ((col == full[:, None]) & (part & ~writes)[:, None])
    others = counted(shared, src) + pins
    tail = torch.where(part & writes, src.gather(1, full.clamp(max=W - 1)[:, None])[:, 0], N)
    first = torch.full((N + 1,), R, dtype=torch.int64, device="cuda").scatter_reduce_(0, tail, row, "amin")
    others = torch.cat([others, others.new_zeros(1)])
    alone = (others[tail] == 0) & (first[tail] == row)
    copied = part & writes & ~alone
    after = others[:N] + ((others[:N] == 0) & (first[:N] < R))
    free = torch.sort(torch.where(after == 0, torch.arange(N, device="cuda"), N)).values
    kept, pages = full + (part & ~copied), (new + PAGE - 1) // PAGE
    need = pages - kept
    at = (torch.cumsum(need, 0) - need)[:, None] + col - kept[:, None]
    fresh = (col >= kept[:, None]) & (col < pages[:, None])
    out = torch.where(col < kept[:, None], src, torch.where(fresh, free[at.clamp(0, N - 1)], -1))
    after = after + counted(fresh, out)
    to = out.gather(1, full.clamp(max=W - 1)[:, None])[:, 0]
    return out.to(torch.int32), after.to(torch.int32), copied, tail, to, keep % PAGE


def _copy_tails(pool, copied, tail, to, tokens):
    """pool [pools, pages, kv_heads, 64, ...]: the first `tokens` positions of page `tail` put into page `to`."""
    at = torch.nonzero(copied)[:, 0]
    seen = torch.arange(PAGE, device="cuda") < tokens[at][:, None]
    seen = seen.view(1, -1, 1, PAGE, *[1] * (pool.dim() - 4))
    pool[:, to[at]] = torch.where(seen, pool[:, tail[at]], pool[:, to[at]])


def _compact_plan(s):
    refs, table, lengths = s["refs"].long(), s["table"].long(), s["lengths"].long()
    N, W = refs.numel(), table.shape[1]
    ids, live = torch.arange(N, device="cuda"), refs > 0
    n = live.sum()
    high, hole = live & (ids >= n), ~live & (ids < n)
    # the k-th page in use above goes to the k-th hole below
    holes = torch.sort(torch.where(hole, ids, N)).values
    to = torch.where(high, holes[(torch.cumsum(high.long(), 0) - 1).clamp(min=0)], torch.where(live, ids, -1))
    held = torch.arange(W, device="cuda") < ((lengths + PAGE - 1) // PAGE)[:, None]
    after = torch.where(held, to[table.clamp(min=0)], table)
    counts = torch.where(ids < n, torch.where(hole, 0, refs), 0).scatter_add_(
        0, torch.where(high, to, 0), torch.where(high, refs, 0))
    return after.to(torch.int32), counts.to(torch.int32), to.to(torch.int32), high


# ---- shared prefixes --------------------------------------------------------------------------------------------------

def _groups(case):
    """(rows of every group, its shared pages, every row's own positions), from the case alone."""
    rng = random.Random(case["rows"] * 31 + case["groups"])
    cuts = sorted(rng.sample(range(1, case["rows"]), case["groups"] - 1))
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [case["rows"]])]
    prefixes = _spaced(case["prefix_lo"], case["prefix_hi"], case["groups"])
    own_lengths = _spaced(case["own_lo"], case["own_hi"], case["rows"])
    rng.shuffle(prefixes)
    rng.shuffle(own_lengths)
    return sizes, prefixes, own_lengths


def _tables(theta, D, T, length):
    """Rotary cos and sin [length, D] in T, or None without rotation."""
    if theta <= 0:
        return None, None
    freq = torch.exp(-torch.arange(D // 2, device="cuda", dtype=torch.float64) * 2 / D * math.log(theta))
    angle = torch.arange(length, device="cuda", dtype=torch.float64)[:, None] * freq
    angle = torch.cat([angle, angle], -1)
    return torch.cos(angle).to(T), torch.sin(angle).to(T)


def _rope(x, s):
    """x [n, heads, D] rotated at the rows' positions, in f32."""
    x = x.float()
    if s["cos"] is None:
        return x
    at = s["positions"].long()
    c, sn = s["cos"][at].float().unsqueeze(1), s["sin"][at].float().unsqueeze(1)
    half = x.shape[-1] // 2
    return x * c + torch.cat([-x[..., half:], x[..., :half]], -1) * sn


def _decode(s):
    """Every row's token over its positions [pos - window + 1, pos]."""
    Hq, Hk, D, R, T = s["heads"], s["kv_heads"], s["head_dim"], s["rows"], TYPES[s["dtype"]]
    page, off = s["table"].long().gather(1, s["positions"].long()[:, None] // PAGE)[:, 0], s["positions"].long() % PAGE
    s["k_pool"][page, :, off] = _rope(s["k_new"], s).to(T)
    s["v_pool"][page, :, off] = s["v_new"]
    q = _rope(s["q"], s).to(T).float().view(R, Hk, Hq // Hk, D)
    at = s["table"].long().clamp(min=0)
    keys, values = (s[n][at].transpose(1, 2).reshape(R, Hk, -1, D).float() for n in ("k_pool", "v_pool"))
    score = (q @ keys.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    t, pos = torch.arange(keys.shape[2], device="cuda"), s["positions"].long()[:, None]
    seen = (t <= pos) & ((t > pos - s["window"]) if s["window"] > 0 else True)
    score = torch.where(seen[:, None, None], score, -math.inf)
    values = torch.where(seen[:, None, :, None], values, 0.0)
    top = score.amax(-1, keepdim=True)
    sink = s["sink"].float().view(Hk, -1, 1) if s["sink"] is not None else torch.full((1, 1, 1), -math.inf, device="cuda")
    top = torch.maximum(top, sink)
    w = torch.exp(score - top)
    return ((w @ values) / (w.sum(-1, keepdim=True) + torch.exp(sink - top))).view(R, Hq, D).to(T)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s, op = dict(case), case["op"]

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    if op == "tables":
        # what is made at start has no inputs but the model's numbers: another seed is another theta
        s["theta"] = case["theta"] * (1.0 + 0.001 * (seed % 1009))
    elif op == "rotary":
        n, Hq, Hk, D, T = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"], TYPES[case["dtype"]]
        x = torch.randn(n, Hq + 2 * Hk, D, generator=g, device="cuda").to(T)
        # slices of one projection of q, k and v, or tensors of their own
        s["q"], s["k"] = x[:, :Hq], x[:, Hq:Hq + Hk]
        if not case["joined"]:
            s["q"], s["k"] = s["q"].contiguous(), s["k"].contiguous()
        s["positions"] = torch.randint(0, case["top"], (n,), generator=g, device="cuda").to(torch.int32)
        s["q_out"], s["k_out"] = (torch.empty(n, h, D, dtype=T, device="cuda") for h in (Hq, Hk))
    elif op in ("update", "compact"):
        table, lengths, refs = _page_state(case, seed)
        pages, width = _page_counts(case)
        s["table"], s["lengths"], s["refs"] = ints(table), ints(lengths), ints(refs)
        s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
        s["map"] = torch.empty_like(s["refs"])
        if op == "update":
            s["parents"], s["new_lengths"] = (ints(x) for x in _asked(case))
        shape = (case["pools"], pages, case["kv_heads"], PAGE, case["head_dim"])
        if case["dtype"] == "int8":
            s["pools"] = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
            s["scales"] = torch.rand(shape[:4], generator=g, device="cuda")
        else:
            s["pools"] = torch.empty(shape, dtype=TYPES[case["dtype"]], device="cuda").normal_(generator=g)
            s["scales"] = None
    else:
        sizes, prefixes, lengths = _groups(case)
        Hq, Hk, D, R, T = case["heads"], case["kv_heads"], case["head_dim"], case["rows"], TYPES[case["dtype"]]
        rows = [(b, p) for (b, p) in zip(sizes, prefixes) for _ in range(b)]
        width = max(p + _pages(n) for (_, p), n in zip(rows, lengths))
        need = sum(prefixes) + sum(_pages(n) for n in lengths)
        pages = need + 1 + need // 10
        ids = torch.randperm(pages, generator=g, device="cuda").tolist()
        table, at, r = [], 0, 0
        for size, p in zip(sizes, prefixes):
            common, at = ids[at:at + p], at + p
            for _ in range(size):
                k = _pages(lengths[r])
                table.append(common + ids[at:at + k] + [-1] * (width - p - k))
                at, r = at + k, r + 1
        s["table"] = ints(table)
        s["positions"] = ints([p * PAGE + n - 1 for (_, p), n in zip(rows, lengths)])
        s["group_start"], s["group_pages"] = ints([sum(sizes[:i]) for i in range(len(sizes) + 1)]), ints(prefixes)
        s["q"], s["k_new"], s["v_new"] = (torch.randn(R, h, D, generator=g, device="cuda").to(T) for h in (Hq, Hk, Hk))
        s["out"] = torch.empty_like(s["q"])
        s["sink"] = torch.randn(Hq, generator=g, device="cuda").to(T) if case["sinks"] else None
        s["cos"], s["sin"] = _tables(case["theta"], D, T, width * PAGE)
        s["k_pool"], s["v_pool"] = (torch.empty(pages, Hk, PAGE, D, dtype=T, device="cuda").normal_(generator=g)
                                    for _ in range(2))
        # some channels of the keys are larger than others
        s["k_pool"] *= torch.exp(0.4 * torch.randn(Hk, 1, D, generator=g, device="cuda")).to(T)
    if own:
        from paged_gqa_decode_step_gb300 import binding as b
        if op in ("tables", "rotary"):
            s["rotary"] = b.make_rotary(case["head_dim"], s["theta"], rot_dim=case.get("rot", case["head_dim"]),
                                        interleaved=case.get("interleaved", False), scaling=case["scaling"],
                                        factor=case["factor"], low=case["low"], high=case["high"],
                                        original_len=case["original"])
            s["ws"] = b.new_status()
        elif op in ("update", "compact"):
            s["params"] = b.make_params(case["rows"], case["kv_heads"], case["kv_heads"], case["head_dim"],
                                        s["table"].shape[1], s["refs"].numel(), torch.bfloat16)
            every = list(s["pools"].unbind()) + (list(s["scales"].unbind()) if s["scales"] is not None else [])
            s["cache"] = b.make_pages(s["params"], every)
            s["ws"] = b.new_pages_workspace(s["params"])
        else:
            s["params"] = b.make_params(R, Hq, Hk, D, s["table"].shape[1], s["k_pool"].shape[0], T,
                                        window=case["window"], rope_cos=s["cos"], rope_sin=s["sin"], sinks=s["sink"])
            s["ws"] = b.new_shared_workspace(s["params"], case["groups"])
    return s


def _run_own(s):
    from paged_gqa_decode_step_gb300 import binding as b
    op = s["op"]
    if op == "tables":
        return b.rotary_tables(s["rotary"], s["length"], TYPES[s["dtype"]])
    if op == "rotary":
        b.rotary_apply(s["rotary"], s["q"], s["k"], s["positions"], s["q_out"], s["k_out"], s["ws"], inverse=s["inverse"])
        return s["q_out"], s["k_out"]
    if op == "update":
        b.pages_update(s["params"], s["cache"], s["table"], s["lengths"], s["refs"], s["parents"], s["new_lengths"],
                       s["ws"], table_out=s["table_out"], refs_out=s["refs_out"])
        return s["table_out"], s["refs_out"], s["pools"], s["scales"]
    if op == "compact":
        b.pages_compact(s["params"], s["cache"], s["table"], s["lengths"], s["refs"], s["map"], s["ws"],
                        table_out=s["table_out"], refs_out=s["refs_out"])
        return s["table_out"], s["refs_out"], s["map"], s["pools"], s["scales"]
    b.decode_shared(s["params"], s["q"], s["k_new"], s["v_new"], s["positions"], s["table"], s["group_start"],
                    s["group_pages"], s["k_pool"], s["v_pool"], s["out"], s["ws"])
    return s["out"], s["k_pool"], s["v_pool"]


def run(s):
    op = s["op"]
    if own:
        return _run_own(s)
    if op == "tables":
        at = torch.arange(s["length"], device="cuda")
        return tuple(torch.cat([t, t], -1).to(TYPES[s["dtype"]]) for t in _cos_sin(s, s["head_dim"], at))
    if op == "rotary":
        return _turned(s["q"], s), _turned(s["k"], s)
    if op == "update":
        table, refs, *copies = _update_plan(s)
        _copy_tails(s["pools"], *copies)
        if s["scales"] is not None:
            _copy_tails(s["scales"], *copies)
        return table, refs, s["pools"], s["scales"]
    if op == "compact":
        table, refs, to, high = _compact_plan(s)
        at = torch.nonzero(high)[:, 0]
        s["pools"][:, to[at].long()] = s["pools"][:, at]
        if s["scales"] is not None:
            s["scales"][:, to[at].long()] = s["scales"][:, at]
        return table, refs, to, s["pools"], s["scales"]
    return _decode(s), s["k_pool"], s["v_pool"]


def work(case):
    op = case["op"]
    e = {"bf16": 2, "f32": 4, "int8": 1}[case["dtype"]]
    if op == "tables":
        return {"bytes": 2 * case["length"] * case["head_dim"] * e, "flops": 20 * case["length"] * case["head_dim"]}
    if op == "rotary":
        vectors = case["tokens"] * (case["heads"] + case["kv_heads"])
        return {"bytes": 2 * vectors * case["head_dim"] * e + 4 * case["tokens"], "flops": 3 * vectors * case["rot"]}
    if op in ("update", "compact"):
        # a position's bytes in all pools
        each = case["pools"] * case["kv_heads"] * (case["head_dim"] * e + (4 if case["dtype"] == "int8" else 0))
        pages, width = _page_counts(case)
        state = 8 * (case["rows"] * width + pages)
        table, lengths, refs = _page_state(case, 1)
        if op == "update":
            parents, new = _asked(case)
            return {"bytes": state + 2 * each * sum(n for _, _, n in _after(table, lengths, refs, parents, new)[2]),
                    "flops": 0}
        n = sum(x > 0 for x in refs)
        return {"bytes": state + 4 * pages + 2 * each * PAGE * sum(x > 0 for x in refs[n:]), "flops": 0}
    sizes, prefixes, lengths = _groups(case)
    Hq, Hk, D, W = case["heads"], case["kv_heads"], case["head_dim"], case["window"]
    keys, seen, r = 0, 0, 0
    for size, p in zip(sizes, prefixes):
        first = p * PAGE
        for n in lengths[r:r + size]:
            total = p * PAGE + n
            lo = max(0, total - W) if W > 0 else 0
            seen += total - lo
            keys += min(n, total - lo)
            first = min(first, lo)
        keys += p * PAGE - first
        r += size
    table = 2 * D * e if case["theta"] > 0 else 0
    return {"bytes": keys * 2 * Hk * D * e + case["rows"] * (2 * Hq * D * e + 4 * Hk * D * e + table),
            "flops": 4 * Hq * D * seen}


def _after(table, lengths, refs, parents, new):
    """The new table, counts and tail copies (from, to, positions), row after row from the rules."""
    held = [0] * len(refs)
    for row, n in zip(table, lengths):
        for x in row[:_pages(n)]:
            held[x] += 1
    count = [a - b for a, b in zip(refs, held)]      # holders that are no row
    rows, writers = [], {}
    for r, (p, n) in enumerate(zip(parents, new)):
        keep = min(lengths[p], n) if p >= 0 else 0
        mine = list(table[p][:keep // PAGE]) if p >= 0 else []
        if keep % PAGE and n == keep:
            mine.append(table[p][keep // PAGE])
        elif keep % PAGE:
            writers.setdefault(table[p][keep // PAGE], []).append(r)
        for x in mine:
            count[x] += 1
        rows.append(mine)
    copies = {}
    for x, who in writers.items():
        if count[x] == 0:
            rows[who[0]].append(x)
            count[x] = 1
            who = who[1:]
        for r in who:
            copies[r] = x
    free = iter([x for x, c in enumerate(count) if c == 0])
    made = []
    for r, (mine, n) in enumerate(zip(rows, new)):
        while len(mine) < _pages(n):
            x = next(free)
            if r in copies:
                made.append((copies.pop(r), x, lengths[parents[r]] % PAGE))
            count[x] = 1
            mine.append(x)
    return [mine + [-1] * (len(old) - len(mine)) for mine, old in zip(rows, table)], count, made


def _exact_pages(case, seed, s):
    table, lengths, refs = (s[n].tolist() for n in ("table", "lengths", "refs"))
    pools, scales = s["pools"], s["scales"]

    def moved(src, dst, n):
        pools[:, dst, :, :n] = pools[:, src, :, :n].clone()
        if scales is not None:
            scales[:, dst, :, :n] = scales[:, src, :, :n].clone()

    if case["op"] == "update":
        table, refs, made = _after(table, lengths, refs, s["parents"].tolist(), s["new_lengths"].tolist())
        for src, dst, n in made:
            moved(src, dst, n)
        found = [table, refs]
    else:
        n = sum(c > 0 for c in refs)
        to = [x if c > 0 else -1 for x, c in enumerate(refs)]
        holes = iter([x for x in range(n) if refs[x] == 0])
        for x in range(n, len(refs)):
            if refs[x] > 0:
                to[x] = next(holes)
                refs[to[x]], refs[x] = refs[x], 0
                moved(x, to[x], PAGE)
        table = [[to[x] if i < _pages(k) else x for i, x in enumerate(row)] for row, k in zip(table, lengths)]
        found = [table, refs, to]
    return tuple(torch.tensor(x, dtype=torch.int32, device="cuda") for x in found) + (
        pools if case["dtype"] == "int8" else pools.double(), None if scales is None else scales.double())


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, D, F = case["op"], case["head_dim"], torch.float64
    if op in ("update", "compact"):
        return _exact_pages(case, seed, s)
    if op in ("tables", "rotary"):
        rot = case.get("rot", D)
        f, gain = [], 1.0
        for i in range(rot // 2):
            w = s["theta"] ** (-2.0 * i / rot)
            if case["scaling"] == "linear":
                w /= case["factor"]
            elif case["scaling"] == "wavelength":
                length = 2 * math.pi / w
                if length > case["original"] / case["low"]:
                    w /= case["factor"]
                elif length >= case["original"] / case["high"]:
                    mix = (case["original"] / length - case["low"]) / (case["high"] - case["low"])
                    w = (1 - mix) * w / case["factor"] + mix * w
            elif case["scaling"] == "ramp":
                a, b = (rot * math.log(case["original"] / (t * 2 * math.pi)) / (2 * math.log(s["theta"]))
                        for t in (case["high"], case["low"]))
                mix = min(1.0, max(0.0, (i - a) / max(b - a, 1e-3)))
                w = w * (1 - mix) + w / case["factor"] * mix
                gain = 0.1 * math.log(case["factor"]) + 1.0
            f.append(w)
        at = torch.arange(case["length"], device="cuda") if op == "tables" else s["positions"]
        turn = torch.polar(torch.tensor(gain, dtype=F, device="cuda"),
                           at.to(F)[:, None] * torch.tensor(f, dtype=F, device="cuda"))
        if op == "tables":
            return turn.real.repeat(1, 2), turn.imag.repeat(1, 2)
        if case["inverse"]:
            turn = turn.conj()

        def turned(x):
            x = x.to(F)
            y = x.clone()
            pairs = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
            z = torch.complex(x[..., pairs[0]], x[..., pairs[1]]) * turn[:, None]
            y[..., pairs[0]], y[..., pairs[1]] = z.real, z.imag
            return y

        return turned(s["q"]), turned(s["k"])
    T, Hk, W = TYPES[case["dtype"]], case["kv_heads"], case["window"]

    def rotated(x):
        x = x.to(F)
        if s["cos"] is None:
            return x
        c, sn = (s[n][s["positions"].long()].to(F)[:, None] for n in ("cos", "sin"))
        a, b = x.split(D // 2, -1)
        return torch.cat([a * c[..., :D // 2] - b * sn[..., :D // 2], b * c[..., D // 2:] + a * sn[..., D // 2:]], -1)

    table, positions = s["table"].long(), s["positions"].tolist()
    # what the cache holds is rounded to its type, and so are the rotated queries that meet it
    k_new, q = rotated(s["k_new"]).float().to(T), rotated(s["q"]).float().to(T).to(F)
    out = torch.empty(s["q"].shape, dtype=F, device="cuda")
    for r, pos in enumerate(positions):
        s["k_pool"][table[r, pos // PAGE], :, pos % PAGE] = k_new[r]
        s["v_pool"][table[r, pos // PAGE], :, pos % PAGE] = s["v_new"][r]
    for r, pos in enumerate(positions):
        t = torch.arange(max(0, pos - W + 1) if W > 0 else 0, pos + 1, device="cuda")
        k, v = (s[n][table[r, t // PAGE], :, t % PAGE].to(F) for n in ("k_pool", "v_pool"))     # [t, Hk, D]
        score = torch.einsum("hgd,thd->hgt", q[r].view(Hk, -1, D), k) / math.sqrt(D)
        norm = torch.logsumexp(score, -1, keepdim=True)
        if s["sink"] is not None:
            norm = torch.logaddexp(norm, s["sink"].to(F).view(Hk, -1, 1))
        out[r] = torch.einsum("hgt,thd->hgd", torch.exp(score - norm), v).reshape(-1, D)
    return out, s["k_pool"].double(), s["v_pool"].double()
