"""Cases of the operators of the 8-bit paged KV cache: writing, reading back, decoding and prefilling over it.

A coded cache holds, for every token and kv head, the D codes of its key and of its value (e4m3 or int8) and one
f32 scale each: scale = max(max|x| / qmax, 2^-126), code = round-to-nearest-even(x / scale), qmax = 448 or 127, and a
code stands for code * scale.  Keys are rotated (RoPE) in f32 and coded from the f32 value.

  write    codes of n new tokens put at their pool slots
  read     codes of n slots turned back into T
  decode   one new token per row: rotate q and k, code and write k and v, attend positions (pos - window, pos]
  prefill  a chunk of new tokens per row, the same over each token's own positions

`run` computes them in elementary torch operations in f32, or, where `own` is true, by the framework's calls.
"""
import math
import random

import torch

own = False

PAGE = 64
TINY_SCALE = 2.0 ** -126
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
QMAX = {"e4m3": 448.0, "int8": 127.0}
LLAMA = dict(heads=32, kv_heads=8, head_dim=128, dtype="bf16", theta=500000.0)
GPTOSS = dict(heads=64, kv_heads=8, head_dim=64, dtype="bf16", theta=150000.0)
GPT2 = dict(heads=12, kv_heads=12, head_dim=64, dtype="f32", theta=0.0)


def listed():
    return [
        # one decode step's new tokens in a cache of their own: latency alone
        dict(name="write_step", op="write", tokens=37, code="int8", **GPT2),
        # a prompt batch of the Llama shape
        dict(name="write_prompt", op="write", tokens=8192, code="e4m3", **LLAMA),
        # a short reused prefix in f32
        dict(name="read_short", op="read", tokens=257, code="int8", **GPT2),
        # many prefixes copied out of the cache (to another worker, or to a bf16 cache)
        dict(name="read_prefixes", op="read", tokens=65536, code="e4m3", **LLAMA),
        # a single user's next token
        dict(name="decode_single", op="decode", rows=1, ctx_lo=777, ctx_hi=777, spread="lin", window=0, sinks=False,
             code="e4m3", **LLAMA),
        # a small batch of long contexts
        dict(name="decode_layer", op="decode", rows=32, ctx_lo=1025, ctx_hi=8192, spread="lin", window=0, sinks=False,
             code="e4m3", **LLAMA),
        # a serving batch: mostly short contexts, a few long ones
        dict(name="decode_serving", op="decode", rows=256, ctx_lo=16, ctx_hi=8192, spread="log", window=0, sinks=False,
             code="e4m3", **LLAMA),
        # the full-attention layer of a pair with sinks, int8
        dict(name="decode_sinks", op="decode", rows=64, ctx_lo=257, ctx_hi=4096, spread="lin", window=0, sinks=True,
             code="int8", **GPTOSS),
        # multi-head attention in f32
        dict(name="decode_f32", op="decode", rows=128, ctx_lo=2, ctx_hi=1024, spread="lin", window=0, sinks=False,
             code="int8", **GPT2),
        # a few drafted tokens per row checked at once
        dict(name="prefill_drafts", op="prefill", rows=32, chunk_lo=1, chunk_hi=8, prefix_lo=500, prefix_hi=8000,
             window=0, sinks=False, code="e4m3", **LLAMA),
        # prompt chunks over the prefixes that earlier chunks left
        dict(name="prefill_chunks", op="prefill", rows=8, chunk_lo=1024, chunk_hi=1024, prefix_lo=0, prefix_hi=7168,
             window=0, sinks=False, code="e4m3", **LLAMA),
        # ragged prompts through a sliding-window layer with sinks, int8
        dict(name="prefill_sliding", op="prefill", rows=11, chunk_lo=3, chunk_hi=901, prefix_lo=0, prefix_hi=2500,
             window=128, sinks=True, code="int8", **GPTOSS),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "prefill", "prefill"])
    kv_heads = rng.choice([1, 2, 4, 8, 12])
    heads = kv_heads * (1 if kv_heads == 12 else rng.choice([1, 2, 3, 4, 5, 8]))
    c = dict(op=op, code=rng.choice(["e4m3", "int8"]), heads=heads, kv_heads=kv_heads, head_dim=rng.choice([64, 128]),
             dtype="bf16" if op == "prefill" else rng.choice(["bf16", "bf16", "f32"]),
             theta=rng.choice([0.0, 10000.0, 500000.0]))
    if op == "write":
        return dict(c, tokens=_log_int(rng, 1, 8192))
    if op == "read":
        return dict(c, tokens=_log_int(rng, 1, 32768))
    c.update(window=rng.choice([0, 0, 0, _log_int(rng, 1, 2000)]), sinks=rng.random() < 0.3)
    if op == "decode":
        rows = _log_int(rng, 1, 256)
        hi = _log_int(rng, 1, min(8192, 400000 // rows))
        return dict(c, rows=rows, ctx_lo=rng.randint(1, hi), ctx_hi=hi, spread=rng.choice(["lin", "log"]))
    rows = _log_int(rng, 1, 40)
    chunk_hi = _log_int(rng, 1, 1024)
    rows = max(1, min(rows, 8192 // chunk_hi))
    prefix_hi = rng.choice([0, _log_int(rng, 1, 7000)])
    return dict(c, rows=rows, chunk_lo=rng.randint(1, chunk_hi), chunk_hi=chunk_hi, prefix_lo=rng.randint(0, prefix_hi),
                prefix_hi=prefix_hi)


def _spaced(lo, hi, n, spread):
    """n whole numbers over [lo, hi], the ends among them where n > 1."""
    at = [i / (n - 1) if n > 1 else 1.0 for i in range(n)]
    if spread == "log":
        return [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * u))) for u in at]
    return [int(round(lo + (hi - lo) * u)) for u in at]


def _lengths(case):
    """(prefix, new tokens) of every row, from the case alone."""
    if case["op"] == "decode":
        return [(c - 1, 1) for c in _spaced(case["ctx_lo"], case["ctx_hi"], case["rows"], case["spread"])]
    chunks = _spaced(case["chunk_lo"], case["chunk_hi"], case["rows"], "lin")
    prefixes = _spaced(case["prefix_lo"], case["prefix_hi"], case["rows"], "lin")
    random.Random(case["rows"]).shuffle(prefixes)
    return list(zip(prefixes, chunks))


def _coded(x, code):
    """Codes and scales of the last dimension of x, in f32."""
    amax = x.abs().amax(-1, keepdim=True)
    scale = torch.clamp(amax / torch.full_like(amax, QMAX[code]), min=TINY_SCALE)
    y = x / scale
    if code == "int8":
        return torch.round(y).clamp(-127, 127).to(torch.int8), scale.squeeze(-1)
    return y.clamp(-448, 448).to(torch.float8_e4m3fn), scale.squeeze(-1)


def _random_pool(case, pages, g, spread):
    """A pool of codes and scales as a cache holds them: some channels and tokens larger than others."""
    Hk, D = case["kv_heads"], case["head_dim"]
    codes = torch.empty(pages, Hk, PAGE, D, dtype=CODES[case["code"]], device="cuda")
    scales = torch.empty(pages, Hk, PAGE, dtype=torch.float32, device="cuda")
    gain = torch.exp(spread * torch.randn(Hk, 1, D, generator=g, device="cuda"))
    for p in range(0, pages, 1024):
        n = min(1024, pages - p)
        x = torch.randn(n, Hk, PAGE, D, generator=g, device="cuda") * gain
        x *= torch.exp(0.3 * torch.randn(n, Hk, PAGE, 1, generator=g, device="cuda"))
        codes[p:p + n], scales[p:p + n] = _coded(x, case["code"])
    return codes, scales


def _tables(case, length):
    """Rotary cos and sin [length, D] in T, or None without rotation."""
    if case["theta"] <= 0:
        return None, None
    D, T = case["head_dim"], TYPES[case["dtype"]]
    freq = torch.exp(-torch.arange(D // 2, device="cuda", dtype=torch.float64) * 2 / D * math.log(case["theta"]))
    angle = torch.arange(length, device="cuda", dtype=torch.float64)[:, None] * freq
    angle = torch.cat([angle, angle], -1)
    return torch.cos(angle).to(T), torch.sin(angle).to(T)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, T = case["op"], TYPES[case["dtype"]]
    Hq, Hk, D = case["heads"], case["kv_heads"], case["head_dim"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(T)

    s = dict(case)
    if op in ("write", "read"):
        n = case["tokens"]
        need = (n + 5 + PAGE - 1) // PAGE + 1
        pages = need + 2 + need // 10
        at = torch.arange(n, device="cuda") + int(torch.randint(0, PAGE, (1,), generator=g, device="cuda"))
        ids = torch.randperm(pages, generator=g, device="cuda")
        s["slots"] = (ids[at // PAGE] * PAGE + at % PAGE).to(torch.int32)
        s["positions"] = torch.randint(0, 8192, (n,), generator=g, device="cuda").to(torch.int32)
        length, width, rows = 8192, 128, 1
        if op == "read":
            s["k_out"], s["v_out"] = torch.empty(n, Hk, D, dtype=T, device="cuda"), torch.empty(n, Hk, D, dtype=T, device="cuda")
    else:
        lengths = _lengths(case)
        order = torch.randperm(len(lengths), generator=g, device="cuda").tolist()
        lengths = [lengths[i] for i in order]
        rows = len(lengths)
        length = max(a + b for a, b in lengths)
        width = (length + PAGE - 1) // PAGE
        need = [(a + b + PAGE - 1) // PAGE for a, b in lengths]
        pages = sum(need) + 1 + sum(need) // 10
        ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).tolist()
        table, used = [], 0
        for k in need:
            table.append(ids[used:used + k] + [-1] * (width - k))
            used += k
        s["table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
        n = sum(b for _, b in lengths)
        s["positions"] = torch.tensor([a + i for a, b in lengths for i in range(b)], dtype=torch.int32, device="cuda")
        s["rows"] = torch.tensor([r for r, (_, b) in enumerate(lengths) for _ in range(b)], dtype=torch.int32, device="cuda")
        s["place"] = torch.tensor([i for _, b in lengths for i in range(b)], dtype=torch.int64, device="cuda")
        s["most"] = max(b for _, b in lengths)
        s["slots"] = (s["table"][s["rows"].long(), s["positions"].long() // PAGE] * PAGE + s["positions"] % PAGE).to(torch.int32)
        s["q"] = normal(n, Hq, D)
        s["out"] = torch.empty_like(s["q"])
        s["sink"] = normal(Hq) if case["sinks"] else None
    if op != "read":
        s["k_new"], s["v_new"] = normal(n, Hk, D), normal(n, Hk, D)
    s["n_rows"] = rows
    s["cos"], s["sin"] = _tables(case, length)
    s["k"], s["ks"] = _random_pool(case, pages, g, 0.5)
    s["v"], s["vs"] = _random_pool(case, pages, g, 0.0)
    if own:
        from paged_gqa_decode_step_gb300 import binding as b
        p = b.make_params(rows, Hq, Hk, D, width, pages, T, window=case.get("window", 0), rope_cos=s["cos"],
                          rope_sin=s["sin"], sinks=s.get("sink"))
        s["params"], s["cache"] = p, b.make_coded_cache(p, s["k"], s["v"], s["ks"], s["vs"])
        s["ws"] = b.new_coded_workspace(p, n)
    return s


def _rope(x, s):
    """x [n, heads, D] rotated at the tokens' positions, in f32."""
    x = x.float()
    if s["cos"] is None:
        return x
    at = s["positions"].long()
    c, sn = s["cos"][at].float().unsqueeze(1), s["sin"][at].float().unsqueeze(1)
    half = x.shape[-1] // 2
    return x * c + torch.cat([-x[..., half:], x[..., :half]], -1) * sn


def _put(pool, scales, x, s):
    """Codes of x [n, kv_heads, D] at the tokens' slots."""
    codes, scale = _coded(x, s["code"])
    page, off = s["slots"].long() // PAGE, s["slots"].long() % PAGE
    pool.view(torch.uint8)[page, :, off] = codes.view(torch.uint8)
    scales[page, :, off] = scale


def _write(s):
    _put(s["k"], s["ks"], _rope(s["k_new"], s), s)
    _put(s["v"], s["vs"], s["v_new"].float(), s)


def _values(pool, scales, page, off, s):
    codes = pool.view(torch.uint8)[page, :, off].view(CODES[s["code"]])
    return codes.float() * scales[page, :, off].unsqueeze(-1)


def _row_values(pool, scales, s):
    """[rows, kv_heads, positions, D] of every row's pages in f32 (page 0 stands for an absent one)."""
    at = s["table"].long().clamp(min=0)
    x = pool.view(torch.uint8)[at].view(CODES[s["code"]]).float() * scales[at].unsqueeze(-1)
    R, P, Hk, _, D = x.shape
    return x.transpose(1, 2).reshape(R, Hk, P * PAGE, D)


def _attend(s):
    """Every new token over its row's positions [pos - window + 1, pos]: tokens padded to [rows, most]."""
    Hq, Hk, D, R, L = s["heads"], s["kv_heads"], s["head_dim"], s["n_rows"], s["most"]
    row, place = s["rows"].long(), s["place"]
    q = torch.zeros(R, L, Hq, D, device="cuda")
    q[row, place] = _rope(s["q"], s)
    pos = torch.zeros(R, L, dtype=torch.int64, device="cuda")
    pos[row, place] = s["positions"].long()
    keys, values = _row_values(s["k"], s["ks"], s), _row_values(s["v"], s["vs"], s)
    # [rows, kv heads, group * tokens, positions]
    q = q.view(R, L, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4).reshape(R, Hk, -1, D)
    score = (q @ keys.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    t = torch.arange(keys.shape[2], device="cuda")
    seen = t <= pos[..., None]
    if s["window"] > 0:
        seen &= t > pos[..., None] - s["window"]
    seen = seen[:, None, None].expand(R, Hk, Hq // Hk, L, -1).reshape(R, Hk, -1, t.numel())
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    sink = None
    if s["sink"] is not None:
        sink = s["sink"].float().view(Hk, -1, 1).expand(Hk, Hq // Hk, L).reshape(1, Hk, -1, 1)
        top = torch.maximum(top, sink)
    w = torch.exp(score - top)
    total = w.sum(-1, keepdim=True)
    if sink is not None:
        total = total + torch.exp(sink - top)
    out = ((w @ values) / total).view(R, Hk, Hq // Hk, L, D).permute(0, 3, 1, 2, 4).reshape(R, L, Hq, D)
    return out[row, place].to(TYPES[s["dtype"]])


def run(s):
    op = s["op"]
    if own:
        from paged_gqa_decode_step_gb300 import binding as b
        if op == "write":
            b.coded_write(s["params"], s["cache"], s["k_new"], s["v_new"], s["positions"], s["slots"], s["ws"])
        elif op == "read":
            b.coded_read(s["params"], s["cache"], s["slots"], s["k_out"], s["v_out"], s["ws"])
            return s["k_out"], s["v_out"]
        elif op == "decode":
            b.coded_decode(s["params"], s["cache"], s["q"], s["k_new"], s["v_new"], s["positions"], s["table"],
                           s["out"], s["ws"])
        else:
            b.coded_prefill(s["params"], s["cache"], s["q"], s["k_new"], s["v_new"], s["positions"], s["rows"],
                            s["slots"], s["table"], s["out"], s["ws"])
        state = (s["k"], s["v"], s["ks"], s["vs"])
        return state if op == "write" else (s["out"],) + state
    if op == "read":
        page, off, T = s["slots"].long() // PAGE, s["slots"].long() % PAGE, TYPES[s["dtype"]]
        return _values(s["k"], s["ks"], page, off, s).to(T), _values(s["v"], s["vs"], page, off, s).to(T)
    _write(s)
    state = (s["k"], s["v"], s["ks"], s["vs"])
    return state if op == "write" else (_attend(s),) + state


def work(case):
    Hq, Hk, D = case["heads"], case["kv_heads"], case["head_dim"]
    e = 2 if case["dtype"] == "bf16" else 4
    coded = 2 * Hk * (D + 4)   # a token's codes and scales, keys and values
    if case["op"] in ("write", "read"):
        n = case["tokens"]
        table = 2 * D * e if case["op"] == "write" and case["theta"] > 0 else 0
        return {"bytes": n * (2 * Hk * D * e + coded + table + (8 if case["op"] == "write" else 4)), "flops": n * Hk * D * 8}
    W, tokens, seen, keys = case["window"], 0, 0, 0
    for a, b in _lengths(case):
        tokens += b
        first = max(0, a - W + 1) if W > 0 else 0
        keys += a + b - first
        for i in range(b):
            seen += min(a + i + 1, W) if W > 0 else a + i + 1
    table = 2 * D * e if case["theta"] > 0 else 0
    moved = keys * coded + tokens * (2 * Hq * D * e + 2 * Hk * D * e + coded + table + 16)
    return {"bytes": moved, "flops": 4 * Hq * D * seen}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, D, F = case["op"], case["head_dim"], torch.float64
    slots = s["slots"].long()
    flat = {n: s[n].view(torch.uint8).transpose(1, 2).reshape(-1, case["kv_heads"], D) for n in "kv"}
    sflat = {n: s[n + "s"].transpose(1, 2).reshape(-1, case["kv_heads"]) for n in "kv"}

    def meant(n, at):
        return flat[n][at].view(CODES[case["code"]]).to(F) * sflat[n][at].to(F)[..., None]

    if op == "read":
        return meant("k", slots), meant("v", slots)

    def turned(x):
        x = x.to(F)
        if case["theta"] <= 0:
            return x
        c, sn = (s[n][s["positions"].long()].to(F)[:, None] for n in ("cos", "sin"))
        a, b = x.split(D // 2, -1)
        return torch.cat([a * c[..., :D // 2] - b * sn[..., :D // 2], b * c[..., D // 2:] + a * sn[..., D // 2:]], -1)

    for n, x in (("k", turned(s["k_new"])), ("v", s["v_new"].to(F))):
        scale = (x.abs().max(-1).values / QMAX[case["code"]]).clamp(min=TINY_SCALE)
        y = x / scale[..., None]
        y = torch.round(y).to(torch.int8) if case["code"] == "int8" else y.to(torch.float8_e4m3fn)
        flat[n][slots] = y.view(torch.uint8)
        sflat[n][slots] = scale.float()
    Hk, pages = case["kv_heads"], s["k"].shape[0]
    pools = [flat[n].view(pages, PAGE, Hk, D).transpose(1, 2).contiguous().view(CODES[case["code"]]) for n in "kv"]
    state = tuple(pools) + tuple(sflat[n].view(pages, PAGE, Hk).transpose(1, 2).contiguous().to(F) for n in "kv")
    if op == "write":
        return state
    q, out = turned(s["q"]), torch.empty(s["q"].shape, dtype=F, device="cuda")
    positions, rows, table = s["positions"].tolist(), s["rows"].tolist(), s["table"].long()
    at = 0
    while at < len(rows):
        end = at
        while end < len(rows) and rows[end] == rows[at] and end - at < 512:
            end += 1
        t = torch.arange(positions[end - 1] + 1, device="cuda")
        where = table[rows[at], t // PAGE] * PAGE + t % PAGE
        k, v = meant("k", where), meant("v", where)
        qq = q[at:end].view(end - at, Hk, -1, D)
        sc = torch.einsum("nhgd,thd->hgnt", qq, k) / math.sqrt(D)
        pos = s["positions"][at:end].long()[:, None]
        hide = t > pos
        if case["window"] > 0:
            hide |= t <= pos - case["window"]
        sc.masked_fill_(hide, -math.inf)
        norm = torch.logsumexp(sc, -1)
        if s["sink"] is not None:
            norm = torch.logaddexp(norm, s["sink"].to(F).view(Hk, -1, 1).expand_as(norm))
        out[at:end] = torch.einsum("hgnt,thd->nhgd", torch.exp(sc - norm[..., None]), v).reshape(end - at, -1, D)
        at = end
    return (out,) + state
