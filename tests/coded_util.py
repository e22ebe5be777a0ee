"""Plain references for the coded (8-bit) cache, on the CPU, and the bounds the GPU results are held to.

The codes and scales are the formula's f32 operations one by one, so the GPU's must equal them bit for bit.  The
attention is computed in 64 bits from what the codes stand for; `bound` is how far an output may be from it, by the
roundings the kernels make (a rounding to a type is off by at most eps / 2 of the value):

  scores   q is held in f16 (f32 inputs: in two f16 parts), prefill holds code * ratio of K in f16 and the ratio too;
           every product sum is f32.  With S = sum_d |q_d k_d| scale the score is off by at most ds = u S + small.
  weights  e^s is off by e^ds - 1, the normalised weight by twice that; the weight times the V scale is f16 (f32:
           two parts), prefill's V ratio and code * ratio too: dw.
  output   |out| eps(T) / 2 + A (2 (e^ds - 1) + dw), A = sum_t w_t |v_t| over the normalised weights.
"""
import math

import torch

F16, QMAX = 2.0 ** -11, {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
TINY = 2.0 ** -126


def rope(x, cos, sin, positions):
    """x [n, heads, D] f32, rotated with separate f32 products and one add."""
    if cos is None:
        return x
    c, s = cos[positions.long()].float()[:, None], sin[positions.long()].float()[:, None]
    h = x.shape[-1] // 2
    return x * c + torch.cat([-x[..., h:], x[..., :h]], -1) * s


def code(x, kind):
    """Codes (as kind) and scales of the last dimension of x f32."""
    amax = x.abs().amax(-1, keepdim=True)
    fine = torch.isfinite(x).all(-1, keepdim=True)
    scale = torch.clamp(amax / torch.full_like(amax, QMAX[kind]), min=TINY)
    y = torch.where(fine, x, torch.zeros_like(x)) / torch.where(fine, scale, torch.ones_like(scale))
    if kind == torch.int8:
        codes = torch.round(y).clamp(-127, 127).to(torch.int8)
    else:
        codes = y.clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes, torch.where(fine, scale, torch.full_like(scale, math.nan)).squeeze(-1)


class Cache:
    """A coded cache on the CPU: codes as bytes [pages, kv_heads, 64, D] and scales."""

    def __init__(self, pages, kv_heads, D, kind, gen=None):
        self.kind = kind
        shape = (pages, kv_heads, 64, D)
        if gen is None:
            self.k, self.v = (torch.zeros(shape, dtype=torch.uint8) for _ in range(2))
            self.ks, self.vs = (torch.zeros(shape[:3]) for _ in range(2))
        else:
            (self.k, self.ks), (self.v, self.vs) = (
                (c.view(torch.uint8), s) for c, s in (code(torch.randn(shape, generator=gen), kind) for _ in range(2)))

    def gpu(self):
        return [self.k.cuda().view(self.kind), self.v.cuda().view(self.kind), self.ks.cuda(), self.vs.cuda()]

    def write(self, k, v, slots):
        """k (rotated), v [n, kv_heads, D] f32 at pool slots."""
        page, off = slots.long() // 64, slots.long() % 64
        for x, codes, scales in ((k, self.k, self.ks), (v, self.v, self.vs)):
            c, s = code(x, self.kind)
            codes[page, :, off] = c.view(torch.uint8)
            scales[page, :, off] = s

    def meant(self, codes, scales, slots, dtype=torch.float64):
        page, off = slots.long() // 64, slots.long() % 64
        return codes[page, :, off].view(self.kind).to(dtype) * scales[page, :, off].to(dtype)[..., None]

    def same(self, tensors):
        for mine, theirs in zip((self.k, self.v), tensors[:2]):
            assert torch.equal(mine, theirs.cpu().view(torch.uint8)), "codes differ"
        for mine, theirs in zip((self.ks, self.vs), tensors[2:]):
            assert torch.equal(mine.view(torch.int32), theirs.cpu().view(torch.int32)), "scales differ"


def attend(cache, q, positions, rows, table, window=0, sinks=None, scale=None, kind="decode", f32=False):
    """Outputs [n, heads, D] in 64 bits and their bounds.  q: rotated, f32."""
    n, Hq, D = q.shape
    Hk = cache.k.shape[1]
    scale = scale or 1.0 / math.sqrt(D)
    out, bound = torch.zeros(n, Hq, D, dtype=torch.float64), torch.zeros(n, Hq, D, dtype=torch.float64)
    uq = 2.0 ** -22 if f32 else F16
    uk = 2 * F16 if kind == "prefill" else 0.0
    uv = uk + uq
    for i in range(n):
        pos = int(positions[i])
        lo = max(0, pos - window + 1) if window > 0 else 0
        t = torch.arange(lo, pos + 1)
        slots = table[int(rows[i])].long()[t // 64] * 64 + t % 64
        k, v = cache.meant(cache.k, cache.ks, slots), cache.meant(cache.v, cache.vs, slots)   # [t, Hk, D]
        qi = q[i].double().view(Hk, Hq // Hk, D)
        s = torch.einsum("hgd,thd->hgt", qi, k) * scale
        S = torch.einsum("hgd,thd->hgt", qi.abs(), k.abs()) * scale
        # f32 sums of D products and of the exponent's argument, the f16 floor of small elements
        ds = (uq + uk) * S + (D + 8) * 2.0 ** -24 * S + 2.0 ** -22 * (s.abs() + 1) + 2.0 ** -23 * S.amax(-1, keepdim=True)
        top = s.amax(-1, keepdim=True)
        if sinks is not None:
            sk = sinks.double().view(Hk, -1, 1)
            top = torch.maximum(top, sk)
        w = torch.exp(s - top)
        total = w.sum(-1, keepdim=True)
        if sinks is not None:
            total = total + torch.exp(sk - top)
        w = w / total
        o = torch.einsum("hgt,thd->hgd", w, v)
        a = torch.einsum("hgt,thd->hgd", w, v.abs())
        most = torch.expm1(ds.amax(-1, keepdim=True))
        small = len(t) * 2.0 ** -33 * v.abs().amax(0)[:, None]        # weights under f16's normal range
        out[i] = o.reshape(Hq, D)
        b = a * (2 * most + uv + (len(t) + 8) * 2.0 ** -24) + small
        bound[i] = (b + o.abs() * (2.0 ** -24 if f32 else 2.0 ** -8)).reshape(Hq, D)
    return out, bound


def hold(got, want, bound, what=""):
    got = got.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    fine = ~torch.isnan(want)
    err = (got - want).abs()[fine]
    over = err > bound[fine]
    assert not over.any(), f"{what}: off by {err[over].max():.3g} where {bound[fine][over].max():.3g} is allowed"
    return err


class Case:
    """Rows with cached prefixes and new tokens: inputs on the CPU, a cache, a table of shuffled pages."""

    def __init__(self, heads, kv_heads, D, prefix, chunk, dtype=torch.bfloat16, kind=torch.float8_e4m3fn, theta=10000.0,
                 window=0, sinks=False, seed=0, order=None):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.kv_heads, self.D, self.dtype, self.kind, self.window = heads, kv_heads, D, dtype, kind, window
        self.n_rows, n = len(prefix), sum(chunk)
        need = [(a + b + 63) // 64 for a, b in zip(prefix, chunk)]
        self.width = max(max(need), 1) + 1
        self.pages = sum(need) + 2
        ids = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((self.n_rows, self.width), -1, dtype=torch.int32)
        used = 0
        for r, k in enumerate(need):
            self.table[r, :k] = ids[used:used + k]
            used += k
        self.rows = torch.tensor([r for r, b in enumerate(chunk) for _ in range(b)], dtype=torch.int32)
        self.positions = torch.tensor([a + i for a, b in zip(prefix, chunk) for i in range(b)], dtype=torch.int32)
        if order is not None:
            at = torch.randperm(n, generator=g) if order == "mixed" else torch.arange(n - 1, -1, -1)
            self.rows, self.positions = self.rows[at], self.positions[at]
        self.slots = (self.table[self.rows.long(), self.positions.long() // 64] * 64 + self.positions % 64).to(torch.int32)
        self.q = torch.randn(n, heads, D, generator=g).to(dtype)
        self.k_new = torch.randn(n, kv_heads, D, generator=g).to(dtype)
        self.v_new = torch.randn(n, kv_heads, D, generator=g).to(dtype)
        self.sinks = torch.randn(heads, generator=g).to(dtype) if sinks else None
        self.cos = self.sin = None
        if theta > 0:
            f = torch.exp(-torch.arange(D // 2, dtype=torch.float64) * 2 / D * math.log(theta))
            ang = torch.arange(self.width * 64, dtype=torch.float64)[:, None] * torch.cat([f, f])
            self.cos, self.sin = torch.cos(ang).to(dtype), torch.sin(ang).to(dtype)
        self.cache = Cache(self.pages, kv_heads, D, kind, g)

    def params(self, b, **kw):
        gpu = lambda t: None if t is None else t.cuda()   # noqa: E731
        kw.setdefault("sinks", gpu(self.sinks))
        return b.make_params(self.n_rows, self.heads, self.kv_heads, self.D, self.width, self.pages, self.dtype,
                             window=self.window, rope_cos=gpu(self.cos), rope_sin=gpu(self.sin), **kw)

    def write(self):
        """The reference cache after the new tokens are written."""
        self.cache.write(rope(self.k_new.float(), self.cos, self.sin, self.positions), self.v_new.float(), self.slots)

    def want(self, kind):
        return attend(self.cache, rope(self.q.float(), self.cos, self.sin, self.positions), self.positions, self.rows,
                      self.table, self.window, self.sinks, kind=kind, f32=self.dtype == torch.float32)
