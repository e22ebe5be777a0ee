"""Rotary positions on the GPU against the same angles in 64 bits.

An angle is pos * turns / 2^64 turns exactly (integers).  The kernels take its place in a quarter turn as an f32 of at
most an eighth of a turn (off by 2^-24 of pi / 4, and by 2^-32 turns cut off), cos and sin by sincospif (2 units in the
last place of 1 at most: 2^-23) and one product with the gain: cos and sin are off by 4.7e-8 + 1.5e-9 + 1.2e-7 + 6e-8
< 2^-22 of the gain.  The two products and their sum round three times more, to 2^-24 of |x0| + |x1| each.
"""
import math

import pytest
import torch

from gpu_util import binding

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF16, F32 = torch.bfloat16, torch.float32
TRIG = 2.0 ** -22
SPECS = {
    "none": dict(),
    "linear": dict(scaling="linear", factor=4.0),
    "wavelength": dict(scaling="wavelength", factor=8.0, low=1.0, high=4.0, original_len=8192),
    "ramp": dict(scaling="ramp", factor=32.0, low=1.0, high=32.0, original_len=4096),
}


def half_rounding(dtype):
    return torch.finfo(dtype).eps / 2


def cos_sin(rot, positions):
    """cos and sin [n, rot / 2] times the gain in 64 bits, from the frequencies' integers."""
    turns = [int(t) for t in rot.turns[:rot.rot_dim // 2]]
    angle = [[((p * t) % 2 ** 64) / 2.0 ** 64 * 2 * math.pi for t in turns] for p in positions.tolist()]
    angle = torch.tensor(angle, dtype=torch.float64).view(len(positions), len(turns))
    return torch.cos(angle) * rot.gain, torch.sin(angle) * rot.gain


def turned(rot, x, positions, inverse):
    """(x turned, in 64 bits; the bound on what f32 arithmetic may be off, without the last rounding)."""
    x = x.detach().cpu().double()
    c, s = (t[:, None] for t in cos_sin(rot, positions.cpu()))
    if inverse:
        s = -s
    d, y, bound = rot.rot_dim, x.clone(), torch.zeros_like(x)
    i = (slice(0, d, 2), slice(1, d, 2)) if rot.interleaved else (slice(0, d // 2), slice(d // 2, d))
    a, b = x[..., i[0]], x[..., i[1]]
    y[..., i[0]], y[..., i[1]] = a * c - b * s, b * c + a * s
    bound[..., i[0]] = bound[..., i[1]] = (a.abs() + b.abs()) * rot.gain * (TRIG + 3 * 2.0 ** -24)
    return y, bound


def hold(got, want, bound, dtype):
    err = (got.detach().cpu().double() - want).abs()
    assert (err <= bound + half_rounding(dtype) * (want.abs() + bound)).all(), float((err - bound).max())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,length,spec", [(64, 1, "none"), (128, 257, "wavelength"), (64, 5000, "ramp"), (128, 70000, "linear")])
def test_tables(dtype, D, length, spec):
    b = binding()
    rot = b.make_rotary(D, 500000.0, **SPECS[spec])
    cos, sin = b.rotary_tables(rot, length, dtype)
    at = torch.arange(length) if length < 1000 else torch.cat([torch.arange(0, length, 577), torch.tensor([length - 1])])
    # long bf16 tables take sums of two angles: 2 sqrt(2) TRIG and three roundings of 2^-24 of values up to the gain
    bound = TRIG if dtype == F32 else 2.83 * TRIG + 3 * 2.0 ** -24
    for got, want in zip((cos, sin), cos_sin(rot, at)):
        got = got[at.cuda()]
        assert torch.equal(got[:, :D // 2], got[:, D // 2:])
        hold(got[:, :D // 2], want, bound * rot.gain, dtype)


def test_tables_of_length_zero():
    b = binding()
    cos, sin = b.rotary_tables(b.make_rotary(64, 1e4), 0, BF16)
    assert cos.shape == (0, 64) and sin.shape == (0, 64) and b.last_launch_count() == 0


CASES = [
    # n, heads, kv heads, D, rot, interleaved, spec, top
    (1, 1, 1, 64, 64, False, "none", 100), (1, 3, 0, 128, 16, True, "ramp", 2 ** 31), (37, 12, 12, 64, 32, False, "none", 1000),
    (5, 5, 1, 128, 48, False, "wavelength", 200000), (130, 32, 8, 128, 128, False, "wavelength", 131072),
    (64, 64, 8, 64, 64, True, "ramp", 4096), (9, 40, 8, 128, 64, True, "linear", 2 ** 20), (300, 2, 2, 64, 48, True, "none", 2 ** 31),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("n,heads,kv,D,d,inter,spec,top", CASES)
def test_apply(dtype, inverse, n, heads, kv, D, d, inter, spec, top):
    b = binding()
    g = torch.Generator().manual_seed(n + heads)
    rot = b.make_rotary(D, 10000.0, rot_dim=d, interleaved=inter, **SPECS[spec])
    pos = torch.randint(0, top, (n,), generator=g).to(torch.int32)
    pos[0] = min(top, 2 ** 31) - 1
    q, k = (torch.randn(n, h, D, generator=g).to(dtype).cuda() for h in (heads, max(kv, 1)))
    qo, ko = torch.full_like(q, 9.0), torch.full_like(k, 9.0)
    ws = b.new_status()
    b.rotary_apply(rot, q, k if kv else None, pos.cuda(), qo, ko if kv else None, ws, inverse=inverse)
    b.check_status(ws)
    hold(qo, *turned(rot, q, pos, inverse), dtype)
    assert torch.equal(qo[..., d:], q[..., d:])
    if kv:
        hold(ko, *turned(rot, k, pos, inverse), dtype)
    else:
        assert (ko == 9).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_apply_on_slices_and_in_place(dtype):
    """Slices of one projection in place, and from one projection into another with other strides."""
    b = binding()
    n, hq, hk, D = 21, 6, 2, 64
    rot = b.make_rotary(D, 10000.0, rot_dim=32)
    x = torch.randn(n, hq + 2 * hk, D, device="cuda").to(dtype)
    y = torch.full((2 * n, hq + hk + 1, D), 3.0, device="cuda").to(dtype)
    pos = torch.arange(n, dtype=torch.int32, device="cuda") * 100
    ws = b.new_status()
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:].clone()
    want = turned(rot, q, pos, False), turned(rot, k, pos, False)
    b.rotary_apply(rot, q, k, pos, y[::2, :hq], y[::2, hq:hq + hk], ws)
    b.rotary_apply(rot, q, k, pos, q, k, ws)
    b.check_status(ws)
    for (qq, kk) in ((q, k), (y[::2, :hq], y[::2, hq:hq + hk])):
        hold(qq, *want[0], dtype)
        hold(kk, *want[1], dtype)
    assert torch.equal(x[:, hq + hk:], v) and (y[1::2] == 3).all() and (y[:, hq + hk:] == 3).all()


@pytest.mark.parametrize("inter", [False, True])
def test_the_inverse_is_the_gradient(inter):
    """Against the adjoint, <rotate(x), g> = <x, inverse(g)>, and against differences along random directions."""
    b = binding()
    n, h, D = 33, 3, 128
    rot = b.make_rotary(D, 10000.0, rot_dim=96, interleaved=inter, **SPECS["ramp"])
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, g, d = (torch.randn(n, h, D, generator=gen, device="cuda") for _ in range(3))
    pos, ws = torch.randint(0, 100000, (n,), generator=gen, device="cuda").to(torch.int32), b.new_status()

    def f(t, inverse=False):
        out = torch.empty_like(t)
        b.rotary_apply(rot, t, None, pos, out, None, ws, inverse=inverse)
        return out.double()

    grad = f(g, True)
    b.check_status(ws)
    # every term is off by at most (TRIG + 3 * 2^-24 + 2^-24) * gain of the pair's |x|, on either side
    size = (TRIG + 2.0 ** -22) * rot.gain * 4 * float((x.abs().max() * g.abs().sum()))
    assert abs(float((f(x) * g.double()).sum() - (x.double() * grad).sum())) <= size
    step = 0.5
    diff = (f(x + step * d) - f(x - step * d)) / (2 * step)
    # the shifted inputs round too (2^-24 of |x| + |d|), and the difference is divided by 2 * step
    size = (TRIG + 2.0 ** -21) * rot.gain * 8 / step * float((x.abs().max() + d.abs().max()) * g.abs().sum())
    assert abs(float((diff * g.double()).sum() - (d.double() * grad).sum())) <= size


def test_negative_positions_leave_their_tokens():
    b = binding()
    rot = b.make_rotary(64, 10000.0)
    q, k = torch.randn(6, 4, 64, device="cuda"), torch.randn(6, 2, 64, device="cuda")
    pos = torch.tensor([3, -1, 0, 5, -2 ** 31, 7], dtype=torch.int32, device="cuda")
    qo, ko, ws = torch.full_like(q, 9.0), torch.full_like(k, 9.0), b.new_status()
    b.rotary_apply(rot, q, k, pos, qo, ko, ws)
    with pytest.raises(b.PdattnError) as e:
        b.check_status(ws)
    assert e.value.status == b.EBADPOS
    b.check_status(ws)
    bad = (pos < 0).cpu()
    assert (qo[bad] == 9).all() and (ko[bad] == 9).all()
    want, bound = turned(rot, q[~bad], pos[~bad], False)
    hold(qo[~bad], want, bound, F32)


def test_values_that_are_not_finite_stay_in_their_pairs():
    b = binding()
    rot = b.make_rotary(64, 10000.0, rot_dim=32)
    q = torch.randn(3, 2, 64, device="cuda")
    q[1, 0, 4] = float("nan")
    q[2, 1, 50] = float("inf")
    pos, out, ws = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda"), torch.empty_like(q), b.new_status()
    b.rotary_apply(rot, q, None, pos, out, None, ws)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[1, 0, 4] = want[1, 0, 20] = want[2, 1, 50] = True
    assert torch.equal(bad, want) and float(out[2, 1, 50]) == float("inf")


def test_apply_in_a_graph_and_rotated_keys_in_a_decode():
    """Captured, replayed with new inputs; and decode without tables over keys and queries that were rotated here gives
    what decode with the tables of the same frequencies gives, up to those tables' rounding to bf16."""
    b = binding()
    n, hq, hk, D = 4, 8, 2, 64
    rot = b.make_rotary(D, 10000.0, **SPECS["wavelength"])
    q, k, v = (torch.randn(n, h, D, device="cuda").to(BF16) for h in (hq, hk, hk))
    pos = torch.tensor([0, 63, 64, 200], dtype=torch.int32, device="cuda")
    qo, ko, ws = torch.empty_like(q), torch.empty_like(k), b.new_status()
    graph = torch.cuda.CUDAGraph()
    b.rotary_apply(rot, q, k, pos, qo, ko, ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        b.rotary_apply(rot, q, k, pos, qo, ko, ws)
    q.copy_(torch.randn_like(q))
    graph.replay()
    b.check_status(ws)
    hold(qo, *turned(rot, q, pos, False), BF16)

    table = torch.arange(n * 4, dtype=torch.int32, device="cuda").view(n, 4)
    pool = torch.randn(2, n * 4, hk, 64, D, device="cuda").to(BF16)
    cos, sin = b.rotary_tables(rot, 256, BF16)
    outs = []
    for tables in (True, False):
        p = b.make_params(n, hq, hk, D, 4, n * 4, BF16, rope_cos=cos if tables else None, rope_sin=sin if tables else None)
        dws, out, kp, vp = b.new_workspace(p), torch.empty_like(q), pool[0].clone(), pool[1].clone()
        b.decode_fused(p, q if tables else qo, k if tables else ko, v, pos, table, kp, vp, out, dws)
        b.check_status(dws)
        outs.append(out.float())
    # tables and rotated values are rounded to bf16 (2^-8 each): a score of about sqrt(64) terms of 1 moves by about
    # 4 * 2^-8, and so does a weight; the outputs are of size 1
    assert (outs[0] - outs[1]).abs().max() < 0.1
