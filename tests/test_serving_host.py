"""Rotary frequencies and the refusals of the calls for continuations of one prompt (rotary positions, page
bookkeeping): CPU only, before any launch."""
import ctypes
import math
import os
import re
import subprocess
import tempfile

import pytest
import torch

NULL = ctypes.c_void_p(0)
AT = ctypes.c_void_p(4096)      # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def b():
    from paged_gqa_decode_step_gb300 import build
    build.build()
    from paged_gqa_decode_step_gb300 import binding
    return binding


def _turns(b, *a, **kw):
    r = b.make_rotary(*a, **kw)
    return [t / 2.0 ** 64 * 2 * math.pi for t in r.turns[:r.rot_dim // 2]], r


def near(got, want):
    # exp, log and three products in double, each off by a few 2^-53, and 2^-64 turns
    return all(abs(a - c) <= 2.0 ** -47 * c + 2.0 ** -60 for a, c in zip(got, want)) and len(got) == len(want)


@pytest.mark.parametrize("D,rot,theta", [(64, 64, 10000.0), (128, 128, 500000.0), (128, 32, 150000.0), (64, 48, 1.5)])
def test_frequencies(b, D, rot, theta):
    f = [theta ** (-2 * i / rot) for i in range(rot // 2)]
    got, r = _turns(b, D, theta, rot_dim=rot)
    assert near(got, f) and r.gain == 1.0 and (r.head_dim, r.rot_dim, r.interleaved) == (D, rot, 0)
    got, r = _turns(b, D, theta, rot_dim=rot, scaling="linear", factor=8.0, interleaved=True, gain=0.5)
    assert near(got, [x / 8 for x in f]) and r.gain == 0.5 and r.interleaved == 1


def test_frequencies_by_wavelength(b):
    f = [500000.0 ** (-i / 64) for i in range(64)]
    want = []
    for x in f:
        length = 2 * math.pi / x
        if length < 8192 / 4.0:
            want.append(x)
        elif length > 8192 / 1.0:
            want.append(x / 8)
        else:
            s = (8192 / length - 1.0) / (4.0 - 1.0)
            want.append((1 - s) * x / 8 + s * x)
    got, r = _turns(b, 128, 500000.0, scaling="wavelength", factor=8.0, low=1.0, high=4.0, original_len=8192)
    assert near(got, want) and r.gain == 1.0
    assert 0 < sum(x / 8 < w < x for x, w in zip(f, want)) < 64


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("rot,theta,factor,low,high,original", [(64, 150000.0, 32.0, 1.0, 32.0, 4096),
                                                               (128, 10000.0, 4.0, 1.0, 32.0, 2048),
                                                               (16, 10000.0, 2.0, 1.0, 1.001, 100)])
def test_frequencies_on_a_ramp(b, whole, rot, theta, factor, low, high, original):
    at = [rot * math.log(original / (t * 2 * math.pi)) / (2 * math.log(theta)) for t in (high, low)]
    if whole:
        at = [min(max(f(x), 0), rot - 1) for f, x in zip((math.floor, math.ceil), at)]
    want = []
    for i in range(rot // 2):
        ramp = min(1.0, max(0.0, (i - at[0]) / max(at[1] - at[0], 0.001)))
        f = theta ** (-2 * i / rot)
        want.append(f / factor * ramp + f * (1 - ramp))
    got, r = _turns(b, 128, theta, rot_dim=rot, scaling="ramp", factor=factor, low=low, high=high, original_len=original,
                    whole_pairs=whole)
    # The ramp's ends are off by 2^-45 (sizes up to 2^6, a few 2^-52 each), so the share of f by 2^-45 over the ramp's
    # width.  w = f / factor + share * f * (1 - 1 / factor) >= f / factor moves by that times f <= factor * w.  And a turn
    # count is a whole number of 2^-64: half of one is 2 pi * 2^-65 < 2^-61 radians, which is no small part of a slow pair.
    share = 2.0 ** -45 / max(at[1] - at[0], 0.001)
    assert all(abs(a - c) <= (2.0 ** -47 + share * factor) * c + 2.0 ** -61 for a, c in zip(got, want))
    assert abs(r.gain - (0.1 * math.log(factor) + 1.0)) <= 2.0 ** -24 * r.gain


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=96), 2), (dict(rot_dim=0), 1), (dict(rot_dim=24), 1), (dict(rot_dim=80), 1), (dict(theta=1.0), 1),
    (dict(theta=math.inf), 1), (dict(theta=math.nan), 1), (dict(factor=0.5), 1), (dict(factor=math.nan), 1),
    (dict(gain=-1.0), 1), (dict(gain=math.inf), 1), (dict(gain=1e300), 1), (dict(gain=1e-60), 1), (dict(scaling="wavelength", low=0.0, high=4.0, original_len=8), 1),
    (dict(scaling="wavelength", low=4.0, high=4.0, original_len=8), 1), (dict(scaling="ramp", low=1.0, high=4.0), 1),
    (dict(scaling="ramp", low=1.0, high=math.inf, original_len=8), 1)])
def test_specs_are_checked(b, kw, status):
    base = dict(head_dim=64, theta=10000.0)
    base.update(kw)
    with pytest.raises(b.PdattnError) as e:
        b.make_rotary(**base)
    assert e.value.status == status
    with pytest.raises(ValueError):
        b.make_rotary(64, 1e4, scaling="other")
    assert b.lib.pdattn_rotary_make(None, b.Rotary()) == b.EINVAL
    for field, value in (("scaling", 4), ("scaling", -1), ("interleaved", 2)):
        spec = b.RotarySpec(64, 64, 0, 0, 0, 0, 1e4, 1.0, 1.0, 2.0, 0.0)
        setattr(spec, field, value)
        assert b.lib.pdattn_rotary_make(spec, b.Rotary()) == b.EINVAL


def test_rotary_calls_are_checked(b):
    L, rot, D = b.lib, b.make_rotary(64, 1e4), 64

    def apply(r=rot, n=3, dtype=b.BF16, inverse=0, hq=2, q=AT, sq=128, qo=ctypes.c_void_p(8192), so=128, hk=1, k=AT, sk=64,
              ko=ctypes.c_void_p(16384), sl=64, pos=AT, ws=AT, nb=256):
        return L.pdattn_rotary_apply(r, n, dtype, inverse, hq, q, sq, qo, so, hk, k, sk, ko, sl, pos, ws, nb, NULL)

    for kw in (dict(r=b.Rotary()), dict(r=None), dict(n=-1), dict(dtype=2), dict(inverse=2), dict(hq=0), dict(hk=-1),
               dict(q=NULL), dict(qo=NULL), dict(k=NULL), dict(ko=NULL), dict(pos=NULL), dict(ws=NULL), dict(nb=255),
               dict(q=ctypes.c_void_p(4104)), dict(ko=ctypes.c_void_p(4100)), dict(sq=120), dict(sq=132), dict(sl=60),
               dict(ws=ctypes.c_void_p(4096 + 128)), dict(qo=AT, so=256)):
        assert apply(**kw) == b.EINVAL, kw
        assert b.last_launch_count() == 0
    assert apply(n=0, q=NULL, ws=NULL) == b.OK
    assert L.pdattn_rotary_tables(rot, -1, b.BF16, AT, AT, NULL) == b.EINVAL
    assert L.pdattn_rotary_tables(rot, 4, 5, AT, AT, NULL) == b.EINVAL
    assert L.pdattn_rotary_tables(rot, 4, b.F32, NULL, AT, NULL) == b.EINVAL
    assert L.pdattn_rotary_tables(rot, 4, b.F32, AT, ctypes.c_void_p(4104), NULL) == b.EINVAL
    assert L.pdattn_rotary_tables(rot, 0, b.F32, NULL, NULL, NULL) == b.OK
    for kw in (dict(interleaved=True), dict(rot_dim=32)):
        assert L.pdattn_rotary_tables(b.make_rotary(64, 1e4, **kw), 4, b.F32, AT, AT, NULL) == b.EUNSUPPORTED


def test_rotary_tensors_are_checked(b):
    rot, t = b.make_rotary(64, 1e4), torch.zeros(2, 3, 64)
    with pytest.raises(TypeError):
        b.rotary_apply(None, t, None, t, t, None, t)
    with pytest.raises(ValueError):
        b.rotary_apply(rot, t.to(torch.float16), None, t, t, None, t)
    with pytest.raises(ValueError):                                  # not on a GPU
        b.rotary_apply(rot, t, None, torch.zeros(2, dtype=torch.int32), t, None, torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError):
        b.rotary_apply(rot, t, t, t, t, None, t)


def _pages_calls(b, p, pools, n=None, at=AT, ws=AT, nb=1 << 40):
    L, k = b.lib, len(pools) if n is None else n
    arr = (b.Pool * max(1, len(pools)))(*pools)
    return {
        "update": lambda: L.pdattn_pages_update(p, k, arr, at, at, at, at, at, at, at, ws, nb, NULL),
        "compact": lambda: L.pdattn_pages_compact(p, k, arr, at, at, at, at, at, at, ws, nb, NULL),
    }


@pytest.mark.parametrize("call", ["update", "compact"])
def test_page_calls_are_checked(b, call):
    def p(**kw):
        base = dict(rows=2, heads=8, kv_heads=2, head_dim=64, pages_per_row=4, num_pages=8, dtype=torch.bfloat16)
        base.update(kw)
        return b.make_params(**base)

    good = b.Pool(4096, 2, 128)
    for kw, status in ((dict(rows=-1), 1), (dict(num_pages=0), 1), (dict(pages_per_row=0), 1),
                       (dict(pages_per_row=2 ** 24), 2), (dict(rows=2 ** 20, pages_per_row=2 ** 11), 2)):
        assert _pages_calls(b, p(**kw), [good])[call]() == status, kw
        assert b.lib.pdattn_pages_workspace_size(p(**kw)) == 0
    q = p()
    q.page_size = 32
    assert _pages_calls(b, q, [good])[call]() == b.EUNSUPPORTED
    for bad in (b.Pool(None, 2, 128), b.Pool(4104, 2, 128), b.Pool(4096, 0, 128), b.Pool(4096, 2, 0), b.Pool(4096, 2, 4097)):
        assert _pages_calls(b, p(), [good, bad])[call]() == b.EINVAL
    assert _pages_calls(b, p(), [], n=0)[call]() == b.EINVAL
    assert _pages_calls(b, p(), [good], at=NULL)[call]() == b.EINVAL
    assert _pages_calls(b, p(), [good], ws=NULL)[call]() == b.EINVAL
    assert _pages_calls(b, p(), [good], ws=ctypes.c_void_p(4096 + 128))[call]() == b.EINVAL
    assert _pages_calls(b, p(), [good], nb=b.lib.pdattn_pages_workspace_size(p()) - 1)[call]() == b.EINVAL
    assert b"workspace" in b.lib.pdattn_last_error() and b.last_launch_count() == 0
    # without rows the pages and their counts are still there
    assert _pages_calls(b, p(rows=0), [good], at=NULL)[call]() == b.EINVAL
    assert _pages_calls(b, p(rows=0), [good], ws=NULL)[call]() == b.EINVAL
    for kw in (dict(num_pages=2 ** 30), dict(rows=2 ** 20, pages_per_row=2 ** 10)):     # counted in 32 bits
        assert _pages_calls(b, p(**kw), [good])[call]() == b.EUNSUPPORTED
        assert b.lib.pdattn_pages_workspace_size(p(**kw)) == 0


@pytest.mark.parametrize("which", range(4))
def test_page_map_is_its_own(b, which):
    p = b.make_params(2, 8, 2, 64, 4, 8, torch.bfloat16)
    pool = (b.Pool * 1)(b.Pool(4096, 2, 128))
    at = [ctypes.c_void_p(4096 * (i + 2)) for i in range(6)]         # table, lengths, refs, table_out, refs_out, page_map
    at[5] = at[(0, 2, 3, 4)[which]]
    assert b.lib.pdattn_pages_compact(p, 1, pool, *at, AT, 1 << 40, NULL) == b.EINVAL
    assert b"page_map" in b.lib.pdattn_last_error()


def test_pools_are_checked(b):
    p = b.make_params(2, 8, 2, 64, 4, 8, torch.bfloat16)
    with pytest.raises(ValueError):
        b.make_pages(p, [])
    with pytest.raises(TypeError):
        b.make_pages(p, [1])
    with pytest.raises(ValueError):
        b.make_pages(p, [torch.zeros(8, 2, 64, 64)])                 # not on a GPU
    with pytest.raises(TypeError):
        b.pages_update(p, None, *[None] * 6)


def test_partials_fit_their_slots():
    """The bounds that the workspace is sized by, whatever number of the CTAs takes the shared pages."""
    import random
    from shared_util import own_runs, shared_slots
    rng = random.Random(1)
    for _ in range(300):
        kv, g = rng.choice([1, 2, 3, 8, 12, 48]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
        groups = [(rng.choice([0, 1, 2, 3, 30, 64, 65, 300]), rng.choice([0, 3, 4, 5, 9, 100, 2000]))
                  for _ in range(rng.choice([1, 2, 9, 40]))]
        rows = sum(n for n, _ in groups)
        grid = rng.choice([2, 148, 152])
        for ctas in (1, rng.randint(1, grid), grid):
            total, share, end = shared_slots(groups, g, kv, ctas)
            assert end <= 2 * (128 // g) * grid + 2 * rows * kv + len(groups) and share * ctas >= total
            for units in (0, 1, rng.randint(1, 1000), rng.randint(1, 10 ** 6)):
                assert own_runs(units, ctas) <= 8 * grid


def test_shared_decode_is_checked(b):
    def p(**kw):
        base = dict(rows=2, heads=8, kv_heads=2, head_dim=64, pages_per_row=4, num_pages=8, dtype=torch.bfloat16)
        base.update(kw)
        return b.make_params(**base)

    def call(q, n=1, at=AT, groups=AT, ws=AT, nb=1 << 40):
        return b.lib.pdattn_decode_shared(q, n, groups, groups, at, at, at, at, at, at, at, at, ws, nb, NULL)

    for kw, status in ((dict(rows=-1), 1), (dict(heads=6, kv_heads=4), 1), (dict(head_dim=96), 2),
                       (dict(heads=32, kv_heads=2), 2), (dict(dtype=torch.float32), 2),
                       (dict(rows=2 ** 20, pages_per_row=2 ** 12), 2)):
        assert call(p(**kw)) == status, kw
        assert b.lib.pdattn_last_error() and b.last_launch_count() == 0
    assert call(p(), n=0) == b.EINVAL and call(p(), n=-1) == b.EINVAL
    assert call(p(), groups=NULL) == b.EINVAL and call(p(), at=NULL) == b.EINVAL
    assert call(p(), at=ctypes.c_void_p(4104)) == b.EINVAL
    assert call(p(), ws=NULL) == b.EINVAL and call(p(), ws=ctypes.c_void_p(4096 + 128)) == b.EINVAL
    assert call(p(rows=0), at=NULL, groups=NULL, ws=NULL) == b.OK
    if torch.cuda.is_available():
        assert call(p(), nb=b.lib.pdattn_shared_workspace_size(p(), 1) - 1) == b.EINVAL


@pytest.mark.parametrize("source", ["rotary.cu", "pages.cu", "shared.cu"])
def test_kernels_compile_without_spills(source):
    from paged_gqa_decode_step_gb300 import build
    with tempfile.TemporaryDirectory() as d:
        r = subprocess.run([build.nvcc(), "-c", os.path.join(build.CSRC, source), "-o", os.path.join(d, "k.o"), "-Xptxas",
                            "-v"] + build._flags(), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    spills = re.findall(r"(\d+) bytes spill stores, (\d+) bytes spill loads", r.stdout + r.stderr)
    assert spills and all(x == ("0", "0") for x in spills), f"{source}: register spills {spills}"
