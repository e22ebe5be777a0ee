"""The coded-cache calls refuse bad arguments on the host, before any launch (CPU only), and the CPU reference that the
GPU tests compare against does what the formula says."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

import coded_util as cu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL = ctypes.c_void_p(0)
AT = ctypes.c_void_p(4096)      # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def b():
    from paged_gqa_decode_step_gb300 import build
    build.build()
    from paged_gqa_decode_step_gb300 import binding
    return binding


def _p(b, **kw):
    base = dict(rows=2, heads=8, kv_heads=2, head_dim=64, pages_per_row=4, num_pages=8, dtype=torch.bfloat16)
    base.update(kw)
    return b.make_params(**base)


def _cache(b, **kw):
    c = b.CodedCache(4096, 4096, 4096, 4096, b.E4M3, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _calls(b, p, c, n=4, ws=AT, bytes_=1 << 40, at=AT):
    L = b.lib
    return {
        "write": lambda: L.pdattn_coded_write(p, c, n, at, at, at, at, ws, bytes_, NULL),
        "read": lambda: L.pdattn_coded_read(p, c, n, at, at, at, ws, bytes_, NULL),
        "decode": lambda: L.pdattn_coded_decode(p, c, at, at, at, at, at, at, ws, bytes_, NULL),
        "prefill": lambda: L.pdattn_coded_prefill(p, c, n, at, at, at, at, at, at, at, at, ws, bytes_, NULL),
    }


CALLS = ("write", "read", "decode", "prefill")


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,status", [(dict(heads=6, kv_heads=4), 1), (dict(head_dim=96), 2), (dict(num_pages=0), 1),
                                       (dict(heads=32, kv_heads=2), 2), (dict(rows=-1), 1)])
def test_parameters_are_checked(b, call, kw, status):
    assert _calls(b, _p(b, **kw), _cache(b))[call]() == status
    assert b.lib.pdattn_last_error() and b.last_launch_count() == 0


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("field,value", [("k", None), ("v", None), ("k_scale", None), ("v_scale", None), ("k", 4104),
                                         ("v", 4097), ("k_scale", 4100), ("v_scale", 4104), ("code", 2), ("code", -1),
                                         ("reserved", 1)])
def test_the_cache_is_checked(b, call, field, value):
    assert _calls(b, _p(b), _cache(b, **{field: value}))[call]() == b.EINVAL
    assert _calls(b, _p(b), None)[call]() == b.EINVAL


@pytest.mark.parametrize("call", CALLS)
def test_pointers_and_workspaces_are_checked(b, call):
    p, c = _p(b), _cache(b)
    assert _calls(b, p, c, at=NULL)[call]() == b.EINVAL
    assert b"NULL" in b.lib.pdattn_last_error()
    assert _calls(b, p, c, at=ctypes.c_void_p(4104))[call]() == b.EINVAL      # 8-byte aligned only
    if call in ("write", "read") or torch.cuda.is_available():
        assert _calls(b, p, c, ws=NULL)[call]() == b.EINVAL
        assert _calls(b, p, c, ws=ctypes.c_void_p(4096 + 128))[call]() == b.EINVAL
        assert _calls(b, p, c, bytes_=255)[call]() == b.EINVAL
        assert b"workspace" in b.lib.pdattn_last_error()


def test_counts(b):
    p, c = _p(b), _cache(b)
    for call in ("write", "read", "prefill"):
        assert _calls(b, p, c, n=-1)[call]() == b.EINVAL
        assert _calls(b, p, c, n=0, at=NULL, ws=NULL)[call]() == b.OK          # nothing to do
        assert _calls(b, p, c, n=2 ** 28)[call]() == b.EUNSUPPORTED
    assert _calls(b, _p(b, rows=0), c, at=NULL, ws=NULL)["decode"]() == b.OK
    assert _calls(b, _p(b, rows=0), c)["prefill"]() == b.EINVAL
    assert _calls(b, _p(b, rows=2 ** 20, pages_per_row=2 ** 10), c)["decode"]() == b.EUNSUPPORTED
    assert _calls(b, _p(b, dtype=torch.float32), c)["prefill"]() == b.EUNSUPPORTED   # f16 tensor-core tiles: bf16 only
    assert b.last_launch_count() == 0
    assert b.lib.pdattn_coded_workspace_size(p, -1) == 0
    assert b.lib.pdattn_coded_workspace_size(_p(b, head_dim=96), 4) == 0


def test_the_binding_refuses_what_is_no_cache_tensor(b):
    p = _p(b)
    with pytest.raises(ValueError):
        b.make_coded_cache(p, torch.zeros(1), torch.zeros(1), torch.zeros(1), torch.zeros(1))
    with pytest.raises(ValueError):       # CPU tensors
        codes = torch.zeros(8, 2, 64, 64, dtype=torch.int8)
        b.make_coded_cache(p, codes, codes, torch.zeros(8, 2, 64), torch.zeros(8, 2, 64))


def test_struct_layout_matches_header(b):
    src = r"""
#include <stddef.h>
#include <stdio.h>
#include "pdattn.h"
int main(void) {
  printf("%zu %zu %zu %zu %d %d\n", sizeof(pdattn_coded_cache), offsetof(pdattn_coded_cache, v_scale),
         offsetof(pdattn_coded_cache, code), offsetof(pdattn_coded_cache, reserved), PDATTN_E4M3, PDATTN_INT8);
  return 0;
}
"""
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "l")
        subprocess.run(["gcc", "-x", "c", "-", "-o", exe, "-I", os.path.join(ROOT, "include")], input=src, text=True,
                       check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    C = b.CodedCache
    assert got == [ctypes.sizeof(C), C.v_scale.offset, C.code.offset, C.reserved.offset, b.E4M3, b.INT8]


@pytest.mark.parametrize("source", ["attend_coded.cu", "prefill_coded.cu"])
def test_the_attention_kernels_compile_without_spills(source):
    import re
    from paged_gqa_decode_step_gb300 import build
    with tempfile.TemporaryDirectory() as d:
        r = subprocess.run([build.nvcc(), "-c", os.path.join(build.CSRC, source), "-o", os.path.join(d, "k.o"), "-Xptxas",
                            "-v"] + build._flags(), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    spills = re.findall(r"(\d+) bytes spill stores, (\d+) bytes spill loads", r.stdout + r.stderr)
    assert spills and all(s == ("0", "0") for s in spills), f"{source}: register spills {spills}"


def test_the_binding_wants_a_cache_that_it_made(b):
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    for cache in (_cache(b), None):                      # a bare block names no tensors and no pool shape
        with pytest.raises(TypeError):
            b.coded_write(_p(b), cache, x, x, x, x, x)


class _Table:
    """Stands for a rope table or sinks on a device."""
    shape = (256, 64)

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device

    def data_ptr(self):
        return 4096


@pytest.mark.parametrize("what", [("rope_cos", "rope_sin"), ("sinks",)])
def test_tables_on_another_device_are_refused(b, monkeypatch, what):
    monkeypatch.setattr(b, "_expect", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    cache = _cache(b)
    cache._pool, cache._device, cache._tensors = (8, 2, 64, 64), 0, ()
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    for call in (b.coded_write, b.coded_read, b.coded_decode, b.coded_prefill):
        n = {b.coded_write: 5, b.coded_read: 4, b.coded_decode: 7, b.coded_prefill: 9}[call]
        with pytest.raises(ValueError, match="cuda:1"):
            call(_p(b, **{k: _Table(1) for k in what}), cache, *[x] * n)
    with pytest.raises(ValueError, match="different devices"):
        _p(b, rope_cos=_Table(0), rope_sin=_Table(0), sinks=_Table(1))


@pytest.mark.parametrize("kind", [torch.float8_e4m3fn, torch.int8])
def test_the_reference_codes(kind):
    x = torch.randn(50, 64, generator=torch.Generator().manual_seed(1))
    codes, scale = cu.code(x, kind)
    # half a step of the largest element's binade (e4m3: 3 bits of fraction) or of the scale (int8)
    step = x.abs() * 2.0 ** -4 + scale[:, None] * 2.0 ** -10 if kind != torch.int8 else scale[:, None] / 2
    assert ((codes.float() * scale[:, None] - x).abs() <= step * 1.0001).all()
    zero, s0 = cu.code(torch.zeros(1, 64), kind)
    assert (zero.float() == 0).all() and s0.item() == cu.TINY
    bad, s1 = cu.code(torch.tensor([[1.0] * 63 + [float("inf")]]), kind)
    assert (bad.float() == 0).all() and torch.isnan(s1).all()


def test_the_shares_of_a_decode_call_cover_every_page_once():
    """The static partition of the coded decode (attend_kernel.cuh), replayed on the host."""
    import random
    rnd = random.Random(4)
    U = 3
    for _ in range(200):
        Hk, grid = rnd.choice([1, 2, 8, 12]), rnd.choice([1, 7, 152])
        pages = [rnd.choice([0, 1, 1, 2, 5, 17, 129]) for _ in range(rnd.randint(1, 40))]
        W = sum(n + U for n in pages if n) * Hk
        share = max(-(-W // grid), U + 1)
        seen, partial = {}, {}
        for c in range(grid):
            x0, x1 = c * share, min(W, (c + 1) * share)
            start, slots = 0, []
            for r, n in enumerate(pages):
                if not n:
                    continue
                for h in range(Hk):
                    u0 = start + h * (n + U) + U
                    p0, p1 = max(x0, u0) - u0, min(x1, u0 + n) - u0
                    if p0 >= p1:
                        continue
                    b0, b1 = u0 // share, (u0 + n - 1) // share
                    for p in range(p0, p1):
                        assert (r, h, p) not in seen
                        seen[r, h, p] = c
                    assert b0 <= c <= b1 and (b0 == b1) == (p1 - p0 == n)
                    if b0 != b1:
                        slot = 2 * c + (1 if p0 == 0 else 0)
                        slots.append(slot)
                        assert slot == 2 * (b0 + (c - b0)) + (1 if c == b0 else 0)
                        partial.setdefault((r, h), []).append((c, b1 - b0 + 1))
                start += Hk * (n + U)
            assert len(slots) == len(set(slots)) <= 2
        assert len(seen) == sum(pages) * Hk
        for got in partial.values():        # every CTA between the first and the last takes part
            assert len(got) == got[0][1]
