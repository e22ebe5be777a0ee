"""The binding under a torch that lacks the private names it takes short ways by: the public ones serve."""
import subprocess
import sys

import pytest
import torch

WITHOUT = """
import types
import torch
from paged_gqa_decode_step_gb300 import build
build.build()
names = [n for n in ("_cuda_getDevice", "_cuda_getCurrentRawStream") if hasattr(torch._C, n)]
kept = [getattr(torch._C, n) for n in names]
for n in names:
    delattr(torch._C, n)
from paged_gqa_decode_step_gb300 import binding as b
for n, x in zip(names, kept):        # torch itself goes on with them
    setattr(torch._C, n, x)
if not torch.cuda.is_available():
    for n in names:
        delattr(torch._C, n)
"""


def run(body):
    r = subprocess.run([sys.executable, "-c", WITHOUT + body], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]


def test_without_a_device():
    run("""
torch.cuda.is_available = lambda: False
assert b._here() == -1
torch.cuda.current_stream = lambda device=None: types.SimpleNamespace(cuda_stream=7 + device)
torch.cuda.current_device = lambda: 3
assert b._stream_of(None, 2) == 9 and b._stream_of(types.SimpleNamespace(cuda_stream=1), 2) == 1
assert b._raw_stream(None) == 10 and b._raw_stream(types.SimpleNamespace(cuda_stream=1)) == 1
torch.cuda.is_available = lambda: True
assert b._here() == 3
""")


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")
def test_a_call_on_a_stream():
    run("""
q = torch.randn(3, 2, 64, device="cuda")
pos, outs, ws = torch.arange(3, dtype=torch.int32, device="cuda"), [torch.empty_like(q) for _ in range(2)], b.new_status()
rot, s = b.make_rotary(64, 1e4), torch.cuda.Stream()
torch.cuda.synchronize()
b.rotary_apply(rot, q, None, pos, outs[0], None, ws)
with torch.cuda.stream(s):
    b.rotary_apply(rot, q, None, pos, outs[1], None, ws)
torch.cuda.synchronize()
b.check_status(ws)
assert torch.equal(*outs) and not torch.equal(outs[0], q)
""")
