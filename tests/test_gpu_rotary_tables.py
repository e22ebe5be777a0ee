"""Long bf16 rotary tables, whose rows come in runs of four by the sum formulas, on the GPU: lengths that end within a run,
both head dims, gains other than 1.  Bounds as in tests/test_gpu_rotary.py."""
import pytest
import torch

from gpu_util import binding
from test_gpu_rotary import BF16, F32, SPECS, TRIG, cos_sin, hold

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,length,spec,gain", [(64, 40001, "ramp", 0.0), (64, 40002, "none", 0.75), (128, 20003, "ramp", 0.0),
                                                (128, 20004, "wavelength", 1.5), (128, 131073, "linear", 2.0)])
def test_long_tables(dtype, D, length, spec, gain):
    b = binding()
    # the whole multiprocessors' worth of runs that the sums are used from
    if dtype == BF16:
        assert length >= torch.cuda.get_device_properties(0).multi_processor_count * (4 * 256 // (D // 16))
    rot = b.make_rotary(D, 150000.0, gain=gain, **SPECS[spec])
    assert rot.gain != 1.0
    cos, sin = b.rotary_tables(rot, length, dtype)
    at = torch.cat([torch.arange(8), torch.arange(8, length - 8, 311), torch.arange(length - 8, length)])
    bound = TRIG if dtype == F32 else 2.83 * TRIG + 3 * 2.0 ** -24
    for got, want in zip((cos, sin), cos_sin(rot, at)):
        assert got.shape == (length, D)
        got = got[at.cuda()]
        assert torch.equal(got[:, :D // 2], got[:, D // 2:])
        hold(got[:, :D // 2], want, bound * rot.gain, dtype)


def test_nothing_behind_a_table():
    """The rows past a table's last one, in a run that it cuts short, stay as they are."""
    b = binding()
    rot, length = b.make_rotary(128, 10000.0, **SPECS["ramp"]), 20001
    cos, sin = (torch.full((length + 4, 128), 7.0, dtype=BF16, device="cuda") for _ in range(2))
    assert b.lib.pdattn_rotary_tables(rot, length, b.BF16, cos.data_ptr(), sin.data_ptr(), torch.cuda.current_stream().cuda_stream) == b.OK
    want = b.rotary_tables(rot, length, BF16)
    for got, table in zip((cos, sin), want):
        assert torch.equal(got[:length], table) and (got[length:] == 7).all()
