"""The arrays of a page call: outputs that overlap what the call reads, or one another, are refused.  CPU only."""
import ctypes

import pytest
import torch

NULL = ctypes.c_void_p(0)
WS = ctypes.c_void_p(1 << 20)
ROWS, WIDTH, PAGES = 4, 2, 4                # lengths, refs and page_map are of one size
BYTES = {"table": 4 * ROWS * WIDTH, "lengths": 4 * ROWS, "refs": 4 * PAGES, "parents": 4 * ROWS, "new_lengths": 4 * ROWS,
         "table_out": 4 * ROWS * WIDTH, "refs_out": 4 * PAGES, "page_map": 4 * PAGES}
ORDER = {"update": ("table", "lengths", "refs", "parents", "new_lengths", "table_out", "refs_out"),
         "compact": ("table", "lengths", "refs", "table_out", "refs_out", "page_map")}
OUTPUTS = ("table_out", "refs_out", "page_map")
IN_PLACE = {"table_out": "table", "refs_out": "refs"}


@pytest.fixture(scope="module")
def b():
    from paged_gqa_decode_step_gb300 import build
    build.build()
    from paged_gqa_decode_step_gb300 import binding
    return binding


def call(b, kind, rows=ROWS, width=WIDTH, **at):
    p = b.make_params(rows, 8, 2, 64, width, PAGES, torch.bfloat16)
    pool = (b.Pool * 1)(b.Pool(4096, 2, 128))
    args = [ctypes.c_void_p(at.get(name, 4096 * (i + 2))) for i, name in enumerate(ORDER[kind])]
    return getattr(b.lib, f"pdattn_pages_{kind}")(p, 1, pool, *args, WS, 1 << 40, NULL)


PAIRS = [(kind, out, other) for kind in ORDER for out in OUTPUTS for other in ORDER[kind]
         if out in ORDER[kind] and other != out]


@pytest.mark.parametrize("kind,out,other", PAIRS)
def test_outputs_are_their_own(b, kind, out, other):
    base = 1 << 16
    places = [base + BYTES[other] - 4, base - BYTES[out] + 4]          # one entry in common, at either end
    if IN_PLACE.get(out) != other:
        places.append(base)
    for at in places:
        assert call(b, kind, **{other: base, out: at}) == b.EINVAL, at
        said = b.lib.pdattn_last_error()
        assert b"overlap" in said and (out.encode() in said or other.encode() in said)
        assert b.last_launch_count() == 0
    if not torch.cuda.is_available():
        # neighbours, and updates in place, get as far as the device, which is not there
        for at in [base + BYTES[other], base - BYTES[out]] + [base] * (IN_PLACE.get(out) == other):
            assert call(b, kind, **{other: base, out: at}) == b.ECUDA


@pytest.mark.parametrize("kind", ORDER)
@pytest.mark.parametrize("out", ["table_out", "refs_out"])
def test_in_place_is_one_input_alone(b, kind, out):
    """An input of the same size that lies where the table (or the counts) does is not what may be updated in place."""
    at = 1 << 16
    assert call(b, kind, width=1, **{IN_PLACE[out]: at, out: at, "lengths": at}) == b.EINVAL


@pytest.mark.parametrize("kind", ORDER)
def test_without_rows_their_arrays_have_no_extent(b, kind):
    if torch.cuda.is_available():
        pytest.skip("would launch")
    at = 4096 * 4                                                      # refs
    assert call(b, kind, rows=0, lengths=at, table=at, table_out=at) == b.ECUDA
