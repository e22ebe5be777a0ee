"""The constants that tests/shared_util.py restates the kernels' arithmetic with are those of the sources.  CPU only."""
import inspect
import os
import re

from paged_gqa_decode_step_gb300 import build
import shared_util


def source(name):
    return open(os.path.join(build.CSRC, name)).read()


def constant(text, name):
    return int(re.search(r"constexpr int %s = (\d+);" % name, text).group(1))


def default(f, name):
    return inspect.signature(f).parameters[name].default


def test_what_groups_share():
    text = source("shared.cuh")
    assert default(shared_util.shared_slots, "min_pages") == constant(text, "kSharedMinPages")
    assert default(shared_util.shared_slots, "min_saved") == constant(text, "kSharedMinSaved")


def test_partial_slots():
    assert "return (nb + share - 2) / share + 1;" in source("shared.cuh")
    assert "return s1 / share + 2 * s2 + index;" in source("shared.cuh")
    text = source("internal.h")
    assert constant(text, "kSharedRuns") == 8
    assert "S.pre_slots = (long long)tile_tokens * grid + 2ll * rows * kv_heads + n_groups;" in text
    assert "S.own_slots = 2ll * kSharedRuns * grid + (long long)rows * kv_heads;" in text


def test_runs_of_own_pages():
    text = source("attend_kernel.cuh")
    assert default(shared_util.own_runs, "start") == constant(text, "kItemUnits")
    assert "even = share <= 6 * (U + 1);" in text
    assert "big = even ? max(share, U + 1) : share / 4 * 3, small = even ? big : max((share + 15) / 16, 5 * (U + 1));" in text
