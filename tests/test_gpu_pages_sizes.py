"""Page calls at pool sizes where one CTA gives way to the cluster, on the GPU, bit for bit as in tests/test_gpu_pages.py."""
import random

import pytest
import torch

from gpu_util import binding
from pages_util import State, pages
from test_gpu_pages import KINDS, Cache, ints

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("num_pages", [4607, 4609, 6001, 8191, 8192, 8193, 9217])
@pytest.mark.parametrize("rows,width", [(16, 64), (40, 128)])
def test_update(num_pages, rows, width):
    rng = random.Random(num_pages + rows)
    lengths = [rng.randint(0, 64 * width // 2) for _ in range(rows)]
    s = State(rows, width, num_pages, lengths, seed=num_pages, share=3, pins=(0, 5, num_pages - 1))
    parents = [rng.choice([r, r, rng.randrange(rows), -1]) for r in range(rows)]
    new = [min(64 * width, (lengths[p] if p >= 0 else 0) + rng.choice([0, 1, 1, 200])) for p in parents]
    c = Cache(s, KINDS)
    table, refs, copies = s.update(parents, new)
    c.update(parents, new)
    c.check()
    c.same(table, refs, copies)


@pytest.mark.parametrize("num_pages", [4607, 4609, 6001, 8191, 8192, 8193, 9217])
@pytest.mark.parametrize("rows,width", [(16, 64), (40, 110)])
def test_compact(num_pages, rows, width):
    rng = random.Random(num_pages + rows)
    lengths = [rng.randint(0, 64 * width) for _ in range(rows)]
    s = State(rows, width, num_pages, lengths, seed=num_pages, share=2, pins=(0, num_pages - 1))
    c = Cache(s, KINDS)
    table, refs, to = s.compact()
    page_map = torch.full((num_pages,), 9, dtype=torch.int32, device="cuda")
    c.compact(page_map)
    c.check()
    c.same(table, refs, [(x, y, 64) for x, y in enumerate(to) if y >= 0 and y != x])
    assert torch.equal(page_map, ints(to))
