"""Tree attention over many short items, against the definition in 64 bits."""

import pytest
import torch

from serve_helpers import Cache, check, random_trees, tree_reference
from test_gpu_tree import _call, _queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_many_short_items(kv):
    """Segments that follow each other quickly: a CTA sends for the next one's queries while it copies
    this one's context."""
    n, lens = 40, [40 + (37 * s) % 150 for s in range(300)]
    c = Cache(lens, 2, 64, 16, kv, seed=9)
    q = _queries(len(lens), n, 8, 64, seed=9)
    mask, seen = random_trees([n] * len(lens), 4, n, seed=9)
    mask = mask.cuda()
    first = _call(c, q, mask, 0.125)
    check(first, *tree_reference(c, q, seen, [n] * len(lens), 0.125))
    for _ in range(10):
        assert torch.equal(first, _call(c, q, mask, 0.125))
