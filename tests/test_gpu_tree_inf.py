"""Tree attention where keys that rows see have scores of -inf."""

import pytest
import torch

from serve_helpers import Cache, check, random_trees, tree_reference
from test_gpu_tree import _call, _queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e5m2"])
@pytest.mark.parametrize("n", [4, 12, 40])
@pytest.mark.parametrize("first,last", [(0, 130), (128, 300), (0, 2000), (500, 1500)])
def test_scores_of_minus_infinity(kv, n, first, last):
    """Keys of -inf scores weigh nothing, in whatever tiles of whichever kernel they fill; contexts
    whole in one CTA and cut between CTAs."""
    lens = [2100, last + n + 3, 129 + n]
    c = Cache(lens, 1, 128, 16, kv, seed=n)
    q = _queries(3, n, 8, 128, seed=1).abs() + 0.1
    mask, seen = random_trees([n] * 3, 3, n)
    for s, length in enumerate(lens):
        for p in range(first, min(last, length - n)):
            row = (c.tables[s, p // 16].item(), 0, p % 16)
            c.caches[0][row] = float("-inf") if kv == "bf16" else 0xFC
            c.values[0][row] = float("-inf")
    want = tree_reference(c, q, seen, [n] * 3, 0.09)
    for status in (None, torch.zeros(1, dtype=torch.int32, device="cuda")):
        check(_call(c, q, mask.cuda(), 0.09, status=status), *want)
