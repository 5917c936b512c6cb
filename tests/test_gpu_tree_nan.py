"""Tree attention of rows that hold NaN."""

import pytest
import torch

from serve_helpers import Cache, check, random_trees, tree_reference
from test_gpu_tree import _call, _queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("n", [4, 12, 40])
def test_nan_queries_stay_nan(kv, n):
    """A NaN in a query row gives NaN in all of its outputs, whether or not its item was cut between
    CTAs and whoever joins it, and in no other row's."""
    lens = [9000, n, 200]
    c = Cache(lens, 1, 128, 16, kv, seed=5)
    q = _queries(3, n, 8, 128, seed=5)
    mask, seen = random_trees([n] * 3, 3, n)
    out, bound = tree_reference(c, q, seen, [n] * 3, 0.09)
    q[0, 1, 2, 7] = float("nan")
    q[2, n - 1, 7, 100] = float("nan")
    for status in (None, torch.zeros(1, dtype=torch.int32, device="cuda")):
        got = _call(c, q, mask.cuda(), 0.09, status=status)
        assert got[0, 1, 2].isnan().all() and got[2, n - 1, 7].isnan().all()
        got[0, 1, 2] = out[0, 1, 2].to(got.dtype)
        got[2, n - 1, 7] = out[2, n - 1, 7].to(got.dtype)
        check(got, out, bound)
