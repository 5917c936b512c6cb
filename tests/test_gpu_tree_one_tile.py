"""Tree attention in every kernel of one whole row tile, against the definition in 64 bits."""

import pytest
import torch

from serve_helpers import Cache, check, random_trees, tree_reference
from test_gpu_tree import _call, _queries, _sizes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,bs", [(128, 16), (128, 32), (64, 16), (64, 32)])
@pytest.mark.parametrize("kv", ["bf16", "int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("n,longest", [(9, 222), (16, 222), (9, 479), (16, 479)])
def test_one_tile_of_65_to_128_rows(d, bs, kv, n, longest):
    """Rows of one whole tile in tables of less than 256 and of 512 tokens: every type, head size
    and block, with context ends inside a tile, at its end and past it; joined by the merge kernel
    and by the last CTA."""
    lens = [n, 128, 129, longest - 99, longest]
    c = Cache(lens, 2, d, bs, kv, seed=n)
    assert c.tables.shape[1] * bs < 512
    q = _queries(len(lens), n, 16, d, seed=n)
    sizes = [n, n, n - 1, n, 0]
    mask, seen = random_trees(sizes, 4, n, seed=n)
    want = tree_reference(c, q, seen, sizes, d ** -0.5)
    check(_call(c, q, mask.cuda(), d ** -0.5, tree_lens=_sizes(sizes)), *want, "folded")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(_call(c, q, mask.cuda(), d ** -0.5, tree_lens=_sizes(sizes), status=status), *want,
          "merged")
    assert status.item() == 0
