"""Tree attention over one-byte caches where weights lie far below the largest, against the
definition in 64 bits."""

import numpy as np
import pytest
import torch

from serve_helpers import Cache, check, random_trees, tree_reference
from test_gpu_tree import _call, _queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("n", [5, 12, 40])
def test_a_long_tail_of_small_weights(kv, n):
    """One token with almost all of the weight and 60000 with 2^-25.2 of it each, whose values are
    larger: together they are a tenth of the result. 160 sequences of one context, so that a CTA's
    stretch holds it all. (fp16 weights that refer to the largest one lose the others: 2^-25 and less
    rounds to 0. Those of a few bits, at 2^-18.2, lose 2^-6.8 of the tail at most: 2^-10 of the
    result, within what the bound has for the fp32 parts.)"""
    d, hq, b, length = 64, 8, 160, 60000
    c = Cache([length], 1, d, 16, kv, seed=1)
    ids = c.tables[0].long()
    # K: the code that stands for 1 in the first column, its sign telling the heavy token; V: +-1
    # times a scale of 1 (heavy), 64 (others)
    one = {"int8": 1, "e4m3": 0x38, "e5m2": 0x3C}[kv]
    minus = {"int8": -1, "e4m3": 0xB8, "e5m2": 0xBC}[kv]
    gen = torch.Generator(device="cuda").manual_seed(3)
    for which in range(2):
        c.caches[which].zero_()
        c.scales[which].fill_(1.0)
    kc, vc = c.caches
    kc[..., 0] = minus
    heavy = (ids[100 // 16], 0, 100 % 16)
    kc[heavy + (0,)] = one
    vc.copy_(torch.where(torch.rand(vc.shape, generator=gen, device="cuda") < 0.9, one, minus))
    c.scales[1].fill_(64.0)
    c.scales[1][heavy] = 1.0
    value = lambda x: torch.where(x == one, 1.0, torch.where(x == minus, -1.0, 0.0))  # noqa: E731
    c.values = [value(x).double() * s[..., None].double() for x, s in zip(c.caches, c.scales)]
    # scores +-x: the weights' ratio is 2^-25.2
    q = torch.zeros(1, n, hq, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    scale = 25.2 / 2 * float(np.log(2.0))
    mask, seen = random_trees([n], 3, n)
    out, bound = tree_reference(c, q, seen, [n], scale)
    assert 0.05 < (length - n) * 2.0 ** -25.2 * 64 * 0.8 < 0.2
    c.tables, c.context_lens = c.tables.repeat(b, 1), c.context_lens.repeat(b)
    got = _call(c, q.repeat(b, 1, 1, 1), mask.cuda().repeat(b, 1, 1), scale)
    check(got, out.expand(got.shape), bound.expand(got.shape))
