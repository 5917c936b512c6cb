"""Tree attention over one-byte caches whose V rows lie far from 1, against the definition in 64 bits."""

import pytest
import torch

from serve_helpers import Cache, check, random_trees, tree_reference
from test_gpu_tree import _call, _queries

pytestmark = pytest.mark.gpu


# rows of a KV head: up to 64, 65 to 128 in a table of less than 256 tokens and of more, more tiles
ROWS = [(8, 5, 300), (8, 12, 200), (8, 12, 400), (8, 12, 900), (8, 40, 900)]


def _scaled(lens, hkv, d, kv, power, seed):
    """A cache whose V rows are the usual ones times powers of two, one per (sequence's) row."""
    c = Cache(lens, hkv, d, 16, kv, seed=seed)
    gen = torch.Generator(device="cpu").manual_seed(seed)
    f = 2.0 ** power(gen, (c.nb, hkv, 16)).float().cuda()
    c.scales[1] = (c.scales[1] * f).contiguous()
    c.values[1] = c.values[1] * f[..., None].double()
    return c


@pytest.mark.parametrize("kv", ["int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("hq,n,length", ROWS)
@pytest.mark.parametrize("power", [-40, -20, 20, 60])
def test_value_rows_of_any_size(kv, hq, n, length, power):
    """All V rows far below and far above what fp16 holds."""
    lens = [n, 129, length]
    c = _scaled(lens, 1, 128, kv, lambda gen, shape: torch.full(shape, power), n)
    q = _queries(3, n, hq, 128, seed=n)
    mask, seen = random_trees([n] * 3, 3, n, seed=n)
    check(_call(c, q, mask.cuda(), 0.09), *tree_reference(c, q, seen, [n] * 3, 0.09))


@pytest.mark.parametrize("kv", ["int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("hq,n,length", ROWS + [(8, 40, 9000), (4, 3, 9000)])
def test_value_rows_of_mixed_size(kv, hq, n, length):
    """V rows whose sizes differ by up to 2^24 from token to token, and from block to block by as much
    again."""
    def power(gen, shape):
        rows = torch.randint(-12, 13, shape, generator=gen)
        return rows + torch.randint(-12, 13, shape[:1], generator=gen)[:, None, None]
    lens = [n, 129, length]
    c = _scaled(lens, 1, 64, kv, power, n)
    q = _queries(3, n, hq, 64, seed=n)
    mask, seen = random_trees([n] * 3, 3, n, seed=n)
    check(_call(c, q, mask.cuda(), 0.125), *tree_reference(c, q, seen, [n] * 3, 0.125))


@pytest.mark.parametrize("kv", ["int8", "e5m2"])
@pytest.mark.parametrize("hq,n", [(8, 5), (8, 12), (8, 40)])
def test_value_rows_that_rise_along_the_context(kv, hq, n):
    """A context whose first rows are all zeros (scales too), whose next ones are tiny, and whose
    last ones are large, with the weight on the tiny ones; a scale past the context that is NaN."""
    d, length = 64, 1000
    c = Cache([length], 1, d, 16, kv, seed=2)
    ids = c.tables[0].long()
    at = torch.arange(length, device="cuda")
    f = torch.where(at < 256, 0.0, torch.where(at < 600, 2.0 ** -30, 2.0 ** 20))
    for p in range(0, length, 16):
        m = min(16, length - p)
        c.scales[1][ids[p // 16], 0, :m] *= f[p:p + m]
        c.values[1][ids[p // 16], 0, :m] *= f[p:p + m, None].double()
    # K: large in the middle part's favour
    q = torch.zeros(1, n, hq, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    codes = c.caches[0]
    one = {"int8": 1, "e5m2": 0x3C}[kv]
    codes[..., 0] = 0
    for p in range(256, 600):
        codes[ids[p // 16], 0, p % 16, 0] = one
        c.scales[0][ids[p // 16], 0, p % 16] = 1.0
    live = c.values[0].clone()
    live[..., 0] = 0.0
    for p in range(256, 600):
        live[ids[p // 16], 0, p % 16] = (codes[ids[p // 16], 0, p % 16].double() if kv == "int8" else
                                         codes[ids[p // 16], 0, p % 16].view(torch.float8_e5m2)
                                         .double())
    c.values[0] = live
    mask, seen = random_trees([n], 3, n)
    for scale in (8.0, 60.0):
        check(_call(c, q, mask.cuda(), scale), *tree_reference(c, q, seen, [n], scale))
