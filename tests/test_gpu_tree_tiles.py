"""Tree attention of more than 128 rows per KV head (two pipelines of row tiles) against the
definition in 64 bits: odd counts of tiles, large groups, masks, scales and values at their ends."""

import pytest
import torch

from serve_helpers import Cache, check, random_trees, tree_reference
from test_gpu_tree import _call, _queries, _sizes

pytestmark = pytest.mark.gpu

CASES = [
    # hq, hkv, d, bs, nodes, contexts (nodes included)
    (192, 1, 64, 16, 3, [3, 63, 64, 65, 129]),     # a group of 192: two parts of 96 heads
    (131, 1, 128, 32, 2, [2, 60, 200]),            # a prime group: a head at a time
    (256, 2, 64, 32, 1, [1, 64, 127]),             # 128 heads a group and one node: one tile
    (129, 1, 64, 16, 1, [1, 64, 127]),             # one head more
    (12, 2, 128, 16, 43, [43, 64, 107, 500]),      # 258 rows of a group of 6: three tiles
    (20, 4, 64, 32, 77, [77, 78, 140, 400]),       # 385 rows of a group of 5: four tiles
    (10, 1, 128, 16, 13, [13, 64, 65, 1000]),      # 130 rows: the second tile has one node
    (1, 1, 64, 16, 129, [129, 192, 193, 1500]),    # one head, 129 nodes
]


@pytest.mark.parametrize("kv", ["bf16", "int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}-{c[1]}-{c[2]}-{c[4]}" for c in CASES])
def test_tiles(case, kv):
    hq, hkv, d, bs, n, lens = case
    c = Cache(lens, hkv, d, bs, kv, seed=hq)
    q = _queries(len(lens), n, hq, d, seed=n)
    sizes = [max(0, n - s) for s in range(len(lens))]
    mask, seen = random_trees(sizes, 5, n, seed=n)
    want = tree_reference(c, q, seen, sizes, d ** -0.5)
    got = _call(c, q, mask.cuda(), d ** -0.5, tree_lens=_sizes(sizes))
    check(got, *want)
    for s, t in enumerate(sizes):
        assert (got[s, t:] == 0).all()


@pytest.mark.parametrize("kv", ["bf16", "e5m2"])
@pytest.mark.parametrize("n", [40, 70])
def test_contexts_cut_over_many_ctas(kv, n):
    """Two and three row tiles, contexts that every CTA has a piece of, one that is shorter."""
    lens = [12000, n, 64 * 40 + 1]
    c = Cache(lens, 1, 128, 16, kv, seed=n)
    q = _queries(3, n, 5, 128, seed=1)
    mask, seen = random_trees([n] * 3, 4, n, seed=2)
    check(_call(c, q, mask.cuda(), 0.09), *tree_reference(c, q, seen, [n] * 3, 0.09))


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_masks_of_any_shape(kv):
    """Masks that leave a node nothing, that see later nodes, all and none; bits past the tree; a
    context that is the tree alone, no context."""
    n, lens, sizes = 66, [66, 0, 130, 66, 300], [66, 0, 60, 64, 66]
    c = Cache(lens, 2, 64, 16, kv, seed=1)
    q = _queries(5, n, 6, 64)
    gen = torch.Generator().manual_seed(5)
    mask = torch.randint(-2 ** 63, 2 ** 63 - 1, (5, n, 2), generator=gen)
    mask[:, 0] = 0
    mask[:, 1] = -1
    mask[:, 65, 0] = 0
    bits = torch.arange(n)
    seen = [(mask[s][:, bits // 64] >> (bits % 64) & 1 == 1)[:t, :t] for s, t in enumerate(sizes)]
    want = tree_reference(c, q, seen, sizes, 0.125)
    got = _call(c, q, mask.cuda(), 0.125, tree_lens=_sizes(sizes))
    check(got, *want)
    assert (got[0, 0] == 0).all() and (got[1] == 0).all()


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("scale", [-0.125, 0.0])
def test_negative_and_zero_scale(kv, scale):
    lens, n = [50, 300], 40
    c = Cache(lens, 1, 64, 16, kv, seed=4)
    q = _queries(2, n, 4, 64)
    mask, seen = random_trees([n] * 2, 3, n)
    check(_call(c, q, mask.cuda(), scale), *tree_reference(c, q, seen, [n] * 2, scale))


@pytest.mark.parametrize("power", [-60, 60])
@pytest.mark.parametrize("kv", ["bf16", "int8", "e5m2"])
def test_queries_of_any_size(kv, power):
    """Query rows far from 1 (an fp16 query would over- or underflow), undone by the scale; one
    row of zeros."""
    lens, n = [77, 200], 40
    c = Cache(lens, 2, 128, 16, kv, seed=2)
    q = _queries(2, n, 8, 128)
    q[:, 3] = 0
    mask, seen = random_trees([n] * 2, 3, n)
    out, bound = tree_reference(c, q, seen, [n] * 2, 0.09)
    check(_call(c, (q.double() * 2.0 ** power).to(q.dtype), mask.cuda(), 0.09 * 2.0 ** -power),
          out, bound)


@pytest.mark.parametrize("nodes", [40, 20])
def test_values_in_masked_places(nodes):
    """Infinities and NaN in what no row sees: nodes that are masked for all, tokens past the
    context in the last block."""
    lens, hq = [100, 90], 8
    c = Cache(lens, 1, 64, 16, seed=3)
    q = _queries(2, nodes, hq, 64)
    mask, seen = random_trees([nodes] * 2, 3, nodes)
    hidden = nodes // 2
    for s in range(2):
        seen[s][:, hidden] = False
        mask[s, :, 0] &= ~(1 << hidden)
    want = tree_reference(c, q, seen, [nodes] * 2, 0.125)
    for s, worst in enumerate((float("inf"), float("-inf"))):
        p = lens[s] - nodes + hidden
        c.caches[0][c.tables[s, p // 16].item(), :, p % 16] = worst  # the score: masked
    check(_call(c, q, mask.cuda(), 0.125), *want)


def test_status_flags():
    from paged_kv_decode_02_gb300 import pagedkv
    n, lens = 40, [60, 60, 60]
    c = Cache(lens, 2, 64, 16, seed=1)
    q = _queries(3, n, 8, 64)
    mask, seen = random_trees([n] * 3, 3, n)
    out, bound = tree_reference(c, q, seen, [n] * 3, 0.125)

    def run(**kw):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = _call(c, q, mask.cuda(), 0.125, status=status, **kw)
        check(got[0], out[0], bound[0])
        check(got[2], out[2], bound[2])
        assert (got[1] == 0).all()
        return status.item()
    bad = pagedkv.DEV_BAD_CONTEXT_LEN
    assert run(tree_lens=_sizes([n, n + 1, n])) == bad
    assert run(tree_lens=_sizes([n, -1, n])) == bad
    c.context_lens[1] = 39
    assert run() == bad
    c.context_lens[1] = 100
    assert run() == bad
    c.context_lens[1] = 60
    c.tables[1, 2] = c.nb
    assert run() == pagedkv.DEV_BAD_BLOCK_ID


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_same_bits_graphs_and_a_stream(kv):
    """The same bits every time; two graphs that share a workspace; a stream of its own."""
    import paged_kv_decode_02_gb300 as pk
    from paged_kv_decode_02_gb300 import pagedkv
    lens, n = [500, 90, 1400], 40
    c = Cache(lens, 2, 128, 16, kv, seed=6)
    q = [_queries(3, n, 8, 128, seed=i) for i in range(2)]
    masks = [random_trees([n] * 3, 4, n, seed=i)[0].cuda() for i in range(2)]
    first = [_call(c, q[i], masks[i], 0.09) for i in range(2)]
    for _ in range(3):
        assert torch.equal(first[0], _call(c, q[0], masks[0], 0.09))
    kvt = {"bf16": pagedkv.KV_BF16, "e4m3": pagedkv.KV_FP8_E4M3}[kv]
    need = pk.tree_workspace_bytes(3, 8, 2, 128, 16, c.nb, c.tables.shape[1], n, kvt)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(x) for x in q]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            _call(c, q[i], masks[i], 0.09, out=outs[i], workspace=ws)
    for _ in range(2):
        for i in range(2):
            outs[i].zero_()
            graphs[i].replay()
    for i in range(2):
        assert torch.equal(outs[i], first[i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _call(c, q[1], masks[1], 0.09)
    side.synchronize()
    assert torch.equal(got, first[1])
    with pytest.raises(RuntimeError):
        _call(c, q[0], masks[0], 0.09, workspace=ws[:need - 256])


@pytest.mark.parametrize("n", [4, 40])
def test_output_in_place_is_refused(n):
    """A query row is read where the context is cut, after other rows have been written."""
    c = Cache([n, 80], 2, 64, 16)
    q = _queries(2, n, 8, 64)
    mask, _ = random_trees([n] * 2, 3, n)
    with pytest.raises(ValueError, match="out"):
        _call(c, q, mask.cuda(), 0.125, out=q)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("b", [1500, 20000])
def test_large_batches(b, kv):
    """More sequences than the decode kernel takes, of few rows each; every one of three lengths."""
    n, hq, hkv, d, bs = 2, 4, 2, 64, 16
    lens = [2, 17, 0][:3]
    c = Cache(lens, hkv, d, bs, kv, seed=7)
    pick = torch.arange(b, device="cuda") % 3
    q3 = _queries(3, n, hq, d, seed=8)
    mask = torch.tensor([[[1], [3]]] * 3)
    seen = [torch.tensor([[True, False], [True, True]])] * 3
    sizes = [2, 2, 0]
    out, bound = tree_reference(c, q3, seen, sizes, 0.125)
    c.tables, c.context_lens = c.tables[pick].contiguous(), c.context_lens[pick].contiguous()
    got = _call(c, q3[pick].contiguous(), mask.cuda()[pick].contiguous(), 0.125,
                tree_lens=_sizes(sizes)[pick].contiguous())
    check(got, out[pick], bound[pick])
