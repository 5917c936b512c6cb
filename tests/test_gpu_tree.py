"""Tree attention over the paged cache against the definition in 64 bits."""

import pytest
import torch

from serve_helpers import Cache, check, random_trees, tree_reference

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _call(c, q, mask, scale, **kw):
    import paged_kv_decode_02_gb300 as pk
    if c.kv == "bf16":
        return pk.paged_decode_attention_tree(q, *c.caches, c.tables, c.context_lens, mask, scale,
                                              **kw)
    return pk.paged_decode_attention_tree_q8(q, *c.caches, *c.scales, c.tables, c.context_lens,
                                             mask, scale, fmt="e5m2" if c.kv == "e5m2" else "e4m3",
                                             **kw)


def _queries(b, n, hq, d, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(b, n, hq, d, generator=gen, device="cuda").to(BF)


def _sizes(sizes):
    return torch.tensor(sizes, dtype=torch.int32, device="cuda")


CASES = [
    # hq, hkv, d, bs, nodes, contexts (nodes included)
    (8, 8, 64, 16, 5, [5, 6, 40, 128]),            # one row per node
    (8, 2, 128, 16, 1, [1, 127, 128, 129, 700]),   # single nodes
    (8, 1, 128, 32, 7, [7, 130, 260, 513]),        # 56 rows: split tile
    (16, 2, 128, 16, 16, [16, 17, 143, 1000]),     # 128 rows: one whole tile
    (12, 4, 64, 32, 33, [33, 160, 161, 480]),      # 99 rows
    (6, 2, 128, 16, 64, [64, 200, 255, 1025]),     # 192 rows: two row tiles, 64 nodes
    (10, 2, 64, 16, 65, [65, 66, 300, 129]),       # a second mask word
    (8, 1, 128, 32, 100, [100, 128, 612]),         # 800 rows
    (4, 4, 64, 16, 256, [256, 300, 1000]),         # the most nodes
]


@pytest.mark.parametrize("kv", ["bf16", "int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}-{c[1]}-{c[2]}-{c[4]}" for c in CASES])
@pytest.mark.parametrize("ragged", [False, True])
def test_trees(case, kv, ragged):
    """Random trees, whole and ragged; with a status word (joined by the merge kernel) and
    without (by the last CTA)."""
    hq, hkv, d, bs, n, lens = case
    sizes = [max(0, n - 3 * s) for s in range(len(lens))] if ragged else [n] * len(lens)
    c = Cache(lens, hkv, d, bs, kv, seed=n)
    q = _queries(len(lens), n, hq, d, seed=n + 1)
    mask, seen = random_trees(sizes, 6, n, seed=n)
    want = tree_reference(c, q, seen, sizes, d ** -0.5)
    kw = dict(tree_lens=_sizes(sizes)) if ragged else {}
    check(_call(c, q, mask.cuda(), d ** -0.5, **kw), *want, "folded")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(_call(c, q, mask.cuda(), d ** -0.5, status=status, **kw), *want, "merged")
    assert status.item() == 0


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_long_context_cut(kv):
    """Few rows, contexts cut over many CTAs, the tree itself across a tile's end."""
    lens, n = [9000, 3967, 128 * 30 + 3], 12
    c = Cache(lens, 2, 128, 16, kv, seed=3)
    q = _queries(3, n, 8, 128)
    mask, seen = random_trees([n] * 3, 4, n, seed=2)
    check(_call(c, q, mask.cuda(), 0.09), *tree_reference(c, q, seen, [n] * 3, 0.09))


def test_masks_of_any_shape():
    """Masks that leave a node nothing, that see later nodes, all and none; bits past the tree."""
    n, lens = 9, [9, 9, 40, 150]
    c = Cache(lens, 2, 64, 16, seed=1)
    q = _queries(4, n, 4, 64)
    gen = torch.Generator().manual_seed(5)
    mask = torch.randint(0, 1 << n, (4, n, 1), generator=gen)
    mask[:, 0] = 0
    mask[:, 1] = (1 << n) - 1
    sizes = [9, 6, 9, 4]
    seen = [(mask[s, :t] >> torch.arange(t)) & 1 == 1 for s, t in enumerate(sizes)]
    mask = mask | (-1 << 40)                  # bits past every node
    want = tree_reference(c, q, seen, sizes, 0.125)
    assert (want[0][0, 0] == 0).all()         # sees nothing: zeros
    got = _call(c, q, mask.cuda(), 0.125, tree_lens=_sizes(sizes))
    check(got, *want)
    assert (got[1, 6:] == 0).all() and (got[3, 4:] == 0).all() and (got[0, 0] == 0).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [2, 16, 70])
def test_chain_is_multi(kv, n):
    """A chain gives what the multi-query decode gives, within both bounds."""
    import paged_kv_decode_02_gb300 as pk
    lens = [n, 200, 333]
    c = Cache(lens, 2, 128, 16, kv, seed=n)
    q = _queries(3, n, 8, 128, seed=n)
    seen = [torch.ones(n, n, dtype=torch.bool).tril()] * 3
    words = (n + 63) // 64
    mask = torch.zeros(3, n, words, dtype=torch.int64)
    for i in range(n):
        for j in range(i + 1):
            mask[:, i, j // 64] |= (1 << (j % 64)) - (1 << 64 if j % 64 == 63 else 0)
    out, bound = tree_reference(c, q, seen, [n] * 3, 0.09)
    check(_call(c, q, mask.cuda(), 0.09), out, bound)
    if kv == "bf16":
        multi = pk.paged_decode_attention_multi(q, *c.caches, c.tables, c.context_lens, 0.09)
        check(multi, out, bound)


def test_negative_and_zero_scale():
    lens, n = [50, 300], 6
    c = Cache(lens, 1, 64, 16, seed=4)
    q = _queries(2, n, 8, 64)
    mask, seen = random_trees([n] * 2, 3, n)
    for scale in (-0.125, 0.0):
        check(_call(c, q, mask.cuda(), scale), *tree_reference(c, q, seen, [n] * 2, scale))


def test_status_flags():
    """Lengths and blocks that do not fit: flagged, zeros; the others are computed."""
    from paged_kv_decode_02_gb300 import pagedkv
    n, lens = 4, [60, 60, 60]
    c = Cache(lens, 2, 64, 16, seed=1)
    q = _queries(3, n, 4, 64)
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
    assert run(tree_lens=_sizes([4, 5, 4])) == bad
    assert run(tree_lens=_sizes([4, -1, 4])) == bad
    c.context_lens[1] = 3
    assert run() == bad
    c.context_lens[1] = 100
    assert run() == bad
    c.context_lens[1] = 60
    c.tables[1, 2] = c.nb
    assert run() == pagedkv.DEV_BAD_BLOCK_ID


def test_same_bits_and_graph():
    import paged_kv_decode_02_gb300 as pk
    lens, n = [500, 90, 1400], 10
    c = Cache(lens, 2, 128, 16, seed=6)
    q = _queries(3, n, 16, 128)
    mask, seen = random_trees([n] * 3, 4, n)
    mask = mask.cuda()
    first = _call(c, q, mask, 0.09)
    for _ in range(3):
        assert torch.equal(first, _call(c, q, mask, 0.09))
    ws = torch.empty(pk.tree_workspace_bytes(3, 16, 2, 128, 16, c.nb, c.tables.shape[1], n),
                     dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(c, q, mask, 0.09, out=out, workspace=ws)
    graph.replay()
    assert torch.equal(first, out)
    mask2, seen = random_trees([n] * 3, 2, n, seed=9)
    mask.copy_(mask2)
    graph.replay()
    check(out, *tree_reference(c, q, seen, [n] * 3, 0.09))
