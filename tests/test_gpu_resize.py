"""Resize of sequences and the move of kept tokens, against lists and row by row."""

import numpy as np
import pytest
import torch

from serve_helpers import Cache, Pool

pytestmark = pytest.mark.gpu


class State:
    """Device state of a batch and the same as lists."""

    def __init__(self, lens, bs, mbs, num_blocks, seed=0, capacity=None):
        ids = np.random.default_rng(seed).permutation(num_blocks).astype(np.int32)
        held = [-(-n // bs) for n in lens]
        tables = np.full((len(lens), mbs), -5, np.int32)
        at = 0
        for s, h in enumerate(held):
            tables[s, :h] = ids[at:at + h]
            at += h
        free = np.full(num_blocks if capacity is None else capacity, -9, np.int32)
        free[:num_blocks - at] = ids[at:]
        put = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.bs = bs
        self.tables, self.lens, self.free = put(tables), put(lens), put(free)
        self.count = put([num_blocks - at])
        self.pool = Pool(lens, bs, mbs, ids[at:].tolist(), tables.tolist())

    def resize(self, targets, num_tokens, **kw):
        import paged_kv_decode_02_gb300 as pk
        from paged_kv_decode_02_gb300 import pagedkv
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = pk.paged_kv_resize(self.tables, self.lens,
                                 torch.tensor(targets, dtype=torch.int32, device="cuda"),
                                 self.free, self.count, self.bs, num_tokens=num_tokens,
                                 status=status, **kw)
        *want, short = self.pool.resize(targets, num_tokens)
        for g, w in zip(got, want):
            assert g.tolist() == w
        self.check()
        assert bool(status.item() & pagedkv.DEV_NO_BLOCKS) == short
        return status.item()

    def check(self):
        assert self.lens.tolist() == self.pool.lens
        assert self.tables.tolist() == self.pool.tables
        n = self.count.item()
        assert self.free[:n].tolist() == self.pool.free


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("seqs", [1, 3, 33, 700, 2500])
def test_random_walk(seqs, bs):
    """Steps of growth by one, prompts, drafts, shrinking and finishing, mixed in one call."""
    r = np.random.default_rng(seqs + bs)
    most = 12
    s = State([int(x) for x in r.integers(0, 70, seqs)], bs, most, seqs * most, seed=seqs)
    for step in range(8):
        old = np.array(s.pool.lens)
        kind = r.integers(0, 5, seqs)
        new = np.where(kind == 0, old + 1, np.where(kind == 1, old + r.integers(0, 90, seqs),
                       np.where(kind == 2, 0, np.where(kind == 3, old // 2, old))))
        new = np.minimum(new, most * bs)
        grown = int(np.maximum(new - old, 0).sum())
        assert s.resize([int(x) for x in new], grown + (step % 3) * 7) == 0


def test_grow_and_back_restores():
    s = State([5, 0, 31, 16], 16, 20, 90, seed=4)
    free, count = s.free.clone(), s.count.clone()
    assert s.resize([300, 7, 32, 16], 500) == 0
    assert s.resize([5, 0, 31, 16], 0) == 0
    assert torch.equal(free, s.free) and torch.equal(count, s.count)


def test_blocks_given_back_serve_the_same_call():
    """No free block: what the last sequence gives up goes to the first one."""
    s = State([16, 16, 64], 16, 4, 6)
    assert s.count.item() == 0
    assert s.resize([40, 16, 16], 24) == 0
    assert s.count.item() == 1


def test_blocks_run_out():
    from paged_kv_decode_02_gb300 import pagedkv
    s = State([16, 16, 16, 10, 0], 16, 8, 6)       # two free blocks
    # the first takes one, the second needs two and stays, so does the third; the fourth needs
    # none and grows; the fifth stays
    assert s.resize([17, 48, 17, 16, 1], 100) == pagedkv.DEV_NO_BLOCKS
    assert s.pool.lens == [17, 16, 16, 16, 0]
    assert s.resize([0, 48, 17, 16, 0], 40) == 0


def test_token_rows_run_out():
    from paged_kv_decode_02_gb300 import pagedkv
    s = State([3, 3, 3], 16, 8, 24)
    assert s.resize([10, 30, 4], 20) == pagedkv.DEV_NO_BLOCKS
    assert s.pool.lens == [10, 3, 3]


def test_bad_lengths():
    """A length past the table row or negative: the sequence stays, the others go on."""
    from paged_kv_decode_02_gb300 import pagedkv
    s = State([3, 5, 7], 16, 4, 12)
    assert s.resize([20, 65, 9], 40) == pagedkv.DEV_BAD_CONTEXT_LEN
    assert s.resize([20, -1, 64], 80) == pagedkv.DEV_BAD_CONTEXT_LEN
    assert s.resize([21, 2 ** 31 - 1, 64], 80) == pagedkv.DEV_BAD_CONTEXT_LEN


def test_bad_free_list():
    """A count past the list is taken as its end; blocks past its capacity are lost, never written
    out of range."""
    import paged_kv_decode_02_gb300 as pk
    from paged_kv_decode_02_gb300 import pagedkv
    put = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    room = put([9] * 8)
    free, count, status = room[:4], put([7]), put([0])
    tables, lens = put([[1, 2, 3, 4]]), put([0])
    pk.paged_kv_resize(tables, lens, put([33]), free, count, 16, num_tokens=33, status=status)
    assert status.item() == pagedkv.DEV_NO_BLOCKS and count.item() == 1 and lens.item() == 33
    status.zero_()
    count.fill_(3)
    pk.paged_kv_resize(tables, lens, put([0]), free, count, 16, status=status)
    assert status.item() == pagedkv.DEV_NO_BLOCKS and count.item() == 4
    assert room[4:].tolist() == [9] * 4


def test_most_sequences_and_refusal():
    import paged_kv_decode_02_gb300 as pk
    s = State([0] * 16384, 16, 1, 16384)
    assert s.resize([1] * 16384, 16384) == 0
    z = torch.zeros(16385, dtype=torch.int32, device="cuda")
    with pytest.raises(pk.PagedKVError):
        pk.paged_kv_resize(torch.zeros(16385, 1, dtype=torch.int32, device="cuda"), z, z + 1,
                           z, z[:1].clone(), 16)
    with pytest.raises(pk.PagedKVError):
        s.bs = 24
        s.resize([1] * 16384, 0)


def test_long_prompts():
    s = State([0, 40000, 3], 32, 4096, 9000)
    assert s.resize([100001, 1, 60000], 170000) == 0


def test_resize_in_a_graph():
    """Captured once, replayed while the targets change."""
    import paged_kv_decode_02_gb300 as pk
    s = State([5, 100, 0], 16, 20, 60)
    target = s.lens.clone()
    slots = torch.empty(64, dtype=torch.int64, device="cuda")
    pos, off = slots.clone(), torch.empty(4, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.paged_kv_resize(s.tables, s.lens, target, s.free, s.count, 16, slot_mapping=slots,
                           positions=pos, token_offsets=off)
    for new in ([6, 101, 16], [7, 90, 50], [0, 92, 51], [40, 93, 0]):
        target.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        a, b, c, _ = s.pool.resize(new, 64)
        assert (slots.tolist(), pos.tolist(), off.tolist()) == (a, b, c)
        s.check()


# ---------------------------------------------------------------------------
# kept tokens
# ---------------------------------------------------------------------------

def _moved(c, base, path, kept):
    """Both caches and scales after the moves, row by row on the host."""
    tables = c.tables.cpu().numpy()
    arrays = [x.cpu().clone() for x in c.caches + [x for x in c.scales if x is not None]]
    for x in arrays:
        old = x.clone()
        for s in range(len(base)):
            for i in range(kept[s]):
                a, b = base[s] + path[s][i], base[s] + i
                x[tables[s, b // c.bs], :, b % c.bs] = old[tables[s, a // c.bs], :, a % c.bs]
    return arrays


def _same(got, want):
    for g, w in zip(got, want):
        assert torch.equal(g.cpu().view(torch.uint8), w.view(torch.uint8))


def _keep(c, base, path, kept, status=None):
    import paged_kv_decode_02_gb300 as pk
    put = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pk.paged_kv_keep(*c.caches, c.tables, put(base), put(path),
                     None if kept is None else put(kept), k_scale=c.scales[0],
                     v_scale=c.scales[1], status=status)
    return c.caches + [x for x in c.scales if x is not None]


@pytest.mark.parametrize("kv", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("hkv,d,bs", [(1, 64, 16), (3, 128, 32), (8, 128, 16)])
@pytest.mark.parametrize("width", [1, 5, 40, 200])
def test_keep(kv, hkv, d, bs, width):
    """Random rising paths: from none to all of the draft, sources and places overlapping."""
    r = np.random.default_rng(width + hkv)
    base = [0, 3, bs - 1, 77, 10]
    draft = width + 30
    c = Cache([b + draft for b in base], hkv, d, bs, kv, seed=width)
    path = [sorted(r.choice(draft, width, replace=False).tolist()) for _ in base]
    path[1] = list(range(width))                        # nothing moves
    path[2] = list(range(1, width + 1))                 # everything, by one
    kept = [width, width, width, 0, width // 2]
    want = _moved(c, base, path, kept)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _same(_keep(c, base, path, kept, status), want)
    assert status.item() == 0


def test_keep_without_lengths():
    c = Cache([50, 60], 2, 64, 16, seed=2)
    base, path = [20, 30], [[1, 4, 9], [0, 7, 8]]
    want = _moved(c, base, path, [3, 3])
    _same(_keep(c, base, path, None), want)


def test_keep_refuses_bad_paths():
    """Paths that do not rise, leave the table row or meet a bad block leave the sequence alone."""
    from paged_kv_decode_02_gb300 import pagedkv
    bad = pagedkv.DEV_BAD_CONTEXT_LEN
    for base, path, kept, flag in (
            ([5, 5], [[1, 1, 3], [2, 5, 6]], [3, 3], bad),
            ([5, 5], [[3, 2, 4], [2, 5, 6]], [3, 3], bad),
            ([5, 5], [[-1, 2, 4], [2, 5, 6]], [3, 3], bad),
            ([5, 5], [[1, 2, 80], [2, 5, 6]], [3, 3], bad),
            ([5, 5], [[1, 2, 2 ** 31 - 1], [2, 5, 6]], [3, 3], bad),
            ([-1, 5], [[1, 2, 4], [2, 5, 6]], [3, 3], bad),
            ([5, 5], [[1, 2, 4], [2, 5, 6]], [4, 3], bad),
            ([5, 5], [[1, 2, 4], [2, 5, 6]], [-1, 3], bad),
            ([5, 5], [[1, 2, 40], [2, 5, 6]], [3, 3], pagedkv.DEV_BAD_BLOCK_ID)):
        c = Cache([30, 80], 2, 64, 16, seed=3)          # row 0's entries end at 2: then -7
        want = _moved(c, base, path, [0, 3])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        _same(_keep(c, base, path, kept, status), want)
        assert status.item() == flag


def test_empty_batch():
    """No sequences: rows that the appends skip, offsets of zero."""
    import paged_kv_decode_02_gb300 as pk
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    slots, positions = (torch.full((5,), 7, dtype=torch.int64, device="cuda") for _ in range(2))
    offs = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    pk.paged_kv_resize(torch.empty(0, 4, dtype=torch.int32, device="cuda"), none, none.clone(),
                       torch.zeros(3, dtype=torch.int32, device="cuda"),
                       torch.ones(1, dtype=torch.int32, device="cuda"), 16, 5, slots, positions,
                       offs)
    assert (slots == -1).all() and (positions == 0).all() and offs.item() == 0
