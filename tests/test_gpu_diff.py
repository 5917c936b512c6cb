"""GPU differential decode against the fp64 oracle, within bounds derived per element."""

import numpy as np
import pytest
import torch

import oracle
from diff_helpers import assert_diff, diff_reference, random_lambda, random_norm
from paged_kv_decode_02_gb300.workloads import make_workload

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pk():
    from paged_kv_decode_02_gb300 import build_lib
    build_lib.build()
    import paged_kv_decode_02_gb300 as pk
    pk.load_library()
    return pk


def call(pk, w, lam, **kw):
    if w.kv_dtype == "bf16":
        return pk.paged_decode_attention_diff(w.q, w.k_cache, w.v_cache, w.block_tables,
                                              w.context_lens, lam, w.scale, **kw)
    return pk.paged_decode_attention_diff_q8(w.q, w.k_cache, w.v_cache, w.k_scale, w.v_scale,
                                             w.block_tables, w.context_lens, lam, w.scale,
                                             fmt=w.kv_dtype[4:] if "fp8" in w.kv_dtype else "e4m3",
                                             **kw)


def build(kv, lengths, hq, hkv, d, bs, **kw):
    name = {"bf16": "70b-gqa", "int8": "int8"}.get(kv, "fp8-" + kv[4:])
    return make_workload(name, device=DEV, lengths=lengths, num_q_heads=hq, num_kv_heads=hkv,
                         head_dim=d, block_size=bs, **kw)


LENGTHS = [1, 0, 15, 16, 17, 31, 32, 33, 100, 333]


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8_e4m3", "fp8_e5m2"])
@pytest.mark.parametrize("d,bs", [(128, 16), (128, 32), (64, 16), (64, 32)])
@pytest.mark.parametrize("hq,hkv,norm", [(8, 4, True), (4, 4, False), (32, 2, True)])
def test_diff_small(pk, kv, d, bs, hq, hkv, norm):
    """Every cache type, head size and block size; one, two and sixteen query pairs per KV
    pair; an empty sequence, single tokens and tails on every side of a tile's edge; unused
    rows hold NaN."""
    w = build(kv, LENGTHS, hq, hkv, d, bs, poison_unused=True)
    lam = random_lambda(hq, DEV)
    nw = random_norm(d, DEV) if norm else None
    kw = dict(norm_weight=nw, eps=1e-5, out_scale=0.6)
    out = call(pk, w, lam, **kw)
    torch.cuda.synchronize()
    ref, bound = diff_reference(w, lam, nw, 1e-5, 0.6)
    assert_diff(out, ref, bound)
    assert torch.all(out[1] == 0)                            # the empty sequence


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8_e5m2"])
@pytest.mark.parametrize("hq,hkv", [(6, 2), (10, 2), (14, 2), (16, 2), (18, 2), (26, 2), (32, 2),
                                    (34, 2), (40, 2)])
def test_diff_group_sizes(pk, kv, hq, hkv):
    """Groups of 3, 5, 7, 8, 9, 13 and 16 query pairs in one unit; 17 and 20 in two, the
    second one partly filled (17: 9 and 8)."""
    w = build(kv, [40, 7, 129], hq, hkv, 64, 16)
    lam = random_lambda(hq, DEV)
    nw = random_norm(64, DEV)
    out = call(pk, w, lam, norm_weight=nw)
    ref, bound = diff_reference(w, lam, nw, 1e-5)
    assert_diff(out, ref, bound)


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("hq", [16, 20, 32])
def test_diff_large_groups_split(pk, kv, hq):
    """Groups of 8, 10 and 16 query pairs over contexts cut between many CTAs, head_dim 128."""
    w = build(kv, [1200, 31, 650], hq, 2, 128, 32)
    lam = random_lambda(hq, DEV)
    nw = random_norm(128, DEV)
    out = call(pk, w, lam, norm_weight=nw, out_scale=0.3)
    ref, bound = diff_reference(w, lam, nw, 1e-5, 0.3)
    assert_diff(out, ref, bound)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_diff_long_and_split(pk, kv):
    """One long sequence cut over the whole GPU, and a long one among short ones."""
    for lengths in ([9001], [5000, 3, 1, 64, 700]):
        w = build(kv, lengths, 4, 2, 128, 16)
        lam = random_lambda(4, DEV)
        nw = random_norm(128, DEV)
        out = call(pk, w, lam, norm_weight=nw, out_scale=0.2)
        ref, bound = diff_reference(w, lam, nw, 1e-5, 0.2)
        assert_diff(out, ref, bound)


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("int8", 128), ("fp8_e5m2", 64)])
@pytest.mark.parametrize("lengths,hq,hkv", [([9000], 2, 2), ([5000], 34, 2), ([7000, 0, 40], 64, 2),
                                            ([2500, 1, 0, 1700, 33], 28, 4),
                                            ([900, 1100, 0, 1000] * 6, 28, 4)])
def test_diff_few_pairs_many_records(pk, kv, d, lengths, hq, hkv):
    """One unit cut over most of the GPU; 32 and up to 384 query pairs, empty sequences among
    them: with and without a norm, with a status word, on a workspace of NaN, twice the same."""
    w = build(kv, lengths, hq, hkv, d, 16)
    lam, nw = random_lambda(hq, DEV), random_norm(d, DEV)
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for more in (dict(), dict(norm_weight=nw, eps=1e-5, out_scale=0.7)):
        out = call(pk, w, lam, workspace=ws, status=status, **more)
        ref, bound = diff_reference(w, lam, more.get("norm_weight"), more.get("eps", 0.0),
                                    more.get("out_scale", 1.0))
        assert_diff(out, ref, bound)
        assert status.item() == 0
        assert torch.equal(out, call(pk, w, lam, **more))
    w.block_tables[0, 3] = -1
    out = call(pk, w, lam, workspace=ws, status=status)
    assert status.item() == pk.pagedkv.DEV_BAD_BLOCK_ID and not out[0].any()


@pytest.mark.parametrize("kv,hq,hkv,d", [("bf16", 8, 8, 64), ("int8", 16, 8, 128),
                                         ("bf16", 48, 4, 64), ("fp8_e4m3", 8, 8, 128)])
def test_diff_more_units_than_ctas(pk, kv, hq, hkv, d):
    """Most units whole, some cut: with empty sequences, a bad page, a bad length, a status word
    and without."""
    lengths = [(37 * i) % 201 if i % 9 else 0 for i in range(300)]
    w = build(kv, lengths, hq, hkv, d, 16)
    lam, nw = random_lambda(hq, DEV), random_norm(d, DEV)
    ref, bound = diff_reference(w, lam, nw, 1e-5, 0.5)
    more = dict(norm_weight=nw, eps=1e-5, out_scale=0.5)
    out = torch.full((300, hq // 2, 2 * d), float("nan"), dtype=torch.bfloat16, device=DEV)
    assert_diff(call(pk, w, lam, out=out, **more), ref, bound)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    good = call(pk, w, lam, status=status, **more)
    assert status.item() == 0 and torch.equal(good, out)
    w.block_tables[[10, 100, 215], 0] = 1 << 30
    w.context_lens[150] = -3
    w.context_lens[151] = w.block_tables.shape[1] * 16 + 1
    got = call(pk, w, lam, status=status, **more)
    assert status.item() == pk.pagedkv.DEV_BAD_BLOCK_ID | pk.pagedkv.DEV_BAD_CONTEXT_LEN
    bad = torch.zeros(300, dtype=torch.bool, device=DEV)
    bad[[10, 100, 215, 150, 151]] = True
    assert not got[bad].any()
    # the rest as before (where cuts fall moves with the lengths: within the bound, not the bits)
    ref[bad.cpu().numpy()] = 0.0
    assert_diff(got, ref, bound)


def test_diff_batches_of_short_sequences(pk):
    """No unit longer than the streams of a CTA take at once: no unit is cut."""
    for n in (3, 90, 300):
        w = build("bf16", [(7 * i) % 65 for i in range(n)], 8, 4, 64, 16)
        lam = random_lambda(8, DEV)
        ref, bound = diff_reference(w, lam)
        assert_diff(call(pk, w, lam), ref, bound)


def test_diff_many_units_per_cta(pk):
    """More units than CTAs, most of them one item long: a CTA folds and writes many."""
    lengths = [1 + (7 * i) % 50 for i in range(200)]
    w = build("bf16", lengths, 16, 8, 64, 16)
    lam = random_lambda(16, DEV)
    out = call(pk, w, lam)
    ref, bound = diff_reference(w, lam)
    assert_diff(out, ref, bound)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_diff_large_batches_and_empty_ones(pk, kv):
    """More sequences than threads of a CTA, many of them empty; a batch without any token; a
    table of one block."""
    lengths = [(5 * i) % 4 for i in range(1500)]
    w = build(kv, lengths, 4, 2, 64, 16)
    lam = random_lambda(4, DEV)
    out = call(pk, w, lam, out_scale=2.0)
    ref, bound = diff_reference(w, lam, out_scale=2.0)
    assert_diff(out, ref, bound)
    w.context_lens.zero_()
    assert torch.all(call(pk, w, lam, out=torch.ones_like(out)) == 0)
    one = build(kv, [16, 3], 4, 2, 128, 32)
    assert one.block_tables.shape[1] == 1
    out = call(pk, one, lam)
    ref, bound = diff_reference(one, lam)
    assert_diff(out, ref, bound)


@pytest.mark.parametrize("kv", ["int8", "fp8_e4m3", "fp8_e5m2"])
def test_diff_small_and_large_values(pk, kv):
    """V rows of absmax 1e-3 and of 3e4 (fp16 weights times V scales neither vanish nor
    overflow), q and K rows far from 1."""
    for vmul, qmul in ((1e-3 / 3, 2.0 ** 20), (1e4, 2.0 ** -20)):
        w = build(kv, [70, 33], 8, 4, 128, 16)
        w.v_scale *= vmul
        w.q = (w.q.float() * qmul).to(torch.bfloat16)
        w.k_scale /= qmul
        lam = random_lambda(8, DEV)
        out = call(pk, w, lam)
        ref, bound = diff_reference(w, lam)
        assert_diff(out, ref, bound)


def test_diff_float8_tensors_are_their_bytes(pk):
    for kv, dt in (("fp8_e4m3", torch.float8_e4m3fn), ("fp8_e5m2", torch.float8_e5m2)):
        w = build(kv, [70, 33], 8, 4, 64, 16)
        lam = random_lambda(8, DEV)
        want = call(pk, w, lam)
        w.k_cache, w.v_cache = w.k_cache.view(dt), w.v_cache.view(dt)
        assert torch.equal(call(pk, w, lam), want)


def test_diff_first_call_of_a_shape_inside_a_capture(pk):
    w = build("bf16", [300, 11], 12, 6, 64, 32)              # a shape no other test plans
    lam = random_lambda(12, DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(pk, w, lam)
    out.fill_(1.0)
    g.replay()
    assert torch.equal(out, call(pk, w, lam))


def test_diff_growing_and_huge_scores(pk):
    """Scores that grow from tile to tile rescale every state; rows of one head far above the
    other's keep apart."""
    w = build("bf16", [400, 65], 8, 4, 128, 16)
    grow = torch.linspace(0.1, 6.0, 400, device=DEV)
    for s, L in enumerate((400, 65)):
        t = torch.arange(L, device=DEV)
        blk, off = w.block_tables[s, t // 16].long(), t % 16
        w.k_cache[blk, :, off] = (w.k_cache[blk, :, off].float() *
                                  grow[:L, None, None]).to(torch.bfloat16)
        w.k_cache[blk, 1, off] = (w.k_cache[blk, 1, off].float() * 0.25).to(torch.bfloat16)
    lam = random_lambda(8, DEV)
    out = call(pk, w, lam)
    ref, bound = diff_reference(w, lam)
    assert_diff(out, ref, bound)


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8_e4m3", "fp8_e5m2"])
def test_diff_nan_stays_in_its_rows(pk, kv):
    """A NaN in a query row, or in a cached K row, makes the pairs that read it NaN, in units
    of one CTA and in cut ones, and no other pair."""
    w = build(kv, [7, 40, 6000], 8, 4, 128, 16)
    lam = torch.linspace(0.2, 0.8, 4, device=DEV)
    clean = call(pk, w, lam)
    assert torch.isfinite(clean).all()
    q = w.q.clone()
    w.q[:, 3, 5] = float("nan")              # second map of query pair 1
    out = call(pk, w, lam)
    assert torch.isnan(out[:, 1]).all()
    assert torch.equal(out[:, [0, 2, 3]], clean[:, [0, 2, 3]])
    w.q.copy_(q)
    if kv != "bf16":
        w.k_scale[w.block_tables[:, 0].long(), 3, 2] = float("nan")  # KV pair 1: pairs 2, 3
    else:
        w.k_cache[w.block_tables[:, 0].long(), 3, 2, 9] = float("nan")
    out = call(pk, w, lam)
    assert torch.isnan(out[:, 2:]).all()
    assert torch.equal(out[:, :2], clean[:, :2])


def test_diff_scores_of_minus_infinity(pk):
    """Tokens whose score is -inf have no weight; a map that has no other gives NaN."""
    lengths = [40, 300, 6000]
    w = build("bf16", lengths, 8, 4, 128, 16)
    w.q[:, :, 0] = 1.0
    for s, L in enumerate(lengths):
        gone = torch.cat([torch.arange(0, 37), torch.arange(38, L, 3)]).to(DEV)
        w.k_cache[w.block_tables[s, gone // 16].long(), :, gone % 16, 0] = float("-inf")
    lam = random_lambda(8, DEV)
    ref, bound = diff_reference(w, lam)
    assert_diff(call(pk, w, lam), ref, bound)
    w.k_cache[..., 0] = float("-inf")
    assert torch.isnan(call(pk, w, lam)).all()


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_diff_far_blocks(pk, kv):
    """Blocks more than 2^32 bytes into the cache give what the same rows give near its
    start."""
    w = build(kv, [100, 3000], 16, 8, 128, 16)
    lam = random_lambda(16, DEV)
    near = call(pk, w, lam)
    n, block_bytes = w.k_cache.shape[0], w.k_cache[0].numel() * w.k_cache.element_size()
    far = 2 ** 32 // block_bytes + 5
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        old = getattr(w, name)
        if old is None:
            continue
        new = torch.zeros((far + n,) + tuple(old.shape[1:]), dtype=old.dtype, device=DEV)
        new[far:] = old
        setattr(w, name, new)
    w.block_tables += far
    assert torch.equal(call(pk, w, lam), near)


def test_diff_lambda_zero_is_plain_decode(pk):
    """lambda 0: the first map alone, as the plain decode of the even heads over each value
    head gives it (both within their rounding: two halves of a bf16 step)."""
    w = build("bf16", [100, 47, 300], 8, 8, 128, 16)
    out = call(pk, w, torch.zeros(4, device=DEV))
    k2 = w.k_cache[:, 0::2].repeat_interleave(2, 1).contiguous()
    q2 = w.q[:, 0::2].repeat_interleave(2, 1).contiguous()
    plain = pk.paged_decode_attention(q2, k2, w.v_cache, w.block_tables, w.context_lens, w.scale)
    a, b = out.float().view(3, 8, 128), plain.float()
    ref, bound = diff_reference(w, torch.zeros(4, device=DEV))
    room = torch.from_numpy(2 * bound).to(DEV).float().view(3, 8, 128)
    assert torch.all((a - b).abs() <= room)


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_diff_status_and_bad_tables(pk, kv):
    """With a status word bad sequences are flagged and zeroed, the others as without one;
    without it nothing faults. (Ids are clamped into the pool before any copy.)"""
    w = build(kv, [40, 100, 64, 20], 8, 4, 64, 16)
    lam = random_lambda(8, DEV)
    good = call(pk, w, lam)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    same = call(pk, w, lam, status=status)
    assert int(status) == 0 and torch.equal(good, same)
    w.block_tables[1, 2] = w.k_cache.shape[0]
    w.block_tables[2, 0] = -5
    w.context_lens[3] = w.block_tables.shape[1] * 16 + 1
    out = call(pk, w, lam, status=status)
    assert int(status) == 0x1 | 0x2
    assert torch.equal(out[0], good[0]) and torch.all(out[1:] == 0)
    assert torch.equal(call(pk, w, lam)[0], good[0])
    status.zero_()
    w.context_lens[3] = -7
    out = call(pk, w, lam, status=status)
    assert int(status) == 0x1 | 0x2 and torch.all(out[3] == 0)


def test_diff_repeats_bit_for_bit_on_dirty_workspace_and_in_graphs(pk):
    """The same call twice, over a workspace full of NaN, on another stream, and captured and
    replayed next to another captured call that shares the workspace: the same bits."""
    w = build("bf16", [700, 40, 1500], 8, 4, 128, 16)
    w2 = build("bf16", [90, 800], 8, 4, 128, 32)
    lam = random_lambda(8, DEV)
    need = max(pk.diff_workspace_bytes(len(x.context_lens), 8, 4, 128, x.block_size,
                                       x.k_cache.shape[0], x.block_tables.shape[1])
               for x in (w, w2))
    ws = torch.full((need // 4,), float("nan"), device=DEV)
    first, first2 = call(pk, w, lam), call(pk, w2, lam)
    assert torch.equal(call(pk, w, lam, workspace=ws), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = call(pk, w, lam, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again, first)
    out, out2 = torch.empty_like(first), torch.empty_like(first2)
    graphs = []
    for x, o in ((w, out), (w2, out2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(pk, x, lam, out=o, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        out.fill_(1.0)
        out2.fill_(1.0)
        graphs[0].replay()
        graphs[1].replay()
        assert torch.equal(out, first) and torch.equal(out2, first2)


def test_diff_writes_nothing_else(pk):
    """Guards around the output and around a workspace of exactly the requested size."""
    w = build("int8", [300, 17, 0, 64], 8, 4, 128, 32)
    lam = random_lambda(8, DEV)
    want = call(pk, w, lam)
    need = pk.diff_workspace_bytes(4, 8, 4, 128, 32, w.k_cache.shape[0], w.block_tables.shape[1],
                                   kv_dtype=1)
    pad = 4096
    ws = torch.full((need + 2 * pad,), 0xA5, dtype=torch.uint8, device=DEV)
    buf = torch.full((want.numel() + pad,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[pad // 2:pad // 2 + want.numel()].view(want.shape)
    for _ in range(2):
        call(pk, w, lam, out=out, workspace=ws[pad:pad + need])
    assert torch.equal(out, want)
    assert torch.all(ws[:pad] == 0xA5) and torch.all(ws[pad + need:] == 0xA5)
    assert torch.all(buf[:pad // 2] == 7.0) and torch.all(buf[pad // 2 + want.numel():] == 7.0)


def test_diff_argument_checks(pk):
    w = build("bf16", [40, 100], 8, 4, 64, 16)
    lam = random_lambda(8, DEV)
    with pytest.raises(ValueError):
        call(pk, w, lam[:3])
    with pytest.raises(ValueError):
        call(pk, w, lam, norm_weight=random_norm(128, DEV))
    with pytest.raises(TypeError):
        call(pk, w, lam.double())
    with pytest.raises(ValueError):
        call(pk, w, lam, out=torch.empty_like(w.q))
    with pytest.raises(pk.PagedKVError):                     # an odd number of KV heads
        pk.paged_decode_attention_diff(w.q[:, :6].contiguous(), w.k_cache[:, :3].contiguous(),
                                       w.v_cache[:, :3].contiguous(), w.block_tables,
                                       w.context_lens, lam[:3].contiguous(), w.scale)
