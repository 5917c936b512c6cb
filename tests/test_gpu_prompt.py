"""Prompt attention (causal, packed, grouped heads) against the definition in 64 bits."""

import pytest
import torch

from serve_helpers import check, offsets, prompt_reference

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _rows(n, heads, d, gen):
    return torch.randn(n, heads, d, generator=gen, device="cuda").to(BF)


def _inputs(hq, hkv, d, q_lens, kv_lens, seed=0, fused=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if fused:
        qkv = _rows(sum(q_lens), hq + 2 * hkv, d, gen)
        return qkv.split([hq, hkv, hkv], 1)
    return (_rows(sum(q_lens), hq, d, gen), _rows(sum(kv_lens), hkv, d, gen),
            _rows(sum(kv_lens), hkv, d, gen))


def _run(q, k, v, q_lens, kv_lens, scale, **kw):
    import paged_kv_decode_02_gb300 as pk
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pk.prompt_attention(q, k, v, offsets(q_lens), scale, kv_offsets=offsets(kv_lens),
                              status=status, **kw)
    assert status.item() == 0
    return out


SHAPES = [
    # one token; one tile and its neighbours; odd lengths
    ([1], [1]), ([3], [3]), ([127], [127]), ([128], [128]), ([129], [129]), ([300], [300]),
    # ragged packs, empty sequences among them
    ([5, 0, 130, 1, 64], [5, 0, 130, 1, 64]),
    ([0, 0, 7], [0, 0, 7]),
    # chunks over longer contexts; one token of a long context; fewer keys than queries; none
    ([16, 1, 40], [500, 1000, 41]), ([1, 1], [2048, 3]), ([9, 20], [4, 0]), ([12], [0]),
    # stretches cut between CTAs
    ([1500], [1500]), ([33, 700, 2], [900, 700, 3000]),
]


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 64), (8, 1, 128), (6, 2, 128), (5, 1, 64)])
@pytest.mark.parametrize("lens", SHAPES, ids=[f"{a}-{b}" for a, b in SHAPES])
def test_lengths(lens, hq, hkv, d):
    q_lens, kv_lens = lens
    q, k, v = _inputs(hq, hkv, d, q_lens, kv_lens, seed=len(q_lens) + q_lens[0])
    got = _run(q, k, v, q_lens, kv_lens, d ** -0.5)
    check(got, *prompt_reference(q, k, v, q_lens, kv_lens, d ** -0.5))


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 8, 11, 12, 16, 33, 64, 100, 128])
def test_groups(group):
    """Every way that a group of heads fills the tile's 128 rows."""
    q_lens, kv_lens = [70, 1, 131], [70, 200, 131]
    q, k, v = _inputs(2 * group, 2, 64, q_lens, kv_lens, seed=group)
    got = _run(q, k, v, q_lens, kv_lens, 0.125)
    check(got, *prompt_reference(q, k, v, q_lens, kv_lens, 0.125))


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (14, 2, 64)])
def test_fused_projection(hq, hkv, d):
    """q, k and v as parts of one projection's rows, out with a stride of its own; rows past the
    last sequence stay as they were, whatever stands there."""
    lens = [311, 17, 640]
    n = sum(lens)
    q, k, v = _inputs(hq, hkv, d, lens + [50], None, seed=3, fused=True)
    q[n:], k[n:], v[n:] = float("nan"), float("nan"), float("nan")
    room = torch.full((n + 50, hq + 3, d), 7.0, device="cuda", dtype=BF)
    out = room[:, 1:1 + hq]
    import paged_kv_decode_02_gb300 as pk
    got = pk.prompt_attention(q, k, v, offsets(lens), d ** -0.5, out=out)
    assert got is out
    check(out[:n], *prompt_reference(q[:n], k[:n], v[:n], lens, lens, d ** -0.5))
    assert (room[n:] == 7).all() and (room[:, 0] == 7).all() and (room[:, 1 + hq:] == 7).all()


def test_neighbours_may_hold_anything():
    """NaN and infinite keys and values of one sequence stay out of the next one's tiles."""
    lens = [100, 90, 60]
    q, k, v = _inputs(4, 2, 64, lens, lens, seed=9)
    want = prompt_reference(q, k, v, lens, lens, 0.125)
    q, k, v = q.clone(), k.clone(), v.clone()
    for t in (q, k, v):
        t[100:150] = float("nan")
        t[150:190] = float("inf")
    got = _run(q, k, v, lens, lens, 0.125)
    for a, b in ((0, 100), (190, 250)):
        check(got[a:b], want[0][a:b], want[1][a:b])
    assert torch.isnan(got[100]).all()


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0, 3.0])
def test_scales(scale):
    lens = [200, 140]
    q, k, v = _inputs(8, 2, 64, lens, lens, seed=5)
    if scale > 0.5:  # scores of some hundred: one key holds nearly all of the weight
        q, k = (q * 2).to(BF), (k * 2).to(BF)
    got = _run(q, k, v, lens, lens, scale)
    out, bound = prompt_reference(q, k, v, lens, lens, scale)
    # fp32 scores of size x are off by 130 * 2^-24 of sum |q k|, here up to 2^11 * scale
    bound = bound + (2.0 ** -6 * abs(scale) * v.float().abs().max().item() if scale > 0.5 else 0)
    check(got, out, bound)


@pytest.mark.parametrize("d", [64, 128])
def test_rising_scores(d):
    """Keys whose scores rise along the sequence: the running maximum moves in every tile, by
    less and by more than the threshold."""
    n = 900
    q, k, v = _inputs(4, 1, d, [n], [n], seed=8)
    ramp = torch.linspace(0.0, 1.0, n, device="cuda")[:, None, None]
    for top in (12.0, 40.0, 300.0):
        unit = torch.zeros(d, device="cuda")
        unit[3] = 1.0
        kk = (0.2 * k.float() + ramp * top * unit).to(BF)
        qq = (0.2 * q.float() + unit).to(BF)
        got = _run(qq, kk, v, [n], [n], 1.0)
        out, bound = prompt_reference(qq, kk, v, [n], [n], 1.0)
        # |score| up to 2 * top + some: 130 * 2^-24 * 2^10 at most
        check(got, out, bound + 2.0 ** -6 * v.float().abs().max().item())


def test_infinite_scores():
    """A key of +inf scores gives NaN to the queries that see it and nothing to the others; one of
    -inf scores weighs nothing."""
    n = 150
    q, k, v = _inputs(2, 2, 64, [n], [n], seed=4)
    q = q.abs() + 0.1
    want = prompt_reference(q, k, v, [n], [n], 0.125)
    k = k.clone()
    k[140, 0] = float("inf")
    got = _run(q, k, v, [n], [n], 0.125)
    check(got[:140], want[0][:140], want[1][:140])
    assert torch.isnan(got[140:, 0]).all() and torch.isfinite(got[:, 1]).all()
    k[140, 0] = float("-inf")
    got = _run(q, k, v, [n], [n], 0.125)
    rest = [i for i in range(n) if i != 140]
    out, bound = prompt_reference(q[rest], k[rest], v[rest], [n - 1], [n - 1], 0.125)
    check(got[141:], out[140:], bound[140:])


def test_same_bits_stream_and_graph():
    """Repeated calls, a call on another stream and a replayed graph give the same bits; the
    graph follows lengths that change on the device."""
    import paged_kv_decode_02_gb300 as pk
    lens = [37, 800, 64, 5]
    q, k, v = _inputs(16, 2, 128, lens, lens, seed=2)
    first = _run(q, k, v, lens, lens, 0.09)
    for _ in range(3):
        assert torch.equal(first, _run(q, k, v, lens, lens, 0.09))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _run(q, k, v, lens, lens, 0.09)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, other)
    off = offsets(lens)
    out = torch.zeros_like(q)
    ws = torch.empty(pk.prompt_workspace_bytes(4, 16, 2, 128, q.shape[0], q.shape[0]),
                     dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.prompt_attention(q, k, v, off, 0.09, out=out, workspace=ws)
    graph.replay()
    assert torch.equal(first, out)
    lens = [200, 3, 0, 703]
    off.copy_(offsets(lens))
    graph.replay()
    check(out, *prompt_reference(q, k, v, lens, lens, 0.09))


def test_bad_offsets():
    """A sequence whose offsets fall or leave the arrays is flagged and not computed; the others
    are. Rows that no good sequence has stay as they were."""
    import paged_kv_decode_02_gb300 as pk
    from paged_kv_decode_02_gb300 import pagedkv
    q, k, v = _inputs(4, 2, 64, [60], [60], seed=1)
    good = prompt_reference(q[:20], k[:20], v[:20], [20], [20], 0.125)
    for off in ([0, 20, 10, 10], [0, 20, 70, 70], [-5, -5, 0, 20], [0, 20, 2 ** 30, -3]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(q, 3.0)
        pk.prompt_attention(q, k, v, torch.tensor(off, dtype=torch.int32, device="cuda"), 0.125,
                            out=out, status=status)
        assert status.item() == pagedkv.DEV_BAD_CONTEXT_LEN
        check(out[:20], *good)
        assert (out[20:] == 3).all()


def test_many_sequences():
    """More sequences than threads, most of them short or empty."""
    gen = torch.Generator().manual_seed(0)
    lens = torch.randint(0, 9, (1500,), generator=gen).tolist()
    lens[700] = 400
    q, k, v = _inputs(4, 4, 64, lens, lens, seed=6)
    got = _run(q, k, v, lens, lens, 0.125)
    check(got, *prompt_reference(q, k, v, lens, lens, 0.125))


def test_long_prompt():
    """A prompt whose keys take many tiles, cut at every place."""
    n, hq, hkv, d = 6001, 8, 2, 128
    q, k, v = _inputs(hq, hkv, d, [n], [n], seed=7)
    got = _run(q, k, v, [n], [n], d ** -0.5)
    check(got, *prompt_reference(q, k, v, [n], [n], d ** -0.5))


def test_refusals():
    import paged_kv_decode_02_gb300 as pk
    q, k, v = _inputs(4, 2, 64, [8], [8])
    off = offsets([8])
    with pytest.raises(ValueError):
        pk.prompt_attention(q, k, v[:4], off, 1.0)
    with pytest.raises(ValueError):
        pk.prompt_attention(q[..., ::2], k, v, off, 1.0)
    with pytest.raises(TypeError):
        pk.prompt_attention(q.float(), k, v, off, 1.0)
    with pytest.raises(ValueError):
        pk.prompt_attention(q, k, v, off, 1.0, kv_offsets=offsets([4, 4]))
    with pytest.raises(pk.PagedKVError):
        pk.prompt_attention(q, k, v, off, 1.0, workspace=torch.empty(256, dtype=torch.uint8,
                                                                     device="cuda"))
    with pytest.raises(pk.PagedKVError):
        pk.prompt_attention(torch.zeros(4, 3, 64, device="cuda", dtype=BF), k[:4], v[:4], off, 1.0)
