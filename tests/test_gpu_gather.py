"""GPU gather of cached rows against the oracle's gathers, and the operators in one run."""

import numpy as np
import pytest
import torch

import oracle
from diff_helpers import assert_diff, diff_reference, random_lambda, random_norm, rows_of
from paged_kv_decode_02_gb300.workloads import make_workload
from parity_helpers import to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pk():
    from paged_kv_decode_02_gb300 import build_lib
    build_lib.build()
    import paged_kv_decode_02_gb300 as pk
    pk.load_library()
    return pk


def build(kv, lengths, hkv, d, bs, **kw):
    name = {"bf16": "70b-gqa", "int8": "int8"}.get(kv, "fp8-" + kv[4:])
    return make_workload(name, device=DEV, lengths=lengths, num_q_heads=hkv, num_kv_heads=hkv,
                         head_dim=d, block_size=bs, **kw)


def gather(pk, w, offsets, **kw):
    q8 = w.kv_dtype != "bf16"
    return pk.paged_kv_gather(w.k_cache, w.v_cache, w.block_tables, offsets,
                              k_scale=w.k_scale if q8 else None,
                              v_scale=w.v_scale if q8 else None,
                              fmt=w.kv_dtype[4:] if "fp8" in w.kv_dtype else "e5m2", **kw)


def offsets_of(n):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)


def assert_rows(got, want, exact):
    """bf16 caches: the same bits. One-byte: half a step of bf16 and the fp32 product's."""
    got = to_f64(got)
    if exact:
        assert np.array_equal(got, want)
    else:
        assert np.all(np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want))


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8_e4m3", "fp8_e5m2"])
@pytest.mark.parametrize("hkv,d,bs", [(1, 64, 16), (3, 128, 32), (8, 128, 16), (2, 64, 32)])
def test_gather_contexts(pk, kv, hkv, d, bs):
    """Whole contexts: empty ones among them (first, last, two in a row), tails inside blocks;
    unused rows hold NaN; rows past the last sequence stay as they were."""
    lengths = [0, 1, 15, 16, 0, 0, 33, 200, 7, 0]
    w = build(kv, lengths, hkv, d, bs, poison_unused=True)
    total = sum(lengths)
    ok = torch.full((total + 9, hkv, d), 3.0, dtype=torch.bfloat16, device=DEV)
    ov = ok.clone()
    a, b = gather(pk, w, offsets_of(lengths), out_k=ok, out_v=ov)
    assert a.data_ptr() == ok.data_ptr() and b.data_ptr() == ov.data_ptr()
    for x, which in ((ok, "k"), (ov, "v")):
        want = np.concatenate([np.stack(rows_of(w, s, which)[0], 1)
                               for s, n in enumerate(lengths) if n])
        assert_rows(x[:total], want, kv == "bf16")
        assert torch.all(x[total:] == 3.0)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_gather_ranges_and_shared_sequences(pk, kv):
    """Ranges that start inside a context (and inside a block), the same sequence's table
    twice, offsets that start past row 0: rows before the first offset stay as they were."""
    kv = kv if kv == "bf16" else "fp8_" + kv
    w = build(kv, [70, 100, 100], 2, 64, 16)
    w.block_tables[2] = w.block_tables[1]
    starts = torch.tensor([69, 17, 0], dtype=torch.int32, device=DEV)
    off = torch.tensor([2, 3, 53, 133], dtype=torch.int32, device=DEV)
    k, v = gather(pk, w, off, token_starts=starts,
                  out_k=torch.full((133, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV),
                  num_tokens=133)
    assert torch.all(k[:2] == 3.0)
    for x, which in ((k, "k"), (v, "v")):
        r0 = np.stack(rows_of(w, 0, which)[0], 1)
        r1 = np.stack(rows_of(w, 1, which)[0], 1)
        want = np.concatenate([r0[69:70], r1[17:67], r1[:80]])
        assert_rows(x[2:], want, kv == "bf16")


@pytest.mark.parametrize("B,n", [(700, 3), (1, 4097), (3000, 1)])
def test_gather_many_and_long(pk, B, n):
    w = build("bf16", [n] * B, 2, 64, 16)
    k, v = gather(pk, w, offsets_of([n] * B), num_tokens=B * n)
    t = torch.arange(n, device=DEV)
    blk, off = w.block_tables[:, t // 16].long(), (t % 16).expand(B, n)
    assert torch.equal(k.view(B, n, 2, 64), w.k_cache[blk, :, off])
    assert torch.equal(v.view(B, n, 2, 64), w.v_cache[blk, :, off])


@pytest.mark.parametrize("hkv,d", [(1, 64), (1, 128), (2, 64)])
@pytest.mark.parametrize("lengths", [[0, 5, 0, 0, 1, 1, 700, 0, 0, 2, 0], [1] * 500 + [0] * 40 + [3] * 90,
                                     [0] * 70 + [200, 129, 128, 127] + [0] * 33, [9000, 0, 1]])
def test_gather_tiles_over_many_sequences(pk, hkv, d, lengths):
    """Tiles of up to 128 tokens (one narrow head) that span many sequences, empty ones among
    them, first and last."""
    w = build("bf16", lengths, hkv, d, 16)
    n = sum(lengths)
    k, v = gather(pk, w, offsets_of(lengths), num_tokens=n)
    for x, which in ((k, "k"), (v, "v")):
        want = np.concatenate([np.stack(rows_of(w, s, which)[0], 1) if L else
                               np.zeros((0, hkv, d)) for s, L in enumerate(lengths)])
        assert_rows(x, want, True)


def test_gather_bad_pages_and_ranges(pk):
    """Bad ids and tokens outside the table give zero rows and a flag, with and without a
    status word; offsets past the buffer or falling are flagged and stay inside it."""
    w = build("int8", [64, 64, 64], 2, 128, 16)
    off = offsets_of([64, 64, 64])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    good = gather(pk, w, off, num_tokens=192, status=status)[0]
    assert int(status) == 0
    w.block_tables[0, 1] = -1
    w.block_tables[1, 3] = w.k_cache.shape[0]
    for st in (status, None):
        k, _ = gather(pk, w, off, num_tokens=192, status=st)
        assert torch.all(k[16:32] == 0) and torch.all(k[112:128] == 0)
        keep = [i for i in range(192) if not (16 <= i < 32 or 112 <= i < 128)]
        assert torch.equal(k[keep], good[keep])
    assert int(status) == 0x2
    status.zero_()
    starts = torch.tensor([0, -3, 10], dtype=torch.int32, device=DEV)
    cap = w.block_tables.shape[1] * 16
    k, _ = gather(pk, w, off, token_starts=starts, num_tokens=192, status=status)
    assert torch.all(k[64:67] == 0) and torch.all(k[128 + cap - 10:] == 0)
    assert int(status) == 0x1 | 0x2
    pad = torch.full((300, 2, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    for bad in ([0, 64, 128, 192], [0, 100, 20, 90], [-5, 20, 60, 90]):
        status.zero_()
        pad.fill_(3.0)
        gather(pk, w, torch.tensor(bad, dtype=torch.int32, device=DEV), out_k=pad[50:150],
               out_v=torch.empty_like(pad[50:150]), status=status)
        assert int(status) & 0x1
        assert torch.all(pad[:50] == 3.0) and torch.all(pad[150:] == 3.0)


def test_gather_in_a_graph(pk):
    """Captured once, replayed over another cache content and other offsets."""
    w = build("fp8_e5m2", [40, 90], 2, 64, 32)
    off = offsets_of([40, 90])
    out = [torch.zeros((130, 2, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    gather(pk, w, off, out_k=out[0], out_v=out[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gather(pk, w, off, out_k=out[0], out_v=out[1])
    off.copy_(offsets_of([10, 90]))
    w.k_scale *= 2
    for x in out:
        x.fill_(3.0)
    g.replay()
    fresh = gather(pk, w, off, num_tokens=100)
    assert torch.equal(out[0][:100], fresh[0]) and torch.equal(out[1][:100], fresh[1])
    assert torch.all(out[0][100:] == 3.0)


def test_gather_argument_checks(pk):
    w = build("bf16", [40, 90], 2, 64, 16)
    off = offsets_of([40, 90])
    with pytest.raises(ValueError):
        gather(pk, w, off)                                   # no size
    with pytest.raises(ValueError):
        gather(pk, w, off[:2], num_tokens=40)
    with pytest.raises(ValueError):
        gather(pk, w, off, num_tokens=130, out_k=torch.empty((129, 2, 64), dtype=torch.bfloat16,
                                                             device=DEV))
    with pytest.raises(TypeError):
        gather(pk, w, off.long(), num_tokens=130)
    with pytest.raises(TypeError):
        pk.paged_kv_gather(w.k_cache.float(), w.v_cache.float(), w.block_tables, off, 130)
    k, v = gather(pk, w, off, num_tokens=0)
    assert k.shape[0] == 0 and v.shape[0] == 0


# ---------------------------------------------------------------------------
# the operators together: a prompt, decode steps, and the cache read back
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_rows_far_into_a_cache(pk, kv):
    """Written to and read from blocks on both sides of 2^32 bytes into the cache: as near its
    start."""
    hkv, d, bs, T = 8, 128, 16, 50
    block_bytes = hkv * bs * d * (2 if kv == "bf16" else 1)
    far = 2 ** 32 // block_bytes - 2
    nb = far + 4
    dt = torch.bfloat16 if kv == "bf16" else torch.int8
    caches = [torch.zeros((nb, hkv, bs, d), dtype=dt, device=DEV) for _ in range(2)]
    scales = [torch.zeros((nb, hkv, bs), device=DEV) for _ in range(2 * (kv != "bf16"))]
    gen = torch.Generator(device=DEV).manual_seed(3)
    q, k, v = (torch.randn((T, hkv, d), generator=gen, device=DEV).to(torch.bfloat16)
               for _ in range(3))
    cs = torch.cat([torch.cos(torch.arange(T * 64.0, device=DEV)).view(T, 64),
                    torch.sin(torch.arange(T * 64.0, device=DEV)).view(T, 64)], 1)
    pos = torch.arange(T, device=DEV)
    write = pk.paged_kv_rotate_append if kv == "bf16" else pk.paged_kv_rotate_append_q8
    got = []
    for first in (0, far):
        slots = first * bs + pos
        write(q, k, v, pos, cs, *caches, *scales, slots)
        tab = first + torch.arange(4, dtype=torch.int32, device=DEV)[None]
        got += pk.paged_kv_gather(*caches, tab, offsets_of([T]), T,
                                  **(dict(k_scale=scales[0], v_scale=scales[1]) if scales else {}))
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])
    assert got[0].abs().amax() > 1 and (kv != "bf16" or torch.equal(got[1], v))


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8_e4m3", "fp8_e5m2"])
def test_prompt_steps_and_read_back(pk, kv):
    """Prompts written in one call, three decode steps (rotate, append, differential
    attention over everything so far), then the caches read back. Each step's output against
    the oracle over the cache as it stands; the rows read back against the values the cache
    holds; the whole step as a captured graph gives the same bits."""
    hq, hkv, d, bs = 8, 4, 64, 16
    prompt, steps = [5, 40, 16], 3
    total = [n + steps for n in prompt]
    w = make_workload({"bf16": "70b-gqa", "int8": "int8"}.get(kv, "fp8-" + kv[4:]), device=DEV,
                      lengths=total, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs)
    for c in (w.k_cache, w.v_cache):
        c.zero_()
    gen = torch.Generator(device=DEV).manual_seed(11)
    f = 10000.0 ** (-np.arange(0, d, 2) / d)
    ang = np.arange(64)[:, None] * f
    cs = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float().to(DEV)
    wn = (1 + 0.2 * torch.randn((2, d), generator=gen, device=DEV)).to(torch.bfloat16)
    lam, nw = random_lambda(hq, DEV), random_norm(d, DEV)

    def slots_at(s, t):
        return int(w.block_tables[s, t // bs]) * bs + t % bs

    def write(q, k, v, pos, slots):
        more = dict(q_norm=wn[0], k_norm=wn[1])
        if kv == "bf16":
            return pk.paged_kv_rotate_append(q, k, v, pos, cs, w.k_cache, w.v_cache, slots, **more)
        return pk.paged_kv_rotate_append_q8(q, k, v, pos, cs, w.k_cache, w.v_cache, w.k_scale,
                                            w.v_scale, slots, fmt=kv[4:], **more)

    def attend(q, lens):
        a = (w.block_tables, lens, lam, w.scale)
        more = dict(norm_weight=nw, out_scale=0.5)
        if kv == "bf16":
            return pk.paged_decode_attention_diff(q, w.k_cache, w.v_cache, *a, **more)
        return pk.paged_decode_attention_diff_q8(q, w.k_cache, w.v_cache, w.k_scale, w.v_scale, *a,
                                                 fmt=kv[4:], **more)

    def rows(T):
        x = torch.randn((T, (hq + 2 * hkv) * d), generator=gen, device=DEV).to(torch.bfloat16)
        return [y.view(T, -1, d) for y in x.split([hq * d, hkv * d, hkv * d], 1)]

    pos = [t for n in prompt for t in range(n)]
    at = [slots_at(s, t) for s, n in enumerate(prompt) for t in range(n)]
    write(*rows(len(pos)), torch.tensor(pos, device=DEV), torch.tensor(at, device=DEV))
    lens = torch.tensor(prompt, dtype=torch.int32, device=DEV)
    for i in range(steps):
        pos = lens.long()
        at = torch.tensor([slots_at(s, prompt[s] + i) for s in range(3)], device=DEV)
        lens = lens + 1
        new = rows(3)
        q = write(*new, pos, at)
        out = attend(q, lens)
        w.q, w.context_lens = q, lens
        ref, bound = diff_reference(w, lam, nw, 1e-5, 0.5)
        assert_diff(out, ref, bound)
    q8 = kv != "bf16"
    k, v = pk.paged_kv_gather(w.k_cache, w.v_cache, w.block_tables, offsets_of(total),
                              sum(total), k_scale=w.k_scale if q8 else None,
                              v_scale=w.v_scale if q8 else None,
                              fmt=kv[4:] if "fp8" in kv else "e5m2")
    for x, which in ((k, "k"), (v, "v")):
        want = np.concatenate([np.stack(rows_of(w, s, which)[0], 1) for s in range(3)])
        assert_rows(x, want, not q8)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = attend(write(*new, pos, at), lens)
    again.zero_()
    g.replay()
    assert torch.equal(again, out)
