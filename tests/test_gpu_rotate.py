"""GPU rotate-and-append against the fp64 oracle."""

import numpy as np
import pytest
import torch

import oracle
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


def table(positions, rot, base=10000.0):
    f = base ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(positions)[:, None] * f
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float().to(DEV)


def inputs(T, hq, hkv, d, bs, seed=0, fused=True, far=500):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    qkv = torch.randn((T, (hq + 2 * hkv) * d), generator=gen, device=DEV)
    qkv = (qkv * torch.logspace(-2, 2, max(T, 1), device=DEV)[:T, None]).to(torch.bfloat16)
    q, k, v = (x.view(T, -1, d) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    nb = -(-T // bs) + 3
    slots = torch.randperm(nb * bs, generator=gen, device=DEV)[:T]
    pos = torch.randint(0, far, (T,), generator=gen, device=DEV)
    w = (1 + 0.3 * torch.randn((2, d), generator=gen, device=DEV)).to(torch.bfloat16)
    return q, k, v, pos, slots, w[0].contiguous(), w[1].contiguous(), nb


def reference(x, weight, pos, cs, eps, interleaved):
    """Rotated rows [T, H, D] in float64, and each element's pair magnitude."""
    x, cs, pos = to_f64(x), to_f64(cs), pos.cpu().numpy()
    wt = None if weight is None else to_f64(weight)
    out, n = np.empty_like(x), cs.shape[1] // 2
    for t in range(x.shape[0]):
        for h in range(x.shape[1]):
            c = cs[pos[t]]
            out[t, h] = oracle.norm_rotate_row(x[t, h], wt, c[:n], c[n:], eps, interleaved)
    mag = np.abs(out).max(-1, keepdims=True) * np.ones_like(out)
    return out, mag


# fp32 arithmetic: the mean of up to 128 squares, the root, two products and a sum, each
# within a few 2^-24 of the row's largest magnitude; taken as 2^-19 in all
FP32 = 2.0 ** -19


def assert_bf16(got, ref, mag):
    off = np.abs(to_f64(got) - ref)
    assert np.all(off <= 2.0 ** -8 * np.abs(ref) + FP32 * mag * 1.5), off.max()


@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (128, 48), (128, 16), (64, 64), (64, 48),
                                   (64, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rotate_bf16(pk, d, rot, interleaved, norm):
    T, hq, hkv, bs = 7, 6, 2, 16
    q, k, v, pos, slots, qw, kw, nb = inputs(T, hq, hkv, d, bs)
    qw, kw = (qw, kw) if norm else (None, None)
    slots[3] = -1                                            # rotated, not written
    slots[5] = nb * bs                                       # past the pool: the same
    cs = table(500, rot)
    kc = torch.randn((nb, hkv, bs, d), device=DEV).to(torch.bfloat16)
    vc = torch.randn_like(kc)
    k0, v0 = kc.clone(), vc.clone()
    out = pk.paged_kv_rotate_append(q, k, v, pos, cs, kc, vc, slots, q_norm=qw, k_norm=kw,
                                    eps=1e-6, interleaved=interleaved)
    torch.cuda.synchronize()
    assert_bf16(out, *reference(q, qw, pos, cs, 1e-6, interleaved))
    ref, mag = reference(k, kw, pos, cs, 1e-6, interleaved)
    for t in range(T):
        slot = int(slots[t])
        if 0 <= slot < nb * bs:
            assert_bf16(kc[slot // bs, :, slot % bs], ref[t], mag[t])
            assert torch.equal(vc[slot // bs, :, slot % bs], v[t])
            kc[slot // bs, :, slot % bs] = k0[slot // bs, :, slot % bs]
            vc[slot // bs, :, slot % bs] = v0[slot // bs, :, slot % bs]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)       # nothing else was written


@pytest.mark.parametrize("T,hq,hkv,d,bs", [(1, 1, 1, 64, 16), (1, 32, 8, 128, 16),
                                           (37, 5, 5, 128, 32), (513, 8, 2, 64, 32)])
def test_rotate_sizes_and_strides(pk, T, hq, hkv, d, bs):
    """One token to several hundred; separate tensors and slices of a fused projection give
    the same bits; q rotated in place too."""
    q, k, v, pos, slots, qw, kw, nb = inputs(T, hq, hkv, d, bs, seed=T)
    cs = table(500, d)
    res = []
    for form in range(3):
        kc = torch.zeros((nb, hkv, bs, d), dtype=torch.bfloat16, device=DEV)
        vc = torch.zeros_like(kc)
        a = [x.clone().contiguous() for x in (q, k, v)] if form else [q, k, v]
        out = pk.paged_kv_rotate_append(*a, pos, cs, kc, vc, slots, q_norm=qw, k_norm=kw,
                                        out=a[0] if form == 2 else None)
        assert form != 2 or out.data_ptr() == a[0].data_ptr()
        res.append((out.clone(), kc, vc))
    for r in res[1:]:
        assert all(torch.equal(x, y) for x, y in zip(r, res[0]))
    assert_bf16(res[0][0], *reference(q, qw, pos, cs, 1e-6, False))
    fused = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1)   # in place in a fused one
    parts = [x.view(T, -1, d) for x in fused.split([hq * d, hkv * d, hkv * d], 1)]
    kc = torch.zeros((nb, hkv, bs, d), dtype=torch.bfloat16, device=DEV)
    out = pk.paged_kv_rotate_append(*parts, pos, cs, kc, torch.zeros_like(kc), slots, q_norm=qw,
                                    k_norm=kw, out=parts[0])
    assert torch.equal(out, res[0][0]) and torch.equal(kc, res[0][1])
    assert torch.equal(parts[1], k) and torch.equal(parts[2], v)


@pytest.mark.parametrize("fmt", ["bf16", "int8", "e5m2"])
@pytest.mark.parametrize("T,hq,hkv,d", [(5300, 5, 5, 128), (13003, 9, 3, 64), (8200, 6, 2, 128)])
def test_rotate_many_tokens(pk, fmt, T, hq, hkv, d):
    """Thousands of tokens, whose lane groups take several rows each (15, 15 and 10 rows per
    token, none a multiple of 4): the same bits as in calls of 500 tokens, and sampled rows
    against the oracle."""
    bs = 16
    q, k, v, pos, slots, qw, kw, nb = inputs(T, hq, hkv, d, bs, seed=T)
    slots[::97] = -1
    cs = table(500, d // 2)
    dt = {"bf16": torch.bfloat16, "int8": torch.int8}.get(fmt, torch.uint8)

    def go(cuts):
        c = [torch.zeros((nb, hkv, bs, d), dtype=dt, device=DEV) for _ in range(2)]
        s = [torch.zeros((nb, hkv, bs), device=DEV) for _ in range(2)]
        outs = []
        for a, b in zip(cuts, cuts[1:]):
            args = (q[a:b], k[a:b], v[a:b], pos[a:b], cs, *c)
            if fmt == "bf16":
                outs.append(pk.paged_kv_rotate_append(*args, slots[a:b], q_norm=qw, k_norm=kw))
            else:
                outs.append(pk.paged_kv_rotate_append_q8(*args, *s, slots[a:b], fmt=fmt,
                                                         q_norm=qw, k_norm=kw))
        return [torch.cat(outs), *c, *s]
    whole = go([0, T])
    for x, y in zip(whole, go([*range(0, T, 500), T])):
        assert torch.equal(x, y)
    some = torch.randperm(T, device=DEV)[:40]
    assert_bf16(whole[0][some], *reference(q[some], qw, pos[some], cs, 1e-6, False))


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("d,bs,interleaved", [(128, 16, False), (64, 32, True)])
def test_rotate_q8(pk, fmt, d, bs, interleaved):
    """K: the stored value is within half a code step of the fp64 row (INT8: half the scale;
    FP8: half a step of the value, or of the smallest subnormal) and the scale is the row's
    absmax over the largest code. V: bit for bit what the append oracle writes. A row of
    zeros gives scale 0."""
    T, hq, hkv = 9, 4, 2
    q, k, v, pos, slots, qw, kw, nb = inputs(T, hq, hkv, d, bs, seed=3)
    k, v = k.contiguous(), v.contiguous()
    k[4], v[4] = 0, 0
    slots[2] = -1
    cs = table(500, d)
    dt = torch.int8 if fmt == "int8" else torch.uint8
    kc = torch.randint(0, 100, (nb, hkv, bs, d), device=DEV).to(dt)
    vc, ks = kc.clone(), torch.rand((nb, hkv, bs), device=DEV)
    vs = ks.clone()
    before = [x.clone() for x in (kc, vc, ks, vs)]
    out = pk.paged_kv_rotate_append_q8(q, k, v, pos, cs, kc, vc, ks, vs, slots, fmt=fmt,
                                       q_norm=qw, k_norm=kw, interleaved=interleaved)
    torch.cuda.synchronize()
    assert_bf16(out, *reference(q, qw, pos, cs, 1e-6, interleaved))
    ref, mag = reference(k, kw, pos, cs, 1e-6, interleaved)
    top = {"int8": 127.0, "e4m3": 448.0, "e5m2": 57344.0}[fmt]
    half, tiny = {"int8": (0, 0.5), "e4m3": (2.0 ** -4, 2.0 ** -10),
                  "e5m2": (2.0 ** -3, 2.0 ** -17)}[fmt]
    for t in range(T):
        slot = int(slots[t])
        if slot < 0:
            continue
        b, o = slot // bs, slot % bs
        s = to_f64(ks[b, :, o])
        assert np.all(np.abs(s - np.abs(ref[t]).max(-1) / top) <= FP32 * 2 * s)
        code = kc[b, :, o].cpu().numpy()
        val = (code.astype(np.float64) if fmt == "int8"
               else oracle.fp8_decode(code.astype(np.int64), fmt)) * s[:, None]
        room = np.maximum(half * np.abs(ref[t]), tiny * s[:, None]) * (1 + 2.0 ** -10)
        assert np.all(np.abs(val - ref[t]) <= room + FP32 * 4 * mag[t])
        assert t != 4 or (np.all(s == 0) and np.all(code == 0))
    args = (v.float().cpu().numpy(), v.float().cpu().numpy(),
            *[x.cpu().numpy() for x in (before[1], before[1], before[3], before[3])],
            slots.cpu().numpy(), bs)
    want = (oracle.append_scatter_int8(*args) if fmt == "int8"
            else oracle.append_scatter_fp8(*args, fmt))
    assert np.array_equal(vc.cpu().numpy(), want[1]) and np.array_equal(vs.cpu().numpy(), want[3])
    written = torch.zeros(nb * bs, dtype=torch.bool, device=DEV)
    written[slots[slots >= 0]] = True
    keep = ~written.view(nb, bs)[:, None, :].expand(nb, hkv, bs)
    assert torch.equal(kc[keep], before[0][keep]) and torch.equal(ks[keep], before[2][keep])


@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3", "e5m2"])
def test_position_zero_is_append(pk, fmt):
    """Without norms, at position 0 (angle 0), the caches hold exactly what append writes."""
    T, hq, hkv, d, bs = 21, 4, 4, 128, 16
    q, k, v, pos, slots, _, _, nb = inputs(T, hq, hkv, d, bs, seed=5, fused=False)
    cs = table(1, d)
    dt = {"bf16": torch.bfloat16, "int8": torch.int8}.get(fmt, torch.uint8)
    a = [torch.zeros((nb, hkv, bs, d), dtype=dt, device=DEV) for _ in range(4)]
    s = [torch.zeros((nb, hkv, bs), device=DEV) for _ in range(4)]
    pos.zero_()
    if fmt == "bf16":
        out = pk.paged_kv_rotate_append(q, k, v, pos, cs, a[0], a[1], slots)
        pk.paged_kv_append(k, v, a[2], a[3], slots)
    else:
        out = pk.paged_kv_rotate_append_q8(q, k, v, pos, cs, a[0], a[1], s[0], s[1], slots,
                                           fmt=fmt)
        if fmt == "int8":
            pk.paged_kv_append_int8(k, v, a[2], a[3], s[2], s[3], slots)
        else:
            pk.paged_kv_append_fp8(k, v, a[2], a[3], s[2], s[3], slots, fmt=fmt)
    assert torch.equal(out, q)
    assert torch.equal(a[0], a[2]) and torch.equal(a[1], a[3])
    assert torch.equal(s[0], s[2]) and torch.equal(s[1], s[3])


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e5m2"])
def test_quantised_rows_of_every_magnitude(pk, fmt):
    """V rows from 1e-38 (scales that are subnormal or 0) to 3e38, zeros, infinities and NaN
    among the elements: the codes and scales that append writes, bit for bit."""
    T, hkv, d, bs = 600, 2, 128, 16
    gen = torch.Generator(device=DEV).manual_seed(9)
    mag = torch.logspace(-38, 38, T, device=DEV)
    v = (torch.randn((T, hkv, d), generator=gen, device=DEV) * mag[:, None, None])
    v *= 10.0 ** (-8 * torch.rand((T, hkv, d), generator=gen, device=DEV))
    v = v.to(torch.bfloat16)
    v[7, 0, 5], v[8, 1, 3], v[9, 0, 0] = float("nan"), float("inf"), -float("inf")
    v[10] = 0
    nb = T // bs + 1
    slots = torch.randperm(nb * bs, generator=gen, device=DEV)[:T]
    dt = torch.int8 if fmt == "int8" else torch.uint8
    a = [torch.zeros((nb, hkv, bs, d), dtype=dt, device=DEV) for _ in range(4)]
    s = [torch.zeros((nb, hkv, bs), device=DEV) for _ in range(4)]
    pk.paged_kv_rotate_append_q8(v, v, v, torch.zeros_like(slots), table(1, d), a[0], a[1], s[0],
                                 s[1], slots, fmt=fmt)
    if fmt == "int8":
        pk.paged_kv_append_int8(v, v, a[2], a[3], s[2], s[3], slots)
    else:
        pk.paged_kv_append_fp8(v, v, a[2], a[3], s[2], s[3], slots, fmt=fmt)
    assert torch.equal(s[1].view(torch.int32), s[3].view(torch.int32))
    assert torch.equal(a[1], a[3])


def test_bad_positions_write_nothing(pk):
    T, hq, hkv, d, bs = 5, 4, 2, 64, 16
    q, k, v, pos, slots, qw, kw, nb = inputs(T, hq, hkv, d, bs, seed=6, far=40)
    cs = table(40, d)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kc = torch.zeros((nb, hkv, bs, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    good = pk.paged_kv_rotate_append(q, k, v, pos, cs, kc, vc, slots, status=status)
    assert int(status) == 0
    pos[1], pos[3] = 40, -1
    for st in (status, None):
        kc.zero_()
        vc.zero_()
        out = pk.paged_kv_rotate_append(q, k, v, pos, cs, kc, vc, slots, status=st)
        assert torch.all(out[[1, 3]] == 0)
        assert torch.equal(out[[0, 2, 4]], good[[0, 2, 4]])
        rows = vc.transpose(1, 2).reshape(nb * bs, hkv, d)
        assert torch.all(rows[slots[[1, 3]]] == 0) and torch.equal(rows[slots[0]], v[0])
        assert torch.count_nonzero(kc.transpose(1, 2).reshape(nb * bs, -1).any(1)) == 3
    assert int(status) == 0x10


def test_rotate_in_a_graph_and_on_another_stream(pk):
    T, hq, hkv, d, bs = 33, 8, 2, 128, 16
    q, k, v, pos, slots, qw, kw, nb = inputs(T, hq, hkv, d, bs, seed=7)
    cs = table(500, d)
    kc = torch.zeros((nb, hkv, bs, d), dtype=torch.bfloat16, device=DEV)
    vc, out = torch.zeros_like(kc), torch.empty((T, hq, d), dtype=torch.bfloat16, device=DEV)

    def go():
        pk.paged_kv_rotate_append(q, k, v, pos, cs, kc, vc, slots, q_norm=qw, k_norm=kw, out=out)
    go()
    want = [x.clone() for x in (out, kc, vc)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for _ in range(2):
        for x in (out, kc, vc):
            x.zero_()
        g.replay()
        assert all(torch.equal(x, y) for x, y in zip((out, kc, vc), want))
    side = torch.cuda.Stream()
    for x in (out, kc, vc):
        x.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip((out, kc, vc), want))


def test_rotate_argument_checks(pk):
    q, k, v, pos, slots, qw, kw, nb = inputs(4, 4, 2, 64, 16)
    cs = table(500, 64)
    kc = torch.zeros((nb, 2, 16, 64), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)

    def go(**kw):
        a = dict(q=q, k=k, v=v, positions=pos, cos_sin=cs, k_cache=kc, v_cache=vc,
                 slot_mapping=slots)
        a.update(kw)
        return pk.paged_kv_rotate_append(**a)
    go()
    for bad in (dict(k=k[:3]), dict(v=v[..., :32]), dict(positions=pos[:2]),
                dict(q_norm=qw[:32].contiguous()), dict(out=torch.empty_like(k)),
                dict(q=q.transpose(0, 1)), dict(v_cache=vc[:1])):
        with pytest.raises(ValueError):
            go(**bad)
    for bad in (dict(q=q.float()), dict(positions=pos.int()), dict(cos_sin=cs.double())):
        with pytest.raises(TypeError):
            go(**bad)
    for bad in (dict(cos_sin=cs[:, :24].contiguous()), dict(cos_sin=cs.repeat(1, 2))):
        with pytest.raises(pk.PagedKVError):                 # rotary_dim 24; more than head_dim
            go(**bad)
    odd = torch.zeros((4, 4 * 64 + 4), dtype=torch.bfloat16, device=DEV)[:, :256].view(4, 4, 64)
    with pytest.raises(pk.PagedKVError):                     # a token stride of 260
        go(q=odd)
    empty = pk.paged_kv_rotate_append(q[:0], k[:0], v[:0], pos[:0], cs, kc, vc, slots[:0])
    assert tuple(empty.shape) == (0, 4, 64)
