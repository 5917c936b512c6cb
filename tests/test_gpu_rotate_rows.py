"""Rotate-and-append of many tokens, whose lane groups take three rows of a token each: every
remainder of a token's rows by three, at both head sizes, in every form of the operator."""

import pytest
import torch

from test_gpu_rotate import DEV, assert_bf16, inputs, pk, reference, table  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norms", ["", "q", "k", "qk"])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (6, 2), (10, 2), (1, 1)])   # 12, 10, 14 and 3 rows
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_every_remainder(pk, fmt, interleaved, norms, hq, hkv, d):  # noqa: F811
    """In one call (q in place, with skipped slots and bad positions among the tokens): the bits
    of calls of 500 tokens, whose lane groups take one row each; sampled rows against the
    oracle."""
    rows, bs, far = hq + 2 * hkv, 32, 700
    T = -(-2 * 152 * 2048 // (rows * (d // 16))) + 5        # enough for several rows each
    q, k, v, pos, slots, qw, kw, nb = inputs(T, hq, hkv, d, bs, seed=rows + d, far=far)
    more = dict(q_norm=qw if "q" in norms else None, k_norm=kw if "k" in norms else None,
                interleaved=interleaved)
    slots[::97] = -1
    pos[::101] = far
    cs = table(far, d // 2)
    dt = {"bf16": torch.bfloat16, "int8": torch.int8}.get(fmt, torch.uint8)

    def go(step):
        c = [torch.zeros((nb, hkv, bs, d), dtype=dt, device=DEV) for _ in range(2)]
        s = [torch.zeros((nb, hkv, bs), device=DEV) for _ in range(2 * (fmt != "bf16"))]
        x = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1)
        x = [y.view(T, -1, d) for y in x.split([hq * d, hkv * d, hkv * d], 1)]
        for a in range(0, T, step):
            args = [y[a:a + step] for y in x] + [pos[a:a + step], cs, *c, *s, slots[a:a + step]]
            if fmt == "bf16":
                pk.paged_kv_rotate_append(*args, out=args[0], **more)
            else:
                pk.paged_kv_rotate_append_q8(*args, fmt=fmt, out=args[0], **more)
        assert torch.equal(x[1], k) and torch.equal(x[2], v)
        return [x[0], *c, *s]
    whole = go(T)
    for a, b in zip(whole, go(500)):
        assert torch.equal(a, b)
    some = torch.randperm(T, device=DEV)[:24]
    some = some[(some % 101 != 0) & (some % 97 != 0)]
    out, kc = whole[0], whole[1]
    assert not out[::101].any()
    assert_bf16(out[some], *reference(q[some], more["q_norm"], pos[some], cs, 1e-6, interleaved))
    blk, off = slots[some] // bs, slots[some] % bs
    if fmt == "bf16":
        assert_bf16(kc[blk, :, off],
                    *reference(k[some], more["k_norm"], pos[some], cs, 1e-6, interleaved))
        assert torch.equal(whole[2][blk, :, off], v[some])
