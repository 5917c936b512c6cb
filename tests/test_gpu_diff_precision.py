"""Differential decode over bf16 caches where the two maps nearly cancel: the error that is
left against 64 bits, which a softmax weight held in one bf16 term would multiply."""

import pytest
import torch

from diff_helpers import random_norm

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pk():
    from paged_kv_decode_02_gb300 import build_lib
    build_lib.build()
    import paged_kv_decode_02_gb300 as pk
    pk.load_library()
    return pk


def attend(x0, x1, v, lam, nw, one_term):
    """[2 D] in float64 from a pair's scores; one_term: weights rounded to bf16 (their sums
    not), as a plain fused kernel would have them."""
    o = []
    for x in (x0, x1):
        w = torch.exp(x - x.amax())
        r = w.to(torch.bfloat16).double() if one_term else w
        o.append(r @ v / w.sum())
    y = o[0] - lam * o[1]
    return y / y.square().mean().sqrt() * nw


@pytest.mark.parametrize("hq,hkv,d,bs", [(4, 2, 128, 16), (16, 2, 128, 16), (24, 2, 64, 16),
                                         (24, 2, 128, 32), (32, 2, 128, 32), (8, 4, 64, 32)])
@pytest.mark.parametrize("n,copies", [(1, 1), (33, 400), (2000, 1), (2000, 330), (30000, 1)])
def test_maps_that_nearly_cancel(pk, hq, hkv, d, bs, n, copies):
    """lambda 1 - 2^-6, maps some 2 % apart, norm on, in units that are cut and whole: the root
    mean square of the error over the output's. Rounding the output adds 2^-8 at most. The maps'
    errors are independent from token to token, so next to a difference of `apart` (root mean
    square over the tokens, by weight) they add sqrt(2) / apart times a weight's: 2^-16 for two
    bf16 terms, 2^-17 for fp32 scores and sums."""
    gen = torch.Generator(device=DEV).manual_seed(n + hq)
    r = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    blocks, g, lam = -(-n // bs), hq // hkv, 1 - 2.0 ** -6
    q = r(hq // 2, 1, d).expand(-1, 2, -1).clone()
    q[:, 1] += 0.02 * r(hq // 2, d)
    q = q.view(1, hq, d).to(torch.bfloat16)
    k = r(blocks, hkv // 2, 1, bs, d).expand(-1, -1, 2, -1, -1).reshape(blocks, hkv, bs, d)
    k, v = k.to(torch.bfloat16).contiguous(), r(blocks, hkv, bs, d).to(torch.bfloat16)
    table = torch.randperm(blocks, generator=gen, device=DEV).int()[None]
    nw, scale = random_norm(d, DEV), d ** -0.5
    got = pk.paged_decode_attention_diff(
        q.repeat(copies, 1, 1), k, v, table.repeat(copies, 1),
        torch.full((copies,), n, dtype=torch.int32, device=DEV),
        torch.full((hq // 2,), lam, device=DEV), scale, norm_weight=nw, eps=0.0).double()
    assert torch.isfinite(got).all()
    t = torch.arange(n, device=DEV)
    blk, off = table[0, t // bs].long(), t % bs
    worst, missed = 0.0, 0.0
    for j in range(hq // 2):
        p = j // g
        x = [(k[blk, 2 * p + m, off].double() @ q[0, 2 * j + m].double()) * scale for m in (0, 1)]
        vv = v[blk, 2 * p:2 * p + 2, off].double().flatten(1)
        ref = attend(*x, vv, lam, nw.double(), False)
        a, b = torch.softmax(x[0], 0), torch.softmax(x[1], 0)
        apart = float(((a - lam * b).square().sum() / a.square().sum()).sqrt())
        room = 2.0 ** -8 + 2 ** 0.5 * (2.0 ** -16 + 2.0 ** -17) / apart
        rms = float(ref.square().mean().sqrt())
        off_by = float((got[:, j] - ref).square().mean(1).sqrt().amax()) / rms
        worst = max(worst, off_by / room)
        one = attend(*x, vv, lam, nw.double(), True)
        missed = max(missed, float((one - ref).square().mean().sqrt()) / rms / room)
    assert worst <= 1.0
    assert n < 33 or missed > 2.0               # what the bound is for
