"""Differential decode over one-byte caches whose V rows are small, large, or of sizes far
apart: against the formula in 64 bits, within bounds that stay small next to the output."""

import pytest
import torch

from diff_helpers import random_norm

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOP = {"int8": 127.0, "e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.fixture(scope="module")
def pk():
    from paged_kv_decode_02_gb300 import build_lib
    build_lib.build()
    import paged_kv_decode_02_gb300 as pk
    pk.load_library()
    return pk


def to_codes(x, fmt):
    return x.round().to(torch.int8) if fmt == "int8" else x.to(F8[fmt]).view(torch.uint8)


def of_codes(c, fmt):
    return c.double() if fmt == "int8" else c.view(F8[fmt]).float().double()


class Case:
    """Sequences with a few peaked tokens each, `gap` nats above the others (whose scores
    scatter by 0.2), and V rows that share their columns' signs, so that what the many other
    tokens add up to is a large part of the output. `copies`: that many rows of the batch for
    each sequence, on the same blocks."""

    def __init__(self, fmt, lengths, gap, absmax, spread, hq, hkv, d, bs, seed=0, copies=1,
                 peaks=None):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
        u = lambda *s: torch.rand(s, generator=gen, device=DEV)  # noqa: E731
        self.fmt, self.d, self.bs, self.lengths = fmt, d, bs, lengths
        self.scale, top = d ** -0.5, TOP[fmt]
        B = len(lengths)
        blocks = [-(-n // bs) for n in lengths]
        nb = sum(blocks) + 1
        ids = torch.randperm(nb, generator=gen, device=DEV)[:nb - 1].int()
        self.tables = torch.zeros((B, max(blocks)), dtype=torch.int32, device=DEV)
        at = 0
        for s, n in enumerate(blocks):
            self.tables[s, :n] = ids[at:at + n]
            at += n
        self.lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        sign = torch.where(u(d) < 0.5, -1.0, 1.0)
        self.q = (sign + 0.1 * r(B, hq, d)).to(torch.bfloat16)
        k = to_codes(top / 4 * r(nb, hkv, bs, d).clamp(-4, 4), fmt)
        ks = torch.full((nb, hkv, bs), 0.2 / (self.scale * d ** 0.5 * top / 4), device=DEV)
        v = to_codes(top * (0.75 * torch.where(u(hkv, 1, d) < 0.5, -1.0, 1.0) +
                            0.25 * (2 * u(nb, hkv, bs, d) - 1)), fmt)
        vs = torch.full((nb, hkv, bs), absmax / top, device=DEV)
        for s, n in enumerate(lengths):
            t = torch.arange(n, device=DEV)
            blk, off = self.tables[s, t // bs].long(), t % bs
            peak = peaks if peaks is not None else [(7 * s + n // 2) % n]
            k[blk[peak], :, off[peak]] = to_codes(top * sign, fmt)
            ks[blk[peak], :, off[peak]] = gap / (self.scale * d * top)
            if spread == "tokens":      # sizes over three orders of magnitude, some negative
                f = 2.0 ** (-10 * u(n, hkv)) * torch.where(u(n, hkv) < 0.1, -1.0, 1.0)
                vs[blk, :, off] *= f
            elif spread == "grow":      # each row larger than the one before
                vs[blk, :, off] *= 2.0 ** torch.linspace(-30, 0, n, device=DEV)[:, None]
            elif spread == "shrink":
                vs[blk, :, off] *= 2.0 ** torch.linspace(0, -12, n, device=DEV)[:, None]
        if spread == "heads":           # a pair's second head far below its first
            vs[:, 1::2] *= 1e-9
        self.k, self.v, self.ks, self.vs = k, v, ks, vs
        self.lam = torch.linspace(0.1, 0.5, hq // 2, device=DEV)
        self.copies = copies
        self.tables, self.lens, self.q = (x.repeat_interleave(copies, 0)
                                          for x in (self.tables, self.lens, self.q))

    def call(self, pk, **kw):
        return pk.paged_decode_attention_diff_q8(
            self.q, self.k, self.v, self.ks, self.vs, self.tables, self.lens, self.lam, self.scale,
            fmt=self.fmt if self.fmt != "int8" else "e5m2", **kw)

    def reference(self, nw=None, eps=0.0, out_scale=1.0):
        """(out, bound) in float64. To first order a map's weighted mean O = sum a v is off by
        * a weight's relative error times |v - O|: the score's (130 fp32 roundings of at most
          2^-23 of the sum of its products' magnitudes, where an INT8 code enters as up to
          code + 1152; 8 more of the score itself) and the exponential's 2^-22;
        * fp32 sums: at most n / 16 steps of 2^-23 of sum a |v|, and n / 8 of 2^-24 of O;
        * a weight times its scale in fp16: 2^-11 of it, or half a subnormal step, 2^-25, in
          units that put the largest V scale of the head at 2^14 or above: 2^-39 of that scale
          per code, next to a largest weight of 1.
        Then lambda, the norm to first order, and half a step of the bf16 output."""
        hkv, d = self.k.shape[1], self.d
        q = self.q[::self.copies].double()
        B, hq, _ = q.shape
        g = hq // hkv
        out = torch.zeros((B, hq // 2, 2 * d), dtype=torch.float64, device=DEV)
        bound = torch.zeros_like(out)
        tables = self.tables[::self.copies]
        for s, n in enumerate(self.lengths):
            t = torch.arange(n, device=DEV)
            blk, off = tables[s, t // self.bs].long(), t % self.bs
            for p in range(hkv // 2):
                hd = slice(2 * p, 2 * p + 2)
                kc = of_codes(self.k[blk, hd, off], self.fmt)          # [n, 2, d]
                ks = self.ks[blk, hd, off].double()
                vc = of_codes(self.v[blk, hd, off], self.fmt)
                vs = self.vs[blk, hd, off].double()
                v = (vc * vs[..., None]).flatten(1)                    # [n, 2 d]
                half_sub = 2.0 ** -39 * vs.abs().amax(0)[:, None] * vc.abs().sum(0)
                half_sub = half_sub.flatten()
                for j in range(p * g, p * g + g):
                    y, e = 0.0, 0.0
                    for m in range(2):
                        qj = q[s, 2 * j + m]
                        x = (kc[:, m] @ qj) * ks[:, m] * self.scale
                        mag = (kc[:, m].abs() + (1152.0 if self.fmt == "int8" else 0.0)) @ qj.abs()
                        mag = (mag * ks[:, m].abs() * self.scale).amax()
                        dx = 130 * 2.0 ** -23 * mag + 2.0 ** -21 * x.abs().amax() + 2.0 ** -22
                        a = torch.softmax(x, 0)
                        o, av = a @ v, a @ v.abs()
                        off_m = (dx * (a @ (v - o).abs()) + (2.0 ** -11 + n / 16 * 2.0 ** -23) * av
                                 + n / 8 * 2.0 ** -24 * o.abs() + half_sub * a.amax())
                        c = 1.0 if m == 0 else float(self.lam[j])
                        y, e = (o, off_m) if m == 0 else (y - c * o, e + abs(c) * off_m)
                    f = 1.0
                    if nw is not None:
                        ms = y.square().mean() + eps
                        e = (e + y.abs() * (y.abs() * e).mean() / ms) * 1.05
                        f = nw.double() / ms.sqrt()
                    out[s, j] = y * f * out_scale
                    bound[s, j] = e * abs(out_scale) * (f.abs() if nw is not None else 1.0)
        bound += 2.0 ** -8 * out.abs()
        return out.repeat_interleave(self.copies, 0), bound.repeat_interleave(self.copies, 0)


def check(got, ref, bound):
    got = got.double()
    assert torch.isfinite(got).all()
    off = (got - ref).abs()
    assert torch.all(off <= bound), f"off by {float((off / ref.abs()).amax()):.3e} of the output"


SHAPES = [(4, 2, 128, 16), (16, 2, 128, 32), (32, 2, 64, 16), (8, 4, 64, 32)]
LONG = [(10.0, 1e-3), (8.0, 1e-4), (12.0, 1.0), (12.0, 1e9), (10.0, 1e-20)]
# of a batch of long contexts: one peak for each stream of items that a unit is read in
MANY = dict(copies=330, peaks=[0, 32, 64, 96])


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("hq,hkv,d,bs", SHAPES)
@pytest.mark.parametrize("gap,absmax", LONG)
def test_many_small_weights(pk, fmt, hq, hkv, d, bs, gap, absmax):
    """Few tokens far above thousands of others that together weigh as much, in one context cut
    over the whole GPU and in a batch of them: with V rows of any size the others' part is
    there, with a norm and without."""
    for n, more in ((131070, {}), (32770, MANY)):
        w = Case(fmt, [n], gap, absmax, None, hq, hkv, d, bs, **more)
        for nw in (None, random_norm(d, DEV)):
            ref, bound = w.reference(nw)
            # nothing that loses a sixteenth of the output passes
            assert torch.all(bound <= ref.abs() / 16)
            check(w.call(pk, norm_weight=nw, eps=0.0), ref, bound)


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("hq,hkv,d,bs", SHAPES)
@pytest.mark.parametrize("spread", ["tokens", "grow", "shrink", "heads"])
def test_rows_of_different_sizes(pk, fmt, hq, hkv, d, bs, spread):
    """Rows whose sizes differ by token, along the context or between a pair's heads, in cut
    units and in whole ones."""
    for lengths in ([9000, 1, 33], [300 + i % 7 for i in range(40)],
                    [40 + i % 25 for i in range(100)]):
        w = Case(fmt, lengths, 3.0, 2.0, spread, hq, hkv, d, bs, seed=len(lengths))
        ref, bound = w.reference(out_scale=0.5)
        check(w.call(pk, out_scale=0.5), ref, bound)


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_scale_that_is_no_number_stays_in_its_head(pk, fmt, hq, bad):
    """A V scale of NaN or infinity shows in every column of its own head and of no other, in
    whole units and cut ones; in a row past the context it shows nowhere."""
    w = Case(fmt, [40, 7000, 17], 2.0, 1.0, None, hq, 2, 128, 16)
    clean = w.call(pk)
    w.vs[w.tables[2, 1].long(), 0, 1:] = bad                # sequence 2 ends at its first row
    w.vs[w.tables[1, 437].long(), :, 8:] = bad              # 7000 = 437 * 16 + 8
    assert torch.equal(w.call(pk), clean)
    w.vs[w.tables[:2, 1].long(), 1, 3] = bad
    out = w.call(pk)
    assert not torch.isfinite(out[:2, :, 128:]).any()
    assert torch.equal(out[:2, :, :128], clean[:2, :, :128])
    assert torch.equal(out[2], clean[2])


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e5m2"])
def test_rows_of_zeros(pk, fmt):
    """Scales of zero (rows of zeros): alone they give zeros, among others they add nothing."""
    w = Case(fmt, [50, 4000], 2.0, 1.0, None, 8, 2, 128, 16)
    w.vs[:, :, ::2] = 0
    ref, bound = w.reference()
    check(w.call(pk), ref, bound)
    w.vs.zero_()
    out = w.call(pk)
    assert torch.all(out == 0)


def test_bounds_see_lost_weights():
    """The batch's bounds next to what a form would lose that dropped the weights below 2^-14
    of the largest (a planted mistake, in the reference alone)."""
    w = Case("int8", [32770], 10.0, 1e-3, None, 4, 2, 128, 16, **MANY)
    ref, bound = w.reference()
    t = torch.arange(32770, device=DEV)
    blk, off = w.tables[0, t // 16].long(), t % 16
    a = torch.softmax((of_codes(w.k[blk, 0, off], "int8") @ w.q[0, 0].double()) *
                      w.ks[blk, 0, off].double() * w.scale, 0)
    lost = float(a[a < a.amax() * 2.0 ** -14].sum())
    assert lost > 0.1 and float((bound / ref.abs()).amax()) < lost / 2
