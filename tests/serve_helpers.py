"""Plain 64-bit forms of the tree and prompt attention, with a bound on what the kernels may be
off, element by element, and of the moves around them. Nothing here touches the CUDA library."""

import numpy as np
import torch

Q8_MAX = {"int8": 127.0, "e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
HALF = 2.0 ** -8        # half a step of bf16, relative to the value
HALF16 = 2.0 ** -11     # of fp16
# fp32 parts of a weight's relative error: a score is a sum of up to 128 products times a scale
# (below 130 * 2^-24 * sum |q k| * scale, which stays below 2^6 here: 2^-11), the exponential's is
# 2^-22, sums over up to 2^14 tokens add 2^-10 at the very worst
FP32 = 2.0 ** -9


def attend(q, k, v, seen, scale, weight=HALF, value=0.0):
    """(out, bound): q [Hq, N, D], k, v [Hkv, L, D] and seen [N, L] -> [N, Hq, D] in 64 bits.

    Weights a rounded by `weight` (relative) and values by `value` move the mean by at most
    (weight + value) * sum a |v|; the fp32 parts move each weight by FP32 of itself, which moves
    the mean by sum a |v - out|; the output is rounded to bf16."""
    hq, n, d = q.shape
    hkv, L, _ = k.shape
    g = hq // hkv
    q, k, v = q.double().reshape(hkv, g * n, d), k.double(), v.double()
    x = (q @ k.transpose(1, 2) * scale).view(hkv, g, n, L)
    x = x.masked_fill(~seen, -np.inf)
    top = x.amax(-1, keepdim=True) if L else x.new_zeros(hkv, g, n, 1)
    a = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    a = a / a.sum(-1, keepdim=True).clamp_min(1e-300)
    a = a.view(hkv, g * n, L)
    out = a @ v
    mag = a @ v.abs()
    bound = (weight + value) * mag + FP32 * (mag + out.abs()) + HALF * out.abs() + 2.0 ** -100
    shape = lambda t: t.view(hq, n, d).transpose(0, 1)  # noqa: E731
    return shape(out), shape(bound)


def check(got, out, bound, what=""):
    off = (got.double() - out).abs()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = (off - bound).max().item() if off.numel() else 0.0
    assert worst <= 0.0, f"{what}: off by {off.max().item():.3e}, over the bound by {worst:.3e}"


def quantise(x, kv):
    """Rows as a cache holds them: (codes, scales or None, values in 64 bits)."""
    if kv == "bf16":
        x = x.to(torch.bfloat16)
        return x, None, x.double()
    top = Q8_MAX[kv]
    s = x.abs().amax(-1).float() / top
    y = (x.float() / torch.where(s > 0, s, 1.0)[..., None]).clamp(-top, top)
    codes = y.round().to(torch.int8) if kv == "int8" else y.to(F8[kv]).view(torch.uint8)
    f = codes.double() if kv == "int8" else codes.view(F8[kv]).double()
    return codes, s, f * s[..., None].double()


class Cache:
    """A paged cache of sequences with given lengths, its blocks in random order, everything
    that no sequence holds poisoned (NaN where the type has one)."""

    def __init__(self, lens, hkv, d, bs, kv="bf16", seed=0, spare=3, dev="cuda", scale=1.0):
        gen = torch.Generator(device="cpu").manual_seed(seed)
        self.lens, self.bs, self.kv, self.hkv, self.d = list(lens), bs, kv, hkv, d
        held = [-(-n // bs) for n in self.lens]
        self.nb = sum(held) + spare
        ids = torch.randperm(self.nb, generator=gen)
        mbs = max(held + [1])
        tables = torch.full((len(self.lens), mbs), -7, dtype=torch.int32)
        at = 0
        for s, h in enumerate(held):
            tables[s, :h] = ids[at:at + h].int()
            at += h
        x = [torch.randn(self.nb, hkv, bs, d, generator=gen) * scale for _ in range(2)]
        live = torch.zeros(self.nb, bs, dtype=torch.bool)
        for s, n in enumerate(self.lens):
            for j in range(held[s]):
                live[tables[s, j], :min(bs, n - j * bs)] = True
        live = live[:, None, :]
        self.values, self.caches, self.scales = [], [], []
        for t in x:
            c, sc, v = quantise(t, kv)
            if kv == "bf16":
                c = torch.where(live[..., None], c, float("nan"))
            elif kv == "e4m3":
                c = torch.where(live[..., None], c, torch.tensor(0x7F, dtype=torch.uint8))
            if sc is not None:
                sc = torch.where(live, sc, float("nan"))
            self.values.append(v)
            self.caches.append(c.to(dev).contiguous())
            self.scales.append(None if sc is None else sc.to(dev).contiguous())
        self.tables = tables.to(dev)
        self.context_lens = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        self.values = [v.to(dev) for v in self.values]

    def rows(self, s, which):
        """[Hkv, L, D] of sequence s, in 64 bits."""
        n = self.lens[s]
        ids = self.tables[s, :-(-n // self.bs)].long()
        return self.values[which][ids].transpose(0, 1).reshape(self.hkv, -1, self.d)[:, :n]


def random_trees(sizes, width, most, seed=0):
    """(mask [B, most, words] int64, seen): node i hangs on one of the `width` nodes before it."""
    r = np.random.default_rng(seed)
    words = (most + 63) // 64
    mask = np.zeros((len(sizes), most, words), np.uint64)
    seen = []
    for s, t in enumerate(sizes):
        m = np.zeros((t, t), bool)
        for i in range(t):
            if i and r.random() < 0.9:
                m[i] = m[i - 1 - r.integers(0, min(i, width))]
            m[i, i] = True
        for i in range(t):
            for j in np.nonzero(m[i])[0]:
                mask[s, i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
        seen.append(torch.from_numpy(m))
    return torch.from_numpy(mask.view(np.int64)), seen


def tree_reference(cache, q, seen, sizes, scale):
    """(out, bound) [B, N, Hq, D] of the tree attention over a Cache."""
    weight = HALF if cache.kv == "bf16" else HALF16
    value = 0.0 if cache.kv == "bf16" else HALF16
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.full_like(out, 2.0 ** -100)
    for s, t in enumerate(sizes):
        n = cache.lens[s]
        if t == 0:
            continue
        m = torch.cat([torch.ones(t, n - t, dtype=torch.bool), seen[s]], 1).to(q.device)
        o, b = attend(q[s, :t].transpose(0, 1), cache.rows(s, 0), cache.rows(s, 1), m, scale,
                      weight, value)
        out[s, :t], bound[s, :t] = o, b
    return out, bound


def prompt_reference(q, k, v, q_lens, kv_lens, scale):
    """(out, bound) [Tq, Hq, D]: packed sequences, the queries their last tokens."""
    outs, a, b = [], 0, 0
    for nq, nk in zip(q_lens, kv_lens):
        i = torch.arange(nq, device=q.device)[:, None]
        seen = torch.arange(nk, device=q.device)[None, :] <= nk - nq + i
        outs.append(attend(q[a:a + nq].transpose(0, 1), k[b:b + nk].transpose(0, 1),
                           v[b:b + nk].transpose(0, 1), seen, scale))
        a, b = a + nq, b + nk
    return torch.cat([o for o, _ in outs]), torch.cat([e for _, e in outs])


def offsets(lens, dev="cuda"):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=dev)


class Pool:
    """Lists of blocks, one per sequence, and a stack of free ones: resize, token by token."""

    def __init__(self, lens, bs, mbs, free, tables):
        self.lens, self.bs, self.mbs, self.free = list(lens), bs, mbs, list(free)
        self.tables = [list(t) for t in tables]

    def resize(self, targets, num_tokens):
        """Returns (slots, positions, offsets, short): whether something did not fit."""
        held = lambda n: -(-n // self.bs)  # noqa: E731
        ok = [0 <= a <= self.mbs * self.bs and 0 <= t <= self.mbs * self.bs
              for a, t in zip(self.lens, targets)]
        back = []
        for s, t in enumerate(targets):
            if ok[s] and t < self.lens[s]:
                back += self.tables[s][held(t):held(self.lens[s])]
                self.lens[s] = t
        self.free += back[::-1]
        slots, positions, offs = [-1] * num_tokens, [0] * num_tokens, [0]
        short = dry = False
        for s, t in enumerate(targets):
            n = self.lens[s]
            new = max(0, t - n) if ok[s] else 0
            need = held(t) - held(n) if new else 0
            offs.append(offs[-1] + new)
            if not new:
                continue
            if offs[-1] > num_tokens or (need and (dry or need > len(self.free))):
                short, dry = True, dry or need > 0
                continue
            for p in range(n, t):
                if p % self.bs == 0:
                    self.tables[s][p // self.bs] = self.free.pop()
                slots[offs[-2] + p - n] = self.tables[s][p // self.bs] * self.bs + p % self.bs
                positions[offs[-2] + p - n] = p
            self.lens[s] = t
        return slots, positions, offs, short
