"""What is measured of three operators that stand beside the paged-cache append and decode:

* ``rotate``: per-head norms and the position rotation of new queries and keys, with the
  write of K and V into the paged cache in the same pass (``paged_kv_rotate_append``);
* ``write_read``: the same write into a one-byte cache (codes and per-row scales), then the
  whole contexts read back as bf16 rows (``paged_kv_rotate_append_q8``, ``paged_kv_gather``),
  as a prefill chunk does before a dense attention over its prefix;
* ``gather``: reading cached contexts back alone (``paged_kv_gather``);
* ``diff``: single-token differential attention over the paged cache, the difference of two
  softmax maps of a head pair (``paged_decode_attention_diff``, ``..._diff_q8``).

``own`` chooses between the operators' plain forms (elementary torch operations in 32
bits) and the framework's calls.
"""

import math

import numpy as np
import torch

own = False

Q8_MAX = {"int8": 127.0, "e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _case(name, op, kv, seqs, q_heads, kv_heads, head_dim, block, median, sigma=0.0, low=1,
          high=1 << 17, lens_seed=0, new=1, rotary=0, interleaved=False, norm=True):
    case = dict(op=op, kv=kv, seqs=seqs, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
                block=block, median=median, sigma=sigma, low=low, high=high, lens_seed=lens_seed)
    if op in ("rotate", "write_read"):
        case.update(new=new, rotary=rotary or head_dim, interleaved=interleaved)
    if op != "gather":
        case.update(norm=norm)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one request's decode step: the smallest write a server makes, all latency
        _case("rotate-one", "rotate", "bf16", 1, 32, 8, 128, 16, 700),
        # the decode step of a 64-request batch (64 query and 8 KV heads), ragged contexts
        _case("rotate-step", "rotate", "bf16", 64, 64, 8, 128, 16, 1024, 1.0, 128, 32768, 2),
        # a prefill of 4 prompts of 2048 tokens, interleaved pairs, half of the head rotated,
        # multi-head (32/32), no norms
        _case("rotate-prefill", "rotate", "bf16", 4, 32, 32, 128, 16, 2048, new=2048, rotary=64,
              interleaved=True, norm=False),
        # a prefill chunk over an INT8 cache: 16 requests write 256 tokens each and read their
        # whole contexts back
        _case("write-read-int8", "write_read", "int8", 16, 64, 8, 128, 16, 1024, 1.0, 256, 32768,
              5, new=256),
        # a decode step of a small model over an FP8 cache, read back for a check
        _case("write-read-e4m3", "write_read", "e4m3", 3, 8, 8, 64, 16, 40, 0.5, 1, 64, 1),
        # one short odd-length context read out of the cache
        _case("gather-one", "gather", "bf16", 1, 8, 8, 64, 16, 47),
        # every context of a ragged batch, E5M2 codes widened
        _case("gather-e5m2", "gather", "e5m2", 64, 64, 8, 128, 32, 1024, 1.0, 128, 32768, 2),
        # a whole multi-head layer's cache moved to dense rows
        _case("gather-bf16", "gather", "bf16", 32, 32, 32, 128, 16, 2048),
        # the smallest decode: four short requests
        _case("diff-tiny", "diff", "bf16", 4, 8, 8, 64, 16, 30, 0.6, 1, 64, 0, norm=False),
        # the ragged 64-request decode (long tail up to eleven thousand tokens)
        _case("diff-ragged", "diff", "bf16", 64, 64, 8, 128, 16, 1024, 1.0, 128, 32768, 2),
        # the largest: 128 requests of 8192 tokens over INT8 codes
        _case("diff-int8", "diff", "int8", 128, 32, 8, 128, 32, 8192),
        # one request with a very long context, split over the whole GPU, E4M3 codes
        _case("diff-long", "diff", "e4m3", 1, 32, 8, 128, 16, 131071),
    ]


def draw(rng):
    """One more case: any operator, cache type and head layout, batch and lengths log-uniform."""
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rotate", "write_read", "gather", "diff", "diff"])
    kv = ("bf16" if op == "rotate" else rng.choice(["int8", "e4m3", "e5m2"]) if op == "write_read"
          else rng.choice(["bf16", "int8", "e4m3", "e5m2"]))
    kv_heads = rng.choice([2, 4, 6, 8, 16])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 12] if kv_heads <= 8 else [1, 2, 3])
    head_dim = rng.choice([64, 128])
    seqs = spread(1, 256)
    # at most 2^28 cached values in all: a quarter of the largest listed case
    most = max(1, (1 << 28) // (seqs * kv_heads * head_dim))
    median = spread(1, min(most, 32768))
    new = 1 if rng.random() < 0.5 else min(median, spread(2, max(2, 16384 // seqs)))
    return _case("", op, kv, seqs, q_heads, kv_heads, head_dim, rng.choice([16, 32]), median,
                 rng.choice([0.0, 0.5, 1.0]), max(1, new if op in ("rotate", "write_read") else 1),
                 max(2 * median, new), rng.randrange(1 << 20), new,
                 rng.choice([head_dim, head_dim // 2, 16, 48]), rng.random() < 0.4,
                 rng.random() < 0.7)


def lengths(case):
    """Context lengths, from the case alone: log-normal around the median, clipped."""
    r = np.random.default_rng(case["lens_seed"])
    x = np.exp(np.log(case["median"]) + case["sigma"] * r.standard_normal(case["seqs"]))
    return np.clip(np.rint(x), case["low"], case["high"]).astype(np.int64)


def work(case):
    n = lengths(case)
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    row = 2 * hkv * (2 * d if case["kv"] == "bf16" else d + 4)  # a token's K and V as cached
    tables = 4 * int(np.sum(-(-n // case["block"]))) + 4 * case["seqs"]
    total = int(n.sum())
    if case["op"] in ("rotate", "write_read"):
        t = case["seqs"] * case["new"]
        moved = t * ((hq + 2 * hkv) * d * 2 + hq * d * 2 + row + 16 + 4 * case["rotary"])
        flops = t * (hq + hkv) * (6 * d if case["norm"] else 3 * d)
        if case["op"] == "write_read":  # rows just written need not come from memory again
            moved += (total - t) * row + total * 4 * hkv * d + tables
            flops += total * 2 * hkv * d
    elif case["op"] == "gather":
        moved, flops = total * (row + 4 * hkv * d) + tables, total * 2 * hkv * d
    else:
        moved = total * row + 2 * case["seqs"] * hq * d * 2 + tables
        flops = total * hq * (2 * d + 4 * d)
    return {"bytes": moved, "flops": flops}


def _cache(case, num_blocks, gen, dev):
    """K (or V) cache and its scales: bf16 N(0, 1) rows, or codes and scales of the shape that
    absmax quantisation of such rows has."""
    shape = (num_blocks, case["kv_heads"], case["block"], case["head_dim"])
    if case["kv"] == "bf16":
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16), None
    top = Q8_MAX[case["kv"]]
    scale = (2.5 + torch.rand(shape[:3], generator=gen, device=dev)) / top
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16) * (top / 3)
    x = x.clamp_(-top, top)
    if case["kv"] == "int8":
        return x.round_().to(torch.int8), scale
    return x.to(F8[case["kv"]]).view(torch.uint8), scale


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = np.random.default_rng(seed)
    n = lengths(case)
    b, bs = case["seqs"], case["block"]
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    blocks = -(-n // bs)
    num_blocks = int(blocks.sum()) + 1
    ids = host.permutation(num_blocks)[:num_blocks - 1].astype(np.int32)
    tables = np.zeros((b, int(blocks.max())), np.int32)
    tables[np.arange(tables.shape[1])[None, :] < blocks[:, None]] = ids
    st = {"case": dict(case), "lens": torch.from_numpy(n.astype(np.int32)).to(dev),
          "tables": torch.from_numpy(tables).to(dev), "max_len": int(n.max()),
          "total": int(n.sum())}
    st["k"], st["ks"] = _cache(case, num_blocks, gen, dev)
    st["v"], st["vs"] = _cache(case, num_blocks, gen, dev)

    if case["op"] in ("rotate", "write_read"):
        new, rot = case["new"], case["rotary"]
        t = b * new
        # a fused projection's output, its channels of different size
        qkv = torch.randn((t, (hq + 2 * hkv) * d), generator=gen, device=dev)
        qkv *= torch.exp(0.5 * torch.randn((qkv.shape[1],), generator=gen, device=dev))
        st["qkv"] = qkv.to(torch.bfloat16)
        pos = (n[:, None] - new + np.arange(new)[None, :])
        slot = np.take_along_axis(tables, pos // bs, 1).astype(np.int64) * bs + pos % bs
        st["pos"] = torch.from_numpy(pos.reshape(-1)).to(dev)
        st["slots"] = torch.from_numpy(slot.reshape(-1)).to(dev)
        freq = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
        angle = torch.arange(int(n.max()), device=dev, dtype=torch.float64)[:, None] * freq
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        st["qw"] = st["kw"] = None
        if case["norm"]:
            w = 1 + 0.2 * torch.randn((2, d), generator=gen, device=dev)
            st["qw"], st["kw"] = w[0].to(torch.bfloat16), w[1].to(torch.bfloat16)
        st["out"] = torch.empty((t, hq, d), device=dev, dtype=torch.bfloat16)
    if case["op"] in ("gather", "write_read"):
        off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        st["offsets"] = torch.from_numpy(off).to(dev)
        rows = (st["total"], hkv, d)
        st["out_k"] = torch.empty(rows, device=dev, dtype=torch.bfloat16)
        st["out_v"] = torch.empty(rows, device=dev, dtype=torch.bfloat16)
    if case["op"] == "diff":
        st["q"] = torch.randn((b, hq, d), generator=gen, device=dev, dtype=torch.bfloat16)
        st["lam"] = 0.2 + 0.6 * torch.rand((hq // 2,), generator=gen, device=dev)
        st["scale"] = d ** -0.5
        st["out"] = torch.empty((b, hq // 2, 2 * d), device=dev, dtype=torch.bfloat16)
        st["workspace"] = torch.empty(1 << 26, device=dev, dtype=torch.uint8)
        st["nw"], st["out_scale"] = None, 1.0
        if case["norm"]:
            w = 1 + 0.2 * torch.randn((2 * d,), generator=gen, device=dev)
            st["nw"], st["out_scale"] = w.to(torch.bfloat16), 1 - (0.8 - 0.6 * math.exp(-3.3))
    return st


EPS = 1e-6


# ---------------------------------------------------------------------------
# plain forms: elementary torch operations, 32 bits, one rounding at the end
# ---------------------------------------------------------------------------

def _split(st):
    c = st["case"]
    t = st["qkv"].shape[0]
    q, k, v = st["qkv"].split([c["q_heads"] * c["head_dim"]] + 2 * [c["kv_heads"] * c["head_dim"]], 1)
    return (q.view(t, c["q_heads"], c["head_dim"]), k.view(t, c["kv_heads"], c["head_dim"]),
            v.view(t, c["kv_heads"], c["head_dim"]))


def _norm_rotate(x, weight, cos, sin, case):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    r = case["rotary"]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if case["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _quantise(x, kv):
    top = Q8_MAX[kv]
    s = x.abs().amax(-1) / top
    y = x / torch.where(s > 0, s, 1.0)[..., None]
    if kv == "int8":
        return y.round().clamp(-top, top).to(torch.int8), s
    return y.clamp(-top, top).to(F8[kv]).view(torch.uint8), s


def _values(codes, scale, kv):
    """What cached rows stand for, in 32 bits."""
    if kv == "bf16":
        return codes.float()
    f = codes.float() if kv == "int8" else codes.view(F8[kv]).float()
    return f * scale[..., None]


def _plain_write(st):
    c, kv = st["case"], st["case"]["kv"]
    q, k, v = _split(st)
    cos, sin = st["cos_sin"][st["pos"]][:, None, :].chunk(2, -1)
    q = _norm_rotate(q, st["qw"], cos, sin, c).to(torch.bfloat16)
    k, v = _norm_rotate(k, st["kw"], cos, sin, c), v.float()
    blk, off = st["slots"] // c["block"], st["slots"] % c["block"]
    if kv == "bf16":
        st["k"][blk, :, off] = k.to(torch.bfloat16)
        st["v"][blk, :, off] = v.to(torch.bfloat16)
        return q
    st["k"][blk, :, off], st["ks"][blk, :, off] = _quantise(k, kv)
    st["v"][blk, :, off], st["vs"][blk, :, off] = _quantise(v, kv)
    return q


def _plain_gather(st):
    c, kv = st["case"], st["case"]["kv"]
    row = torch.arange(st["total"], device=st["lens"].device)
    s = torch.bucketize(row, st["offsets"][1:].long(), right=True)
    t = row - st["offsets"][s]
    blk, off = st["tables"][s, t // c["block"]].long(), t % c["block"]
    pick = lambda x: None if x is None else x[blk, :, off]  # noqa: E731
    return tuple(_values(pick(st[x]), pick(st[x + "s"]), kv).to(torch.bfloat16) for x in "kv")


def _plain_diff(st):
    c, kv = st["case"], st["case"]["kv"]
    b, hq, d = st["q"].shape
    pairs, g = c["kv_heads"] // 2, hq // c["kv_heads"]
    t = torch.arange(st["max_len"], device=st["lens"].device)
    hidden = t[None, :] >= st["lens"][:, None]
    blk = st["tables"][:, t // c["block"]].long()
    off = (t % c["block"]).expand_as(blk)
    pick = lambda x: None if x is None else x[blk, :, off]  # noqa: E731
    k = _values(pick(st["k"]), pick(st["ks"]), kv).view(b, -1, pairs, 2, d)
    q = st["q"].float().view(b, pairs, g, 2, d)
    x = torch.einsum("bpgmd,blpmd->bpgml", q, k) * st["scale"]
    del k
    x = x.masked_fill(hidden[:, None, None, None, :], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    x = x / x.sum(-1, keepdim=True)
    v = _values(pick(st["v"]), pick(st["vs"]), kv).view(b, -1, pairs, 2 * d)
    o = torch.einsum("bpgml,blpe->bpgme", x, v)
    o = o[..., 0, :] - st["lam"].view(pairs, g, 1) * o[..., 1, :]
    if st["nw"] is not None:
        o = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS) * st["nw"].float()
    return (o * st["out_scale"]).view(b, hq // 2, 2 * d).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own_write(st):
    import paged_kv_decode_02_gb300 as pk
    c = st["case"]
    q, k, v = _split(st)
    more = dict(q_norm=st["qw"], k_norm=st["kw"], eps=EPS, interleaved=c["interleaved"],
                out=st["out"])
    if c["kv"] == "bf16":
        return pk.paged_kv_rotate_append(q, k, v, st["pos"], st["cos_sin"], st["k"], st["v"],
                                         st["slots"], **more)
    return pk.paged_kv_rotate_append_q8(q, k, v, st["pos"], st["cos_sin"], st["k"], st["v"],
                                        st["ks"], st["vs"], st["slots"], fmt=_fmt(c), **more)


def _fmt(case):
    return "e5m2" if case["kv"] == "e5m2" else "e4m3"  # (an INT8 cache goes by its dtype)


def _own_gather(st):
    import paged_kv_decode_02_gb300 as pk
    return pk.paged_kv_gather(st["k"], st["v"], st["tables"], st["offsets"], k_scale=st["ks"],
                              v_scale=st["vs"], fmt=_fmt(st["case"]), out_k=st["out_k"],
                              out_v=st["out_v"])


def _own_diff(st):
    import paged_kv_decode_02_gb300 as pk
    more = dict(norm_weight=st["nw"], eps=EPS, out_scale=st["out_scale"], out=st["out"],
                workspace=st["workspace"])
    if st["case"]["kv"] == "bf16":
        return pk.paged_decode_attention_diff(st["q"], st["k"], st["v"], st["tables"], st["lens"],
                                              st["lam"], st["scale"], **more)
    return pk.paged_decode_attention_diff_q8(st["q"], st["k"], st["v"], st["ks"], st["vs"],
                                             st["tables"], st["lens"], st["lam"], st["scale"],
                                             fmt=_fmt(st["case"]), **more)


def run(st):
    op = st["case"]["op"]
    if op == "diff":
        return {"out": _own_diff(st) if own else _plain_diff(st)}
    if op == "gather":
        k, v = _own_gather(st) if own else _plain_gather(st)
        return {"k": k, "v": v}
    q = _own_write(st) if own else _plain_write(st)
    if op == "rotate":
        return {"q": q, "k_cache": st["k"], "v_cache": st["v"]}
    k, v = _own_gather(st) if own else _plain_gather(st)
    return {"q": q, "k": k, "v": v}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one sequence (or one token's position) at a time
# ---------------------------------------------------------------------------

def _exact_cached(codes, scale, kv):
    if kv == "bf16":
        return codes.double()
    f = codes if kv == "int8" else codes.view(F8[kv]).float()
    return f.double() * scale.double().unsqueeze(-1)


def _exact_turn(rows, weight, table, case):
    """Norm, then each pair as a complex number times e^(i angle)."""
    y = rows.double()
    if weight is not None:
        y = y / torch.sqrt(torch.sum(y * y, 2, True) / y.shape[2] + EPS) * weight.double()
    half = case["rotary"] // 2
    turn = torch.complex(table[:, :half].double(), table[:, half:].double()).unsqueeze(1)
    first = torch.arange(half, device=y.device) * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else half)
    z = torch.complex(y[:, :, first], y[:, :, second]) * turn
    y[:, :, first], y[:, :, second] = z.real, z.imag
    return y


def _exact_stored(rows, kv):
    """What a row stands for once it was quantised."""
    top = Q8_MAX[kv]
    s = rows.abs().max(2, True).values / top
    y = torch.where(s > 0, rows / s, 0.0)
    y = torch.round(y).clamp(-top, top) if kv == "int8" else y.float().clamp(-top, top).to(F8[kv]).double()
    return y * s


def exact(case, seed):
    st = prepare(case, seed)
    kv, bs = case["kv"], case["block"]
    n = [int(x) for x in lengths(case)]

    def rows(s, x):
        """Sequence s's cached rows [L, Hkv, D]."""
        ids = st["tables"][s, :-(-n[s] // bs)].long()
        scale = None if st[x + "s"] is None else st[x + "s"][ids]
        return _exact_cached(st[x][ids], scale, kv).transpose(1, 2).flatten(0, 1)[:n[s]]

    if case["op"] == "diff":
        b, hq, d = st["q"].shape
        g, out = hq // case["kv_heads"], []
        for s in range(b):
            k, q = rows(s, "k"), st["q"][s].double()
            # query head h = 2 j + m reads key head 2 (j // g) + m
            h = torch.arange(hq, device=q.device)
            key = 2 * (h // 2 // g) + h % 2
            a = torch.softmax(torch.stack([k[:, int(key[i])] @ q[i] for i in range(hq)]) * st["scale"], 1)
            v = rows(s, "v").flatten(1).view(n[s], -1, 2 * d)
            a = (a[0::2] - st["lam"].double()[:, None] * a[1::2]).view(-1, g, n[s])
            o = torch.stack([a[p] @ v[:, p] for p in range(v.shape[1])]).view(hq // 2, 2 * d)
            if st["nw"] is not None:
                o = o / torch.sqrt(o.square().sum(1, True) / (2 * d) + EPS) * st["nw"].double()
            out.append(o * st["out_scale"])
        return {"out": torch.stack(out)}
    if case["op"] == "gather":
        return {x: torch.cat([rows(s, x) for s in range(len(n))]) for x in "kv"}
    q, k, v = _split(st)
    table = st["cos_sin"][st["pos"]]
    q, k, v = _exact_turn(q, st["qw"], table, case), _exact_turn(k, st["kw"], table, case), v.double()
    if case["op"] == "rotate":
        caches = {}
        for name, x in (("k_cache", k), ("v_cache", v)):
            c = st[name[0]].double().transpose(1, 2).flatten(0, 1)
            c[st["slots"]] = x
            caches[name] = c.view(-1, bs, case["kv_heads"], case["head_dim"]).transpose(1, 2)
        return {"q": q, **caches}
    out, new = {"q": q}, case["new"]
    for name, x in (("k", k), ("v", v)):
        x = _exact_stored(x, kv)
        out[name] = torch.cat([torch.cat([rows(s, name)[:n[s] - new], x[s * new:(s + 1) * new]])
                               for s in range(len(n))])
    return out
