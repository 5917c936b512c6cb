"""What is measured of four operators around the paged cache's append and decode:

* ``resize``: block tables, slots and positions of new tokens from the requests' lengths, and
  the blocks given back (``paged_kv_resize``);
* ``keep``: the accepted tokens of a verified draft moved up in the cache (``paged_kv_keep``);
* ``tree``: attention of a tree of drafted tokens over the cache
  (``paged_decode_attention_tree``, ``..._tree_q8``);
* ``prompt``: causal attention of whole prompts, packed one after the other, or of their last
  chunk (``prompt_attention``).

``own`` chooses between the operators' plain forms (elementary torch operations, 32 bits where
they compute) and the framework's calls.
"""

import math

import numpy as np
import torch

own = False

Q8_MAX = {"int8": 127.0, "e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _case(name, op, kv, seqs, q_heads, kv_heads, head_dim, block, median, sigma=0.0, low=0,
          high=1 << 17, lens_seed=0, **more):
    """median, sigma, low, high: context lengths (log-normal, clipped), new tokens included
    except for ``resize``. ``new``: new, drafted or chunk tokens of a request."""
    case = dict(op=op, kv=kv, seqs=seqs, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
                block=block, median=median, sigma=sigma, low=low, high=high, lens_seed=lens_seed,
                **more)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one request grows by the token it decodes: what a server does at the very least
        _case("resize-one", "resize", "bf16", 1, 8, 8, 128, 16, 700, new=1, new_sigma=0.0),
        # 256 prompts come in together, and leave together
        _case("resize-prompts", "resize", "bf16", 256, 8, 8, 128, 16, 0, new=1024, new_sigma=1.0,
              lens_seed=2),
        # the accepted tokens of 64 requests, each from one of four drafts of four tokens
        _case("keep-bf16", "keep", "bf16", 64, 8, 8, 128, 16, 1024, 1.0, 128, 32768, 2, chains=4,
              depth=4),
        # the same for a large batch over INT8 codes, longer drafts
        _case("keep-int8", "keep", "int8", 256, 8, 8, 128, 32, 512, 0.5, 64, 4096, 3, chains=3,
              depth=21),
        # four short requests of a small model, trees of five tokens
        _case("tree-tiny", "tree", "bf16", 4, 8, 8, 64, 16, 30, 0.6, 5, 64, 0, new=5,
              ragged=False),
        # the ragged 64-request batch, 16 drafted tokens each
        _case("tree-ragged", "tree", "bf16", 64, 64, 8, 128, 16, 1024, 1.0, 128, 32768, 2, new=16,
              ragged=True),
        # 16 long requests over INT8 codes, trees of up to 60 tokens
        _case("tree-int8", "tree", "int8", 16, 32, 8, 128, 32, 8192, new=60, ragged=True),
        # one request with a very long context, a tree of 33 tokens, E4M3 codes
        _case("tree-long", "tree", "e4m3", 1, 32, 8, 128, 16, 131071, new=33, ragged=False),
        # three short prompts of odd lengths
        _case("prompt-short", "prompt", "bf16", 3, 8, 8, 64, 16, 47, 0.5, 1, 200, 4, new=0),
        # prompts of a serving batch: 16 of log-normal length
        _case("prompt-mixed", "prompt", "bf16", 16, 64, 8, 128, 16, 1024, 1.0, 128, 32768, 5,
              new=0),
        # the last 256 tokens of each as a chunk, over what the cache already holds of the rest
        _case("prompt-chunk", "prompt", "bf16", 16, 64, 8, 128, 16, 1024, 1.0, 256, 32768, 5,
              new=256),
        # one very long prompt
        _case("prompt-long", "prompt", "bf16", 1, 32, 8, 128, 16, 32768, new=0),
    ]


def draw(rng):
    """One more case: any operator, cache type and head layout, batch and lengths log-uniform."""
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["resize", "keep", "tree", "tree", "prompt", "prompt"])
    kv = "bf16" if op in ("prompt", "resize") else rng.choice(["bf16", "int8", "e4m3", "e5m2"])
    kv_heads = rng.choice([1, 2, 4, 6, 8, 16])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 12] if kv_heads <= 8 else [1, 2, 3])
    head_dim = rng.choice([64, 128])
    block = rng.choice([16, 32])
    seqs = spread(1, 256)
    sigma = rng.choice([0.0, 0.5, 1.0])
    seed = rng.randrange(1 << 20)
    # at most 2^28 cached values in all
    most = max(1, min(32768, (1 << 28) // (seqs * kv_heads * head_dim)))
    if op == "resize":
        held = rng.choice([0, spread(1, 8192)])
        new = spread(1, 64) if held else spread(1, 4096)
        return _case("", op, kv, seqs, kv_heads, kv_heads, head_dim, block, held, sigma, 0, 65536,
                     seed, new=new, new_sigma=rng.choice([0.0, 0.5]))
    if op == "keep":
        chains, depth = spread(1, 8), spread(1, 30)
        return _case("", op, kv, seqs, kv_heads, kv_heads, head_dim, block, spread(1, most), sigma,
                     0, 2 * most, seed, chains=chains, depth=depth)
    if op == "tree":
        new = spread(1, 64)
        # at most 2^36 products of a query with a key's element
        most = max(new, min(most, (1 << 36) // (seqs * new * q_heads * head_dim)))
        return _case("", op, kv, seqs, q_heads, kv_heads, head_dim, block, spread(new, most), sigma,
                     1, 2 * most, seed, new=new, ragged=rng.random() < 0.5)
    seqs = spread(1, 64)
    # at most 2^39 such products (a quarter of the longest prompt's), 2^16 tokens
    median = spread(1, max(1, min(16384, (1 << 16) // seqs,
                                  int(math.sqrt((1 << 39) / (seqs * q_heads * head_dim))))))
    new = 0 if rng.random() < 0.6 else spread(1, 512)
    return _case("", op, kv, seqs, q_heads, kv_heads, head_dim, block, median, min(sigma, 0.5), 1,
                 2 * median, seed, new=new)


def _normal_lengths(median, sigma, low, high, n, rng):
    if median <= 0:
        return np.zeros(n, np.int64)
    x = np.exp(np.log(median) + sigma * rng.standard_normal(n))
    return np.clip(np.rint(x), low, high).astype(np.int64)


def lengths(case):
    """(context lengths, new tokens) of every request, from the case alone."""
    r = np.random.default_rng(case["lens_seed"])
    b = case["seqs"]
    n = _normal_lengths(case["median"], case["sigma"], case["low"], case["high"], b, r)
    op = case["op"]
    if op == "resize":
        return n, _normal_lengths(case["new"], case["new_sigma"], 1, 32768, b, r)
    if op == "keep":
        new = np.full(b, 1 + case["chains"] * case["depth"])
        return n + new, new
    if op == "tree":
        new = r.integers(1, case["new"] + 1, b) if case["ragged"] else np.full(b, case["new"])
        return np.maximum(n, new), new
    return n, np.minimum(n, case["new"]) if case["new"] else n


def _kept(case):
    """(path [B, depth + 1], kept [B]): the draft is a root and ``chains`` runs of ``depth``
    tokens; a request keeps the root and the first tokens of one run, or nothing."""
    r = np.random.default_rng(case["lens_seed"] + 1)
    b, depth = case["seqs"], case["depth"]
    chain = r.integers(0, case["chains"], b)
    kept = r.integers(0, depth + 2, b)
    path = np.zeros((b, depth + 1), np.int64)
    path[:, 1:] = 1 + chain[:, None] * depth + np.arange(depth)
    return path, kept


def work(case):
    n, new = lengths(case)
    hq, hkv, d, bs = case["q_heads"], case["kv_heads"], case["head_dim"], case["block"]
    row = 2 * hkv * (2 * d if case["kv"] == "bf16" else d + 4)  # a token's K and V as cached
    b, op = case["seqs"], case["op"]
    if op == "resize":  # two calls: lengths, targets, offsets; the blocks' ids there and back
        blocks = int(np.sum(-(-(n + new) // bs) + -n // bs))
        return {"bytes": 2 * 16 * b + 2 * 8 * blocks + 16 * int(new.sum()), "flops": 0}
    if op == "keep":
        path, kept = _kept(case)
        moved = int(np.sum((np.arange(path.shape[1]) < kept[:, None])
                           & (path != np.arange(path.shape[1]))))
        return {"bytes": moved * 2 * row + b * 8 + 4 * int(kept.sum()), "flops": 0}
    if op == "tree":
        tables = 4 * int(np.sum(-(-n // bs)))
        most = case["new"]
        moved = int(n.sum()) * row + 2 * b * most * hq * d * 2 + tables + 8 * b + 8 * b * most
        return {"bytes": moved, "flops": 4 * d * hq * int(np.sum(new * (n - new + 1)))}
    pairs = int(np.sum(new * (n - new) + new * (new + 1) // 2))
    return {"bytes": int(new.sum()) * hq * d * 4 + int(n.sum()) * hkv * d * 4 + 8 * (b + 1),
            "flops": 4 * d * hq * pairs}


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
    n, new = lengths(case)
    op, b, bs = case["op"], case["seqs"], case["block"]
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]

    def put(x, dtype=np.int32):
        return torch.from_numpy(np.ascontiguousarray(x).astype(dtype)).to(dev)

    def rows(count, heads):
        return torch.randn((count, heads, d), generator=gen, device=dev, dtype=torch.bfloat16)

    st = {"case": dict(case), "n": n, "new": new}
    if op == "prompt":
        st["scale"] = d ** -0.5
        st["q_offsets"] = put(np.concatenate([[0], np.cumsum(new)]))
        st["out"] = torch.empty((int(new.sum()), hq, d), device=dev, dtype=torch.bfloat16)
        st["workspace"] = torch.empty(1 << 27, device=dev, dtype=torch.uint8)
        if case["new"]:  # the chunk's queries, and the keys and values read back from the cache
            st["q"] = rows(int(new.sum()), hq)
            st["k"], st["v"] = rows(int(n.sum()), hkv), rows(int(n.sum()), hkv)
            st["kv_offsets"] = put(np.concatenate([[0], np.cumsum(n)]))
        else:  # parts of a fused projection's output
            qkv = rows(int(n.sum()), hq + 2 * hkv)
            st["q"], st["k"], st["v"] = qkv.split([hq, hkv, hkv], 1)
            st["kv_offsets"] = st["q_offsets"]
        return st

    total = n + new if op == "resize" else n
    blocks = -(-total // bs)
    num_blocks = int(blocks.sum()) + 1 + int(blocks.sum()) // 5
    ids = host.permutation(num_blocks).astype(np.int32)
    tables = np.zeros((b, int(blocks.max())), np.int32)
    if op == "resize":
        held = -(-n // bs)
        used = int(held.sum())
        tables[np.arange(tables.shape[1])[None, :] < held[:, None]] = ids[:used]
        free = np.zeros(num_blocks, np.int32)
        free[:num_blocks - used] = ids[used:]
        st.update(tables=put(tables), lens=put(n), small=put(n), large=put(total), free=put(free),
                  free_count=put([num_blocks - used]),
                  slots=torch.empty(int(new.sum()), device=dev, dtype=torch.int64),
                  positions=torch.empty(int(new.sum()), device=dev, dtype=torch.int64),
                  offsets=torch.empty(b + 1, device=dev, dtype=torch.int32),
                  none=torch.empty(0, device=dev, dtype=torch.int64),
                  no_offsets=torch.empty(b + 1, device=dev, dtype=torch.int32))
        return st
    tables[np.arange(tables.shape[1])[None, :] < blocks[:, None]] = ids[:int(blocks.sum())]
    st.update(tables=put(tables), lens=put(n))
    st["k"], st["ks"] = _cache(case, num_blocks, gen, dev)
    st["v"], st["vs"] = _cache(case, num_blocks, gen, dev)
    if op == "keep":
        path, kept = _kept(case)
        st.update(base=put(n - new), path=put(path), kept=put(kept))
        return st
    most = case["new"]
    st["q"] = torch.randn((b, most, hq, d), generator=gen, device=dev, dtype=torch.bfloat16)
    # a random tree per request: node i hangs on one of the eight nodes before it
    mask = np.zeros((b, most, (most + 63) // 64), np.uint64)
    for i in range(most):
        if i:
            mask[:, i] = mask[np.arange(b), i - 1 - host.integers(0, min(i, 8), b)]
        mask[:, i, i // 64] |= np.uint64(1 << (i % 64))
    st.update(mask=put(mask.view(np.int64), np.int64), scale=d ** -0.5,
              tree_lens=put(new) if case["ragged"] else None, out=torch.empty_like(st["q"]),
              workspace=torch.empty(1 << 28, device=dev, dtype=torch.uint8))
    return st


# ---------------------------------------------------------------------------
# plain forms: elementary torch operations, 32 bits, one rounding at the end
# ---------------------------------------------------------------------------

def _values(codes, scale, kv):
    """What cached rows stand for, in 32 bits."""
    if kv == "bf16":
        return codes.float()
    f = codes.float() if kv == "int8" else codes.view(F8[kv]).float()
    return f * scale[..., None]


def _owner(offsets, count):
    """Sequence of each of ``count`` items, and the item's place in it."""
    i = torch.arange(count, device=offsets.device)
    s = torch.bucketize(i, offsets[1:], right=True)
    return s, i - offsets[s]


def _starts(x):
    return torch.cat([torch.zeros(1, device=x.device, dtype=torch.int64), x.cumsum(0)])


def _plain_resize(st):
    bs, free, count = st["case"]["block"], st["free"], st["free_count"]
    old, new = st["small"].long(), st["large"].long()
    first, last = (old + bs - 1) // bs, (new + bs - 1) // bs
    moved = int((-(-(st["n"] + st["new"]) // bs) + -st["n"] // bs).sum())  # known on the host
    # blocks for the grown requests, from the end of the list
    s, i = _owner(_starts(last - first), moved)
    order = torch.arange(moved, device=s.device)
    st["tables"][s, first[s] + i] = free[count - 1 - order]
    count -= moved
    # the new tokens' positions and slots
    offsets = _starts(new - old)
    t, j = _owner(offsets, st["slots"].shape[0])
    pos = old[t] + j
    st["positions"].copy_(pos)
    st["slots"].copy_(st["tables"][t, pos // bs].long() * bs + pos % bs)
    st["offsets"].copy_(offsets)
    st["lens"].copy_(st["large"])
    # and back: the blocks return in reverse order
    free[(count + moved - 1 - order).long()] = st["tables"][s, first[s] + i]
    count += moved
    st["lens"].copy_(st["small"])


def _plain_keep(st):
    bs = st["case"]["block"]
    i = torch.arange(st["path"].shape[1], device=st["path"].device)
    s, i = torch.nonzero(i < st["kept"][:, None], as_tuple=True)
    src, dst = st["base"][s] + st["path"][s, i], st["base"][s] + i
    sb, db = st["tables"][s, src // bs].long(), st["tables"][s, dst // bs].long()
    for x in (st["k"], st["v"], st["ks"], st["vs"]):
        if x is not None:
            x[db, :, dst % bs] = x[sb, :, src % bs]


def _sequence(st, s, x):
    """Sequence s's cached rows [Hkv, L, D], in 32 bits."""
    n, bs = int(st["n"][s]), st["case"]["block"]
    ids = st["tables"][s, :-(-n // bs)].long()
    scale = st[x + "s"]
    v = _values(st[x][ids], None if scale is None else scale[ids], st["case"]["kv"])
    return v.transpose(0, 1).flatten(1, 2)[:, :n]


def _attend(q, k, v, seen, scale):
    """q [Hq, N, D], k and v [Hkv, L, D] in 32 bits, seen [N, L]: softmax(scale q k) v."""
    hkv, g = k.shape[0], q.shape[0] // k.shape[0]
    x = torch.matmul(q.reshape(hkv, -1, q.shape[2]), k.transpose(1, 2)) * scale
    x = x.view(hkv, g, *seen.shape).masked_fill_(~seen, -math.inf)
    x = torch.exp_(x.sub_(x.amax(-1, keepdim=True)))
    x = x.div_(x.sum(-1, keepdim=True))
    return torch.matmul(x.view(hkv, -1, seen.shape[1]), v).view(q.shape)


def _plain_tree(st):
    out = st["out"].zero_()
    bit = torch.arange(st["case"]["new"], device=out.device)
    for s in range(out.shape[0]):
        n, t = int(st["n"][s]), int(st["new"][s])
        bits = (st["mask"][s, :t, bit[:t] // 64] >> (bit[:t] % 64)) & 1
        seen = torch.cat([torch.ones((t, n - t), device=out.device, dtype=torch.bool),
                          bits.bool()], 1)
        q = st["q"][s, :t].float().transpose(0, 1)
        o = _attend(q, _sequence(st, s, "k"), _sequence(st, s, "v"), seen, st["scale"])
        out[s, :t] = o.transpose(0, 1).to(torch.bfloat16)
    return out


def _plain_prompt(st):
    out, row, key = st["out"], 0, 0
    for n, new in zip(st["n"].tolist(), st["new"].tolist()):
        k = st["k"][key:key + n].float().transpose(0, 1)
        v = st["v"][key:key + n].float().transpose(0, 1)
        step = max(1, (1 << 28) // (n * out.shape[1]))  # queries at a time
        for a in range(0, new, step):
            b = min(new, a + step)
            t = torch.arange(a, b, device=out.device)
            seen = torch.arange(n, device=out.device)[None, :] <= n - new + t[:, None]
            q = st["q"][row + a:row + b].float().transpose(0, 1)
            out[row + a:row + b] = _attend(q, k, v, seen, st["scale"]).transpose(0, 1).to(
                torch.bfloat16)
        row, key = row + new, key + n
    return out


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _fmt(case):
    return "e5m2" if case["kv"] == "e5m2" else "e4m3"  # (an INT8 cache goes by its dtype)


def _own_resize(st):
    import paged_kv_decode_02_gb300 as pk
    bs = st["case"]["block"]
    pk.paged_kv_resize(st["tables"], st["lens"], st["large"], st["free"], st["free_count"], bs,
                       slot_mapping=st["slots"], positions=st["positions"],
                       token_offsets=st["offsets"])
    pk.paged_kv_resize(st["tables"], st["lens"], st["small"], st["free"], st["free_count"], bs,
                       slot_mapping=st["none"], positions=st["none"],
                       token_offsets=st["no_offsets"])


def _own_keep(st):
    import paged_kv_decode_02_gb300 as pk
    pk.paged_kv_keep(st["k"], st["v"], st["tables"], st["base"], st["path"], st["kept"],
                     k_scale=st["ks"], v_scale=st["vs"])


def _own_tree(st):
    import paged_kv_decode_02_gb300 as pk
    more = dict(tree_lens=st["tree_lens"], out=st["out"], workspace=st["workspace"])
    if st["case"]["kv"] == "bf16":
        return pk.paged_decode_attention_tree(st["q"], st["k"], st["v"], st["tables"], st["lens"],
                                              st["mask"], st["scale"], **more)
    return pk.paged_decode_attention_tree_q8(st["q"], st["k"], st["v"], st["ks"], st["vs"],
                                             st["tables"], st["lens"], st["mask"], st["scale"],
                                             fmt=_fmt(st["case"]), **more)


def _own_prompt(st):
    import paged_kv_decode_02_gb300 as pk
    return pk.prompt_attention(st["q"], st["k"], st["v"], st["q_offsets"], st["scale"],
                               kv_offsets=st["kv_offsets"], out=st["out"],
                               workspace=st["workspace"])


def run(st):
    op = st["case"]["op"]
    if op == "resize":
        (_own_resize if own else _plain_resize)(st)
        return {x: st[x] for x in ("slots", "positions", "offsets", "tables", "lens", "free",
                                   "free_count")}
    if op == "keep":
        (_own_keep if own else _plain_keep)(st)
        return {x: st[x] for x in ("k", "v", "ks", "vs") if st[x] is not None}
    if op == "tree":
        return {"out": _own_tree(st) if own else _plain_tree(st)}
    return {"out": _own_prompt(st) if own else _plain_prompt(st)}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits, one sequence (and one KV head) at a time
# ---------------------------------------------------------------------------

def _exact_resize(st):
    """A list of free blocks, a list of blocks per request, one token after the other."""
    bs, n, new = st["case"]["block"], st["n"].tolist(), st["new"].tolist()
    tables, free = st["tables"].cpu().numpy().copy(), st["free"].cpu().numpy()
    spare = free[:int(st["free_count"])].tolist()
    slots, positions, offsets = [], [], [0]
    for s, (have, more) in enumerate(zip(n, new)):
        for p in range(have, have + more):
            if p % bs == 0:
                tables[s, p // bs] = spare.pop()
            slots.append(int(tables[s, p // bs]) * bs + p % bs)
            positions.append(p)
        offsets.append(offsets[-1] + more)
    dev = st["lens"].device
    put = lambda x, like: torch.as_tensor(np.array(x), dtype=like.dtype, device=dev)  # noqa: E731
    return {"slots": put(slots, st["slots"]), "positions": put(positions, st["positions"]),
            "offsets": put(offsets, st["offsets"]), "tables": put(tables, st["tables"]),
            "lens": st["small"].clone(), "free": st["free"].clone(),
            "free_count": st["free_count"].clone()}


def _exact_keep(st):
    path, kept = _kept(st["case"])
    base, bs = st["n"] - st["new"], st["case"]["block"]
    out = {x: st[x].clone() for x in ("k", "v", "ks", "vs") if st[x] is not None}
    tables = st["tables"].cpu().numpy()
    src, dst = [], []
    for s in range(len(base)):
        for i in range(int(kept[s])):
            a, b = int(base[s] + path[s, i]), int(base[s]) + i
            src.append(int(tables[s, a // bs]) * bs + a % bs)
            dst.append(int(tables[s, b // bs]) * bs + b % bs)
    dev = st["k"].device
    src, dst = (torch.tensor(x, device=dev, dtype=torch.int64) for x in (src, dst))
    for x in out.values():
        by_token = x.transpose(1, 2).flatten(0, 1).clone()  # one row of heads per slot
        by_token[dst] = by_token[src]
        x.copy_(by_token.view(x.shape[0], bs, *by_token.shape[1:]).transpose(1, 2))
    return {x: t.double() if t.is_floating_point() else t for x, t in out.items()}


def _exact_rows(st, s, x):
    n, bs, kv = int(st["n"][s]), st["case"]["block"], st["case"]["kv"]
    t = torch.arange(n, device=st["tables"].device)
    blk, off = st["tables"][s, t // bs].long(), t % bs
    r = st[x][blk, :, off]
    if kv == "bf16":
        return r.double()
    r = r.double() if kv == "int8" else r.view(F8[kv]).double()
    return r * st[x + "s"][blk, :, off].double().unsqueeze(2)


def _exact_attend(q, k, v, bias, scale):
    """One head: q [N, D], k and v [L, D], bias [N, L] of 0 and -inf."""
    x = torch.addmm(bias, q, k.T, alpha=scale)
    e = torch.exp(x - x.max(1, True).values)
    return (e @ v) / e.sum(1, True)


def exact(case, seed):
    d, hq, hkv = case["head_dim"], case["q_heads"], case["kv_heads"]
    n, new = lengths(case)
    if 4.0 * d * hq * float(np.sum(n * new)) > 6e12:
        return None
    st = prepare(case, seed)
    if case["op"] == "resize":
        return _exact_resize(st)
    if case["op"] == "keep":
        return _exact_keep(st)
    dev, g = st["q"].device, hq // hkv
    out = torch.zeros(st["q"].shape, device=dev, dtype=torch.float64)
    if case["op"] == "tree":
        words = st["mask"].cpu().numpy().view(np.uint64)
        for s in range(len(n)):
            t, length = int(new[s]), int(n[s])
            bias = np.zeros((t, length))
            for j in range(t):
                hit = (words[s, :t, j // 64] >> np.uint64(j % 64)) & np.uint64(1)
                bias[hit == 0, length - t + j] = -math.inf
            bias = torch.from_numpy(bias).to(dev)
            k, v = _exact_rows(st, s, "k"), _exact_rows(st, s, "v")
            for h in range(hq):
                out[s, :t, h] = _exact_attend(st["q"][s, :t, h].double(), k[:, h // g],
                                              v[:, h // g], bias, st["scale"])
        return {"out": out}
    a = b = 0
    for length, t in zip(n.tolist(), new.tolist()):
        for i in range(0, t, 4096):
            rows = torch.arange(i, min(t, i + 4096), device=dev)
            hidden = torch.arange(length, device=dev) > (rows + length - t).unsqueeze(1)
            bias = torch.zeros(hidden.shape, device=dev, dtype=torch.float64)
            bias[hidden] = -math.inf
            for h in range(hq):
                out[a + rows, h] = _exact_attend(
                    st["q"][a + rows, h].double(), st["k"][b:b + length, h // g].double(),
                    st["v"][b:b + length, h // g].double(), bias, st["scale"])
        a, b = a + t, b + length
    return {"out": out}
