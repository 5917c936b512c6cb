"""A server's rounds: resize, rotate and append, prompt attention, tree attention, kept tokens and
decode in turn over one paged cache, against the definition in 64 bits on what the cache holds."""

import numpy as np
import pytest
import torch

from serve_helpers import attend, check, offsets, prompt_reference, random_trees, tree_reference
from serve_helpers import HALF, HALF16

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """Caches, tables and the free list of a server, and the calls of a step."""

    def __init__(self, b, hq, hkv, d, bs, kv, nb, mbs, seed=0):
        import paged_kv_decode_02_gb300 as pk
        self.pk, self.hq, self.hkv, self.d, self.bs, self.kv = pk, hq, hkv, d, bs, kv
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        dtype = BF if kv == "bf16" else torch.int8
        self.caches = [torch.zeros(nb, hkv, bs, d, dtype=dtype, device="cuda") for _ in range(2)]
        self.scales = [torch.zeros(nb, hkv, bs, device="cuda") for _ in range(2)]
        self.tables = torch.full((b, mbs), -1, dtype=torch.int32, device="cuda")
        self.len_t = torch.zeros(b, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(nb, generator=self.gen, device="cuda").int()
        self.count = _i32([nb])
        self.status = _i32([0])
        angle = torch.arange(4096, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(0, d, 2, device="cuda") / d)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        self.scale = d ** -0.5

    @property
    def lens(self):
        return self.len_t.tolist()

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.gen, device="cuda").to(BF)

    def resize(self, targets, num_tokens=None):
        return self.pk.paged_kv_resize(self.tables, self.len_t, targets, self.free, self.count,
                                       self.bs, num_tokens=num_tokens, status=self.status)

    def append(self, q, k, v, positions, slots):
        if self.kv == "bf16":
            return self.pk.paged_kv_rotate_append(q, k, v, positions, self.cos_sin, *self.caches,
                                                  slots, status=self.status)
        return self.pk.paged_kv_rotate_append_q8(q, k, v, positions, self.cos_sin, *self.caches,
                                                 *self.scales, slots, status=self.status)

    def tree(self, q, mask, sizes, **kw):
        if self.kv == "bf16":
            return self.pk.paged_decode_attention_tree(
                q, *self.caches, self.tables, self.len_t, mask, self.scale, tree_lens=sizes,
                status=self.status, **kw)
        return self.pk.paged_decode_attention_tree_q8(
            q, *self.caches, *self.scales, self.tables, self.len_t, mask, self.scale,
            tree_lens=sizes, status=self.status, **kw)

    def keep(self, base, path, kept):
        self.pk.paged_kv_keep(*self.caches, self.tables, base, path, kept,
                              *(self.scales if self.kv != "bf16" else ()), status=self.status)

    def decode(self, q):
        if self.kv == "bf16":
            return self.pk.paged_decode_attention(q, *self.caches, self.tables, self.len_t,
                                                  self.scale, status=self.status)
        return self.pk.paged_decode_attention_int8(q, *self.caches, *self.scales, self.tables,
                                                   self.len_t, self.scale, status=self.status)

    def rows(self, s, which):
        """What the cache holds of sequence s: [Hkv, L, D] in 64 bits."""
        n = self.lens[s]
        ids = self.tables[s, :-(-n // self.bs)].long()
        x = self.caches[which][ids].double()
        if self.kv != "bf16":
            x = x * self.scales[which][ids].double()[..., None]
        return x.transpose(0, 1).reshape(self.hkv, -1, self.d)[:, :n]


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("hq,hkv,d,bs,n", [(8, 2, 64, 16, 11), (16, 2, 128, 16, 21),
                                           (8, 8, 128, 32, 7)])
def test_prompts_drafts_and_kept_tokens(kv, hq, hkv, d, bs, n):
    prompts = [37, 0, 150, 5]
    b, t = len(prompts), sum(prompts)
    m = Server(b, hq, hkv, d, bs, kv, nb=60, mbs=20, seed=n)
    # prompts: tokens take their places, are rotated and cached, and attend to their sequence
    slots, positions, offs = m.resize(_i32(prompts), t + 3)
    assert offs.tolist() == offsets(prompts).tolist() and (slots[t:] == -1).all()
    assert positions[:t].tolist() == [i for x in prompts for i in range(x)]
    q = m.append(m.rand(t + 3, hq, d), m.rand(t + 3, hkv, d), m.rand(t + 3, hkv, d), positions,
                 slots)
    k, v = (torch.empty(t + 3, hkv, d, dtype=BF, device="cuda") for _ in range(2))
    m.pk.paged_kv_gather(*m.caches, m.tables, offs, out_k=k, out_v=v,
                         **({} if kv == "bf16" else dict(k_scale=m.scales[0], v_scale=m.scales[1])))
    out = torch.full_like(q, 7.0)
    m.pk.prompt_attention(q, k, v, offs, m.scale, out=out, status=m.status)
    check(out[:t], *prompt_reference(q, k, v, prompts, prompts, m.scale), "prompts")
    assert (out[t:] == 7.0).all()                     # rows behind the last sequence
    if kv == "bf16":
        for s in range(b):
            assert torch.equal(k[offs[s]:offs[s + 1]].double().transpose(0, 1), m.rows(s, 0))
    r = np.random.default_rng(n)
    for step in range(3):
        # a draft: its nodes take the next places, at positions of their depths
        base = m.len_t.clone()
        sizes = [n, max(1, n - 2), n // 2, n]
        mask, seen = random_trees(sizes, 4, n, seed=step)
        depth = torch.zeros(b, n, dtype=torch.int64)
        for s, x in enumerate(seen):
            depth[s, :sizes[s]] = x.sum(1) - 1
        slots, _, offs = m.resize(base + _i32(sizes), b * n)
        node_slots = torch.full((b, n), -1, dtype=torch.int64, device="cuda")
        for s in range(b):
            node_slots[s, :sizes[s]] = slots[offs[s]:offs[s + 1]]
        places = (base[:, None].long() + depth.cuda()).view(-1)
        q = m.append(m.rand(b * n, hq, d), m.rand(b * n, hkv, d), m.rand(b * n, hkv, d), places,
                     node_slots.view(-1)).view(b, n, hq, d)
        out = m.tree(q, mask.cuda(), _i32(sizes))
        check(out, *tree_reference(m, q, seen, sizes, m.scale), f"draft {step}")
        # one path stays, the rest goes back
        path, kept = np.zeros((b, n), np.int32), np.zeros(b, np.int32)
        for s in range(b):
            nodes = np.nonzero(seen[s][r.integers(0, sizes[s])].numpy())[0]
            kept[s] = 0 if step == 1 and s == 2 else len(nodes)
            path[s, :len(nodes)] = nodes
        want = [[m.rows(s, w)[:, [*range(base[s]), *(int(base[s]) + i for i in path[s, :kept[s]])]]
                 for w in range(2)] for s in range(b)]
        m.keep(base, torch.from_numpy(path).cuda(), torch.from_numpy(kept).cuda())
        m.resize(base + torch.from_numpy(kept).cuda())
        assert m.lens == [int(x) + int(y) for x, y in zip(base.tolist(), kept)]
        for s in range(b):
            for w in range(2):
                assert torch.equal(m.rows(s, w), want[s][w])
        # and one token goes the plain way
        slots, positions, offs = m.resize(m.len_t + 1, b)
        q = m.append(m.rand(b, hq, d), m.rand(b, hkv, d), m.rand(b, hkv, d), positions, slots)
        out = m.decode(q)
        for s in range(b):
            all_seen = torch.ones(1, m.lens[s], dtype=torch.bool, device="cuda")
            o, e = attend(q[s][:, None], m.rows(s, 0), m.rows(s, 1), all_seen, m.scale, HALF,
                          0.0 if kv == "bf16" else HALF16)
            check(out[s], o[0], e[0], f"decode {step}")
    assert m.status.item() == 0
    m.resize(_i32([0] * b))
    assert m.count.item() == 60 and sorted(m.free.tolist()) == list(range(60))


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_a_draft_round_in_a_graph(kv):
    """Growing, tree attention, keeping and shrinking as one captured graph, replayed, next to
    the same calls made one by one, on another stream than the caller's."""
    b, hq, hkv, d, bs, n = 3, 16, 2, 64, 16, 20
    runs = []
    for captured in (False, True):
        m = Server(b, hq, hkv, d, bs, kv, nb=40, mbs=12, seed=5)
        m.resize(_i32([30, 1, 64]), 0)                 # (rows do not fit: nothing grows)
        assert m.lens == [0, 0, 0] and m.status.item() == m.pk.pagedkv.DEV_NO_BLOCKS
        m.status.zero_()
        t = 95
        slots, positions, _ = m.resize(_i32([30, 1, 64]), t)
        m.append(m.rand(t, hq, d), m.rand(t, hkv, d), m.rand(t, hkv, d), positions, slots)
        mask, _ = random_trees([n] * b, 3, n, seed=1)
        mask = mask.cuda()
        sizes, grown, back = _i32([n] * b), m.len_t + n, m.len_t + 2
        base, path, kept = m.len_t.clone(), _i32([[0, 3]] * b), _i32([2, 2, 2])
        q, k, v = m.rand(b * n, hq, d), m.rand(b * n, hkv, d), m.rand(b * n, hkv, d)
        rows = [torch.empty(b * n, dtype=torch.int64, device="cuda") for _ in range(2)]
        offs = torch.empty(b + 1, dtype=torch.int32, device="cuda")
        rotated, out = torch.empty_like(q), torch.empty(b, n, hq, d, dtype=BF, device="cuda")
        ws = torch.empty(m.pk.tree_workspace_bytes(b, hq, hkv, d, bs, 40, 12, n,
                                                   m.pk.pagedkv.KV_BF16 if kv == "bf16"
                                                   else m.pk.pagedkv.KV_INT8),
                         dtype=torch.uint8, device="cuda")

        def step():
            m.pk.paged_kv_resize(m.tables, m.len_t, grown, m.free, m.count, bs, b * n, *rows, offs,
                                 status=m.status)
            if kv == "bf16":
                m.pk.paged_kv_rotate_append(q, k, v, rows[1], m.cos_sin, *m.caches, rows[0],
                                            out=rotated)
            else:
                m.pk.paged_kv_rotate_append_q8(q, k, v, rows[1], m.cos_sin, *m.caches, *m.scales,
                                               rows[0], out=rotated)
            m.tree(rotated.view(b, n, hq, d), mask, sizes, out=out, workspace=ws)
            m.keep(base, path, kept)
            m.resize(back)
            grown.add_(2), back.add_(2), base.add_(2)

        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            if captured:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=stream):
                    step()
            outs = []
            for _ in range(3):
                graph.replay() if captured else step()
                outs.append(out.clone())
        stream.synchronize()
        assert m.status.item() == 0
        runs.append((outs, m.lens, m.tables.tolist(), m.free.tolist(), m.count.item(),
                     [m.rows(s, w) for s in range(b) for w in range(2)]))
    assert runs[0][1] == [36, 7, 70]
    assert runs[0][1:5] == runs[1][1:5]
    for x, y in zip(runs[0][0] + runs[0][5], runs[1][0] + runs[1][5]):
        assert torch.equal(x, y)
