"""The oracle's differential attention of a workload on the GPU, with a bound on what the
kernel may be off, element by element. Nothing here touches the CUDA library."""

import numpy as np
import torch

import oracle
from parity_helpers import sequence_blocks, to_f64

# fp32 parts of a weight's relative error: a score is a sum of up to 128 products plus a
# scale (its absolute error is below 130 * 2^-24 * sum |q k| * scale, and sum |q k| * scale
# stays below 2^6 on these inputs: 2^-11), the exponential's is 2^-22, sums over up to
# 2^14 tokens add 2^-10 at the very worst
FP32_SLACK = 2.0 ** -9


def rows_of(w, s, which):
    """Hkv arrays [L, D] of sequence s's cached K or V values, and the codes' magnitudes."""
    L, blocks = sequence_blocks(w, s)
    cache = (w.k_cache if which == "k" else w.v_cache)[blocks]
    scale = w.k_scale if which == "k" else w.v_scale
    table, bs = np.arange(len(blocks)), w.block_size
    vals, codes = [], []
    for h in range(cache.shape[1]):
        if scale is None:
            v = oracle.gather_sequence(to_f64(cache), table, L, h, bs)
            codes.append(np.abs(v))
        else:
            sc = scale[blocks].cpu().numpy()
            c = cache.cpu().numpy()
            if w.kv_dtype == "int8":
                v = oracle.gather_sequence_int8(c, sc, table, L, h, bs)
            else:
                v = oracle.gather_sequence_fp8(c, sc, table, L, h, bs, w.kv_dtype[4:])
            flat = sc[:, h].reshape(-1)[:L]
            codes.append(np.abs(v) / flat[:, None] if L else v)
        vals.append(v)
    return vals, codes


def diff_reference(w, lam, norm_weight=None, eps=0.0, out_scale=1.0):
    """(out, bound) [B, Hq / 2, 2 D] in float64.

    Per map, the weighted mean O_m = sum a v of rounded weights a (1 + d): off by at most
    u * sum a |v|. bf16 caches: a weight is two bf16 terms, u = 2^-8 * 2^-8 = 2^-16; one-byte
    caches: weight times V scale in fp16, u = 2^-11, plus half a subnormal step of fp16,
    2^-25, times the code, over the row sum, which is at least 1, of the scaled weight. Then |lambda| times that for the second map, through the
    norm to first order, and half a step of the bf16 output."""
    B, Hq, D = w.q.shape
    q = to_f64(w.q)
    lam = to_f64(lam)
    nw = None if norm_weight is None else to_f64(norm_weight)
    up = {"bf16": 1.0, "int8": 64.0, "fp8_e4m3": 256.0, "fp8_e5m2": 32768.0}[w.kv_dtype]
    out = np.zeros((B, Hq // 2, 2 * D))
    bound = np.zeros_like(out)
    g = w.group
    for s in range(B):
        keys, _ = rows_of(w, s, "k")
        values, codes = rows_of(w, s, "v")
        if len(keys[0]) == 0:
            continue
        raw, maps = oracle.decode_attention_diff(q[s], keys, values, lam, w.scale)
        for j in range(Hq // 2):
            p = j // g
            v = np.concatenate([values[2 * p], values[2 * p + 1]], 1)
            c = np.concatenate([codes[2 * p], codes[2 * p + 1]], 1)
            e = np.zeros(2 * D)
            for m in range(2):
                a = maps[j, m][:, None]
                o = np.sum(a * v, 0)
                off = FP32_SLACK * np.sum(a * np.abs(v - o), 0) + 2.0 ** -20 * np.abs(o)
                if w.kv_dtype == "bf16":
                    off += 2.0 ** -16 * np.sum(a * np.abs(v), 0)
                else:
                    off += 2.0 ** -11 * np.sum(a * np.abs(v), 0)
                    off += 2.0 ** -25 / up * np.sum(c, 0) * maps[j, m].max()
                e += off * (1.0 if m == 0 else abs(lam[j]))
            y, f = raw[j], 1.0
            if nw is not None:
                ms = np.mean(y * y) + eps
                # d(y / rms): its own error, and the row's through the root mean square
                e = (e + np.abs(y) * np.sum(np.abs(y) * e) / (2 * D) / ms) * 1.05
                f = np.abs(nw) / np.sqrt(ms)
                y = y / np.sqrt(ms) * nw
            out[s, j] = y * out_scale
            bound[s, j] = e * f * abs(out_scale) + 2.0 ** -8 * np.abs(out[s, j])
    return out, bound


def assert_diff(got, ref, bound):
    got = to_f64(got)
    assert np.all(np.isfinite(got))
    off = np.abs(got - ref)
    worst = np.max(off - bound)
    assert np.all(off <= bound + 1e-30), f"off by {off.max():.3e}, over the bound by {worst:.3e}"


def random_lambda(num_q_heads, dev, seed=0):
    gen = torch.Generator(device=dev).manual_seed(seed)
    lam = 0.1 + 0.9 * torch.rand(num_q_heads // 2, generator=gen, device=dev)
    lam[0] = 0.0
    lam[-1] = -0.5
    return lam


def random_norm(D, dev, seed=0):
    gen = torch.Generator(device=dev).manual_seed(seed + 1)
    return (1 + 0.3 * torch.randn(2 * D, generator=gen, device=dev)).to(torch.bfloat16)
