"""Refusals of resize, keep, tree and prompt attention, by the library's host checks and by the
binding's, without a GPU."""

import ctypes

import pytest
import torch

from test_cabi import lib_path  # noqa: F401

P = ctypes.c_void_p(0x1000)
MIS = ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def lib(lib_path):  # noqa: F811
    from paged_kv_decode_02_gb300 import pagedkv
    lib = pagedkv.load_library(lib_path)
    before = lib.pkv_kernel_launch_count()
    yield lib
    assert lib.pkv_kernel_launch_count() == before          # nothing reached a launch


def _good(**kw):
    from paged_kv_decode_02_gb300 import pagedkv
    f = dict(num_seqs=4, num_q_heads=8, num_kv_heads=4, head_dim=64, block_size=16,
             num_blocks=64, max_blocks_per_seq=4)
    f.update(kw)
    return pagedkv.Dims(**f)


def test_resize_refusals(lib):
    from paged_kv_decode_02_gb300.pagedkv import Status

    def resize(tables=P, lens=P, free=P, count=P, cap=10, slots=P, offsets=P, n=5, **dims):
        return lib.pkv_resize_sequences(tables, lens, P, free, count, cap, slots, P, offsets, n,
                                        ctypes.byref(_good(**dims)), None, None)
    for name in ("tables", "lens", "free", "count", "slots", "offsets"):
        assert resize(**{name: None}) == Status.ERR_NULL
    assert resize(cap=-1) == Status.ERR_SHAPE
    assert resize(n=-1) == Status.ERR_SHAPE
    assert resize(block_size=24) == Status.ERR_UNSUPPORTED
    assert resize(num_seqs=16385) == Status.ERR_UNSUPPORTED
    assert resize(cap=1 << 30) == Status.ERR_UNSUPPORTED
    assert resize(n=1 << 30) == Status.ERR_UNSUPPORTED
    assert resize(num_seqs=16384, max_blocks_per_seq=1 << 16) == Status.ERR_UNSUPPORTED
    assert resize(num_seqs=0) == Status.OK


def test_keep_refusals(lib):
    from paged_kv_decode_02_gb300.pagedkv import Status

    def keep(k=P, ks=None, tables=P, path=P, width=3, kv=0, **dims):
        return lib.pkv_keep_tokens(k, P, ks, ks, tables, P, path, None, width, kv,
                                   ctypes.byref(_good(**dims)), None, None)
    for name in ("k", "tables", "path"):
        assert keep(**{name: None}) == Status.ERR_NULL
    assert keep(kv=1) == Status.ERR_NULL                    # one-byte caches need scales
    assert keep(kv=4) == Status.ERR_DTYPE
    assert keep(width=-1) == Status.ERR_SHAPE
    assert keep(k=MIS) == Status.ERR_ALIGNMENT
    assert keep(head_dim=96) == Status.ERR_UNSUPPORTED
    assert keep(width=0) == Status.OK
    assert keep(num_seqs=0) == Status.OK


def test_tree_refusals(lib):
    from paged_kv_decode_02_gb300.pagedkv import Status
    n = ctypes.c_size_t(0)

    def tree(out=P, mask=P, q_len=4, kv=0, scale=P, **dims):
        d = ctypes.byref(_good(**dims))
        if kv == 0:
            return lib.pkv_decode_tree_bf16(out, P, P, P, P, P, mask, None, q_len, 0.1, d, P,
                                            1 << 30, None, None)
        return lib.pkv_decode_tree_q8(out, P, P, P, scale, P, P, P, mask, None, q_len, 0.1, kv, d,
                                      P, 1 << 30, None, None)
    for kv in (0, 1):
        assert tree(mask=None, kv=kv) == Status.ERR_NULL
        assert tree(out=None, kv=kv) == Status.ERR_NULL
        assert tree(out=MIS, kv=kv) == Status.ERR_ALIGNMENT
        assert tree(q_len=0, kv=kv) == Status.ERR_SHAPE
        assert tree(q_len=257, kv=kv) == Status.ERR_SHAPE
        assert tree(num_q_heads=9, kv=kv) == Status.ERR_SHAPE
        assert tree(num_seqs=0, kv=kv) == Status.OK
    assert tree(kv=1, scale=None) == Status.ERR_NULL
    assert tree(kv=1, scale=MIS) == Status.ERR_ALIGNMENT
    assert tree(kv=7) == Status.ERR_DTYPE
    good = _good()
    ws = lib.pkv_decode_tree_workspace_bytes
    assert ws(ctypes.byref(good), 4, 0, None) == Status.ERR_NULL
    assert ws(ctypes.byref(good), 4, 9, ctypes.byref(n)) == Status.ERR_DTYPE
    assert ws(ctypes.byref(good), 257, 0, ctypes.byref(n)) == Status.ERR_SHAPE


def _prompt(**kw):
    from paged_kv_decode_02_gb300 import pagedkv
    f = dict(num_seqs=2, num_q_heads=8, num_kv_heads=4, head_dim=64, num_q_tokens=10,
             num_kv_tokens=12, out_stride=512, q_stride=1024, k_stride=256, v_stride=256)
    f.update(kw)
    return pagedkv._pack_prompt(*f.values())


def test_prompt_host_checks(lib):
    """Checks that come before the device is asked for anything."""
    from paged_kv_decode_02_gb300.pagedkv import Status
    n = ctypes.c_size_t(0)

    def size(**kw):
        return lib.pkv_prompt_workspace_bytes(_prompt(**kw), ctypes.byref(n))
    assert lib.pkv_prompt_workspace_bytes(_prompt(), None) == Status.ERR_NULL
    assert lib.pkv_prompt_workspace_bytes(None, ctypes.byref(n)) == Status.ERR_NULL
    assert size(num_seqs=-1) == Status.ERR_SHAPE
    assert size(num_q_heads=6) == Status.ERR_SHAPE
    assert size(num_kv_heads=0) == Status.ERR_SHAPE
    assert size(num_q_tokens=-1) == Status.ERR_SHAPE
    assert size(head_dim=96) == Status.ERR_UNSUPPORTED
    assert size(num_q_heads=129, num_kv_heads=1) == Status.ERR_UNSUPPORTED
    assert size(num_kv_tokens=1 << 30) == Status.ERR_UNSUPPORTED

    def call(out=P, q=P, k=P, off=P, ws=P, **kw):
        return lib.pkv_prompt_attention_bf16(out, q, k, P, off, P, 0.1, _prompt(**kw), ws, 1 << 40,
                                             None, None)
    assert call(q_stride=504) == Status.ERR_SHAPE
    assert call(v_stride=248) == Status.ERR_SHAPE
    assert call(k_stride=260) == Status.ERR_ALIGNMENT
    assert call(out_stride=1 << 38) == Status.ERR_UNSUPPORTED
    for name in ("out", "q", "k", "off"):
        assert call(**{name: None}) == Status.ERR_NULL
    assert call(q=MIS) == Status.ERR_ALIGNMENT
    assert call(k=MIS) == Status.ERR_ALIGNMENT
    assert call(ws=None) == Status.ERR_WORKSPACE
    assert call(ws=MIS) == Status.ERR_WORKSPACE
    assert call(num_seqs=0) == Status.OK
    assert call(num_q_tokens=0) == Status.OK


def test_binding_refuses_host_tensors():
    """Every entry point of the binding turns down host memory before any library call."""
    import paged_kv_decode_02_gb300 as pk
    bf = torch.bfloat16
    kc = torch.zeros(6, 2, 16, 64, dtype=bf)
    codes, sc = torch.zeros(6, 2, 16, 64, dtype=torch.int8), torch.zeros(6, 2, 16)
    q, rows = torch.zeros(3, 2, 4, 64, dtype=bf), torch.zeros(3, 4, 64, dtype=bf)
    tab, lens = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    mask, off = torch.zeros(3, 2, 1, dtype=torch.int64), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: pk.paged_kv_resize(tab, lens, lens + 1, lens, lens[:1], 16),
                 lambda: pk.paged_kv_keep(kc, kc, tab, lens, tab),
                 lambda: pk.paged_decode_attention_tree(q, kc, kc, tab, lens, mask, 1.0),
                 lambda: pk.paged_decode_attention_tree_q8(q, codes, codes, sc, sc, tab, lens, mask,
                                                           1.0),
                 lambda: pk.prompt_attention(rows, rows, rows, off, 1.0)):
        with pytest.raises(ValueError):
            call()
