"""Refusals of rotate-and-append, gather and differential decode, by the library's host
checks and by the binding's, without a GPU."""

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


def _good():
    from paged_kv_decode_02_gb300 import pagedkv
    return pagedkv.Dims(4, 8, 4, 64, 16, 64, 4)


def _rotary(**kw):
    from paged_kv_decode_02_gb300 import pagedkv
    f = dict(cos_sin=0x1000, q_norm=None, k_norm=None, out_stride=512, q_stride=1024,
             k_stride=1024, v_stride=1024, num_positions=100, rotary_dim=64, interleaved=0,
             eps=1e-6)
    f.update(kw)
    return pagedkv.Rotary(**f)


def _rotate(lib, ro, dims=None, q=P, T=3, slots=P):
    dims = dims or _good()
    return lib.pkv_rotate_append_bf16(P, q, P, P, P, ctypes.byref(ro) if ro else None, P, P, slots,
                                      T, ctypes.byref(dims), None, None)


def test_rotate_refusals(lib):
    from paged_kv_decode_02_gb300.pagedkv import Dims, Status
    assert _rotate(lib, None) == Status.ERR_NULL
    assert _rotate(lib, _rotary(), q=None) == Status.ERR_NULL
    assert _rotate(lib, _rotary(), slots=None) == Status.ERR_NULL
    assert _rotate(lib, _rotary(cos_sin=None)) == Status.ERR_NULL
    assert _rotate(lib, _rotary(), q=MIS) == Status.ERR_ALIGNMENT
    assert _rotate(lib, _rotary(q_norm=0x1008)) == Status.ERR_ALIGNMENT
    assert _rotate(lib, _rotary(cos_sin=0x1004)) == Status.ERR_ALIGNMENT
    assert _rotate(lib, _rotary(k_stride=1028)) == Status.ERR_ALIGNMENT
    assert _rotate(lib, _rotary(k_stride=248)) == Status.ERR_SHAPE      # less than Hkv * D
    assert _rotate(lib, _rotary(q_stride=504)) == Status.ERR_SHAPE
    assert _rotate(lib, _rotary(rotary_dim=0)) == Status.ERR_SHAPE
    assert _rotate(lib, _rotary(rotary_dim=80)) == Status.ERR_SHAPE     # more than D
    assert _rotate(lib, _rotary(rotary_dim=24)) == Status.ERR_UNSUPPORTED
    assert _rotate(lib, _rotary(num_positions=0)) == Status.ERR_SHAPE
    assert _rotate(lib, _rotary(), T=-1) == Status.ERR_SHAPE
    assert _rotate(lib, _rotary(), T=0) == Status.OK
    assert _rotate(lib, _rotary(), dims=Dims(4, 8, 4, 96, 16, 64, 4)) == Status.ERR_UNSUPPORTED
    # in place, the rows of q and q_out have to be the same
    assert _rotate(lib, _rotary(out_stride=512, q_stride=1024)) == Status.ERR_SHAPE
    good = _good()
    ro = _rotary()
    for kv in (0, 9):
        assert lib.pkv_rotate_append_q8(P, P, P, P, P, ctypes.byref(ro), P, P, P, P, P, 3, kv,
                                        ctypes.byref(good), None, None) == Status.ERR_DTYPE
    assert lib.pkv_rotate_append_q8(P, P, P, P, P, ctypes.byref(ro), P, P, None, P, P, 3, 1,
                                    ctypes.byref(good), None, None) == Status.ERR_NULL


def test_gather_refusals(lib):
    from paged_kv_decode_02_gb300.pagedkv import Status
    good = _good()

    def gather(out=P, scale=None, offsets=P, n=5, kv=0, cache=P):
        return lib.pkv_gather_tokens(out, P, cache, P, scale, scale, P, None, offsets, n, kv,
                                     ctypes.byref(good), None, None)
    assert gather(out=None) == Status.ERR_NULL
    assert gather(offsets=None) == Status.ERR_NULL
    assert gather(kv=1) == Status.ERR_NULL                  # one-byte caches need scales
    assert gather(kv=4) == Status.ERR_DTYPE
    assert gather(n=-1) == Status.ERR_SHAPE
    assert gather(n=0) == Status.OK
    assert gather(out=MIS) == Status.ERR_ALIGNMENT
    assert gather(cache=MIS) == Status.ERR_ALIGNMENT


def test_diff_refusals(lib):
    from paged_kv_decode_02_gb300.pagedkv import Dims, Status
    n = ctypes.c_size_t(0)

    def diff(dims=None, out=P, lam=P, nw=None, kv=0, scale=P):
        dims = dims or _good()
        if kv == 0:
            return lib.pkv_decode_diff_bf16(out, P, P, P, P, P, lam, nw, 1e-5, 1.0, 0.1,
                                            ctypes.byref(dims), P, 1 << 30, None, None)
        return lib.pkv_decode_diff_q8(out, P, P, P, scale, P, P, P, lam, nw, 1e-5, 1.0, 0.1, kv,
                                      ctypes.byref(dims), P, 1 << 30, None, None)
    assert diff(out=None) == Status.ERR_NULL
    assert diff(lam=None) == Status.ERR_NULL
    assert diff(nw=MIS) == Status.ERR_ALIGNMENT
    assert diff(kv=1, scale=None) == Status.ERR_NULL
    assert diff(kv=1, scale=MIS) == Status.ERR_ALIGNMENT
    assert diff(kv=7) == Status.ERR_DTYPE
    odd = Dims(4, 6, 3, 64, 16, 64, 4)                       # an odd number of KV heads
    odd_q = Dims(4, 1, 1, 64, 16, 64, 4)
    for dims in (odd, odd_q):
        assert diff(dims) == Status.ERR_SHAPE
        assert lib.pkv_decode_diff_workspace_bytes(ctypes.byref(dims), 0, ctypes.byref(n)) == \
            Status.ERR_SHAPE
    assert diff(Dims(0, 8, 4, 64, 16, 64, 4)) == Status.OK   # no sequences
    huge = Dims(17, 8, 4, 64, 16, 64, (1 << 27) - 1)         # more items than 32 bits count
    assert diff(huge) == Status.ERR_UNSUPPORTED
    good = _good()
    assert lib.pkv_decode_diff_workspace_bytes(ctypes.byref(good), 0, None) == Status.ERR_NULL
    assert lib.pkv_decode_diff_workspace_bytes(ctypes.byref(good), 4, ctypes.byref(n)) == \
        Status.ERR_DTYPE


def test_binding_refuses_host_tensors():
    """Every entry point of the binding turns down host memory before any library call."""
    import paged_kv_decode_02_gb300 as pk
    bf = torch.bfloat16
    kc = torch.zeros(6, 2, 16, 64, dtype=bf)
    codes, sc = torch.zeros(6, 2, 16, 64, dtype=torch.int8), torch.zeros(6, 2, 16)
    q, k = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, 2, 64, dtype=bf)
    pos = torch.zeros(3, dtype=torch.int64)
    cs = torch.zeros(8, 64)
    tab, lens = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    for call in (lambda: pk.paged_kv_rotate_append(q, k, k, pos, cs, kc, kc, pos),
                 lambda: pk.paged_kv_rotate_append_q8(q, k, k, pos, cs, codes, codes, sc, sc, pos),
                 lambda: pk.paged_kv_gather(kc, kc, tab, torch.zeros(4, dtype=torch.int32), 3),
                 lambda: pk.paged_decode_attention_diff(q, kc, kc, tab, lens, torch.zeros(2), 1.0),
                 lambda: pk.paged_decode_attention_diff_q8(q, codes, codes, sc, sc, tab, lens,
                                                           torch.zeros(2), 1.0)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        pk.paged_decode_attention_diff_q8(q, kc, kc, sc, sc, tab, lens, torch.zeros(2), 1.0)
