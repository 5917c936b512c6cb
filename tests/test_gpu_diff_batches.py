"""Differential decode of very large batches: the sequences' table in shared memory."""

import ctypes

import pytest
import torch

from diff_helpers import assert_diff, diff_reference, random_lambda
from paged_kv_decode_02_gb300.workloads import make_workload

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pk():
    from paged_kv_decode_02_gb300 import build_lib
    build_lib.build()
    import paged_kv_decode_02_gb300 as pk
    pk.load_library()
    return pk


def call(pk, w, lam, **kw):
    if w.kv_dtype == "bf16":
        return pk.paged_decode_attention_diff(w.q, w.k_cache, w.v_cache, w.block_tables,
                                              w.context_lens, lam, w.scale, **kw)
    return pk.paged_decode_attention_diff_q8(w.q, w.k_cache, w.v_cache, w.k_scale, w.v_scale,
                                             w.block_tables, w.context_lens, lam, w.scale, **kw)


@pytest.mark.parametrize("kv,hq,hkv,d", [("bf16", 8, 2, 128), ("bf16", 16, 2, 128),
                                         ("int8", 16, 2, 128), ("int8", 4, 2, 64)])
@pytest.mark.parametrize("copies", [500, 1250])
def test_batches_that_leave_room_for_fewer_ctas(pk, kv, hq, hkv, d, copies):
    """24 short sequences, 500 and 1250 times over (on the same blocks): every copy gives what
    the oracle gives for its sequence, and the bits that the 24 alone give (no unit is cut)."""
    lengths = [0, 1, 2, 15, 16, 17, 31, 32] * 3
    w = make_workload({"bf16": "70b-gqa", "int8": "int8"}[kv], device=DEV, lengths=lengths,
                      num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=16)
    lam = random_lambda(hq, DEV)
    few = call(pk, w, lam)
    ref, bound = diff_reference(w, lam)
    assert_diff(few, ref, bound)
    w.q, w.block_tables, w.context_lens = (x.repeat((copies,) + (1,) * (x.dim() - 1))
                                           for x in (w.q, w.block_tables, w.context_lens))
    many = call(pk, w, lam, status=torch.zeros(1, dtype=torch.int32, device=DEV))
    assert torch.equal(many.view(copies, *few.shape), few.expand(copies, *few.shape))


@pytest.mark.parametrize("kv", [0, 1, 2, 3])
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 32)])
def test_batches_past_the_table_are_refused(pk, kv, d, bs):
    """30000 sequences are taken whatever the shape; 60000 are refused by the query and by the
    call (before any launch)."""
    lib = pk.load_library()
    n, p = ctypes.c_size_t(0), ctypes.c_void_p(0x1000)
    for g in (1, 4, 8, 12, 16, 17):
        for seqs, want in ((30000, pk.Status.OK), (60000, pk.Status.ERR_UNSUPPORTED)):
            dims = pk.Dims(seqs, 2 * g, 2, d, bs, 64, 4)
            assert lib.pkv_decode_diff_workspace_bytes(ctypes.byref(dims), kv,
                                                       ctypes.byref(n)) == want
        before = lib.pkv_kernel_launch_count()
        tail = (p, p, p, None, 1e-5, 1.0, 0.1) + ((kv,) if kv else ()) + \
            (ctypes.byref(dims), p, 1 << 40, None, None)
        if kv == 0:
            st = lib.pkv_decode_diff_bf16(p, p, p, p, *tail)
        else:
            st = lib.pkv_decode_diff_q8(p, p, p, p, p, p, *tail)
        assert st == pk.Status.ERR_UNSUPPORTED and lib.pkv_kernel_launch_count() == before
