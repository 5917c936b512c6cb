"""Resize of batches whose sums are about as large as the shared memory of a CTA that asks for none."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_batches_around_the_default_shared_memory():
    """The sums of some 4030 sequences and more pass what a CTA has without asking. In a process of
    its own, in rising order: a larger batch before would have asked for all that follow."""
    code = """
import torch, paged_kv_decode_02_gb300 as pk
put = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
for tokens in (4096, 9000):          # one CTA; CTAs on every SM and the commit
    for b in (4028, 4029, 4030, 4031, 4095, 4096, 4097):
        ids = torch.randperm(2 * b).int().cuda()
        tables, lens, count = put([[-5] * 2] * b), put([0] * b), put([2 * b])
        want = put([(s % 3 if tokens > 4096 else s % 2) for s in range(b)])
        status = put([0])
        slots, pos, offs = pk.paged_kv_resize(tables, lens, want, ids, count, 16,
                                              num_tokens=tokens, status=status)
        assert status.item() == 0 and torch.equal(lens, want)
        n = int(want.sum())
        assert offs.tolist() == [0] + want.cumsum(0).tolist()
        assert count.item() == 2 * b - int((want > 0).sum())
        assert (slots[:n] // 16 == tables[:, 0].repeat_interleave(want.long()).long()).all()
        assert (slots[n:] == -1).all()
    z = put([0] * 4090)              # and without tokens: both forms of a call that only shrinks
    for width in (1, 64):
        tables = torch.zeros(4090, width, dtype=torch.int32, device="cuda")
        pk.paged_kv_resize(tables, z.clone(), z, put([0]), put([0]), 16)
torch.cuda.synchronize()
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
