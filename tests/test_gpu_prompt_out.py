"""Prompt attention: outputs that are an input."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_output_in_place_is_refused():
    """A query row is read where the keys are cut, after other rows have been written."""
    import paged_kv_decode_02_gb300 as pk
    rows = torch.zeros(20, 4, 64, dtype=torch.bfloat16, device="cuda")
    k, v = torch.zeros_like(rows), torch.zeros_like(rows)
    off = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    for out in (rows, k, v):
        with pytest.raises(ValueError, match="out"):
            pk.prompt_attention(rows, k, v, off, 1.0, out=out)
    # (parts of one buffer that do not overlap are taken)
    both = torch.zeros(20, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    got = pk.prompt_attention(both[:, 0], k, v, off, 1.0, out=both[:, 1])
    assert (got == 0).all()
