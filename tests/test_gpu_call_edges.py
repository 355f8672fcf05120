"""Calls at the edge of what the header allows: the largest bounds, unused axes, very many prompts."""
from __future__ import annotations

import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("w", [2, 6, 11, 32])
def test_reorder_without_a_bound_on_columns(cuda, w):
    """max_cols up to the largest whole number: the grid follows the table."""
    b, room, cols = 3, 40, 25
    table = torch.arange(b * w * room, dtype=torch.int32, device=cuda)
    start = (torch.arange(b * w, dtype=torch.int32, device=cuda) * room).view(b, w)
    first = torch.full((b,), 5, dtype=torch.int32, device=cuda)
    par = torch.arange(w, dtype=torch.int32, device=cuda).flip(0).repeat(b, 1).contiguous()
    want = table.clone().view(b, w, room)
    want[:, :, 5:5 + cols] = want[:, :, 5:5 + cols].flip(1)
    for bound in (cols, 2 ** 31 - 1, 2 ** 31 - 128, 2 ** 31 - 600):
        out, err = table.clone(), torch.zeros(1, dtype=torch.int32, device=cuda)
        ra.beam_reorder(out, start, first, first + cols, par, bound, err=err)
        assert ra.rc_sync(err) == ra.RC_OK
        assert torch.equal(out.view(b, w, room), want)
    # more columns than the table has entries is more than any bound
    out = table.clone()
    ra.beam_reorder(out, start, first, first + b * w * room + 1, par, 2 ** 31 - 1, err=err)
    assert ra.rc_sync(err) == ra.RC_ERR_DEVICE and torch.equal(out, table)
    # an empty table: rows without columns are fine, others are not in it
    zero = torch.zeros_like(start)
    for last, st in ((first, ra.RC_OK), (first + 1, ra.RC_ERR_DEVICE)):
        torch.cuda.synchronize()
        got = ra.lib().beam_reorder(out.data_ptr(), out.data_ptr(), 0, zero.data_ptr(), first.data_ptr(), last.data_ptr(),
                                    par.data_ptr(), b, w, 2 ** 31 - 1, err.data_ptr(), None)
        assert got == ra.RC_OK and ra.rc_sync(err) == st
    assert torch.equal(out, table)
