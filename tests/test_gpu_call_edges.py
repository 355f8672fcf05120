"""Calls at the edge of what the header allows: the largest bounds, unused axes, very many prompts."""
from __future__ import annotations

import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra
from tests.test_gpu_pool_rows import make_pool

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


@pytest.mark.parametrize("sections", [[32, 32, 0], [64, 0, 0], [20, 0, 44, 0]])
@pytest.mark.parametrize("n", [1, 300])
def test_positions_on_an_axis_that_no_pair_turns_by(cuda, sections, n):
    """A model of three axes whose last section is empty passes its [3, n] positions; the last row has no effect."""
    g = torch.Generator(device=cuda).manual_seed(n)
    axis = ra.rope_axes(sections)
    used, rope = max(axis) + 1, ra.make_rope_desc(ra.rope_table(50, 128, device=cuda), pair_axis=axis)
    pos = torch.randint(0, 50, (len(sections), n), generator=g, device=cuda).to(torch.int32)
    pos[used:] = -7
    k, v = (torch.randn(n, 2, 128, generator=g, device=cuda).to(BF) for _ in range(2))
    slots = torch.randperm(n, generator=g, device=cuda).to(torch.int32)
    got = []
    for p in (pos, pos[:used].contiguous() if used > 1 else pos[0]):
        pool, arrays, err = make_pool("bf16", n, 2, 128, cuda)
        ra.kv_store_rope(pool, rope, slots, p, k, v)
        assert ra.rc_sync(err) == ra.RC_OK
        got.append(arrays)
    assert all(torch.equal(a, b) for a, b in zip(*got)) and torch.equal(got[0][1][slots.long()], v)
