"""attn_extend and the decode cascade mask before they scale, so they need a
positive scale, whatever the pool's format: refused on the host (CPU)."""
from __future__ import annotations

import ctypes as C

import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra
from tests.test_workspace_bounds import attn_desc

FORMATS = ["bf16", "fp8", "fp4"]
BAD = [0.0, -0.1, float("nan")]


def call(name, fmt, scale, cascade=False):
    """The call with host pointers, which only its checks may meet."""
    desc = attn_desc(fmt, 32, 8, 128)
    desc.sm_scale = scale
    buf = torch.zeros(1 << 12, dtype=torch.uint8)
    b = (buf.data_ptr() + 255) // 256 * 256
    kv = ra.rc_kv_table(slots=b, start=b, len=b, max_len=16, table_len=64)
    L = ra.lib()
    if name == "extend":
        return L.attn_extend(C.byref(desc), b, b, C.byref(kv), 2, 8, b, None, None, 0, None)
    casc = ra.rc_cascade(n_seg=1, total_seg_rows=2, max_seg_rows=2, max_seg_len=8, seg_slots=b, seg_indptr=b,
                         seg_row_indptr=b, seg_rows=b, req_seg_indptr=b, req_seg_pos=b)
    if name == "append":
        return L.attn_decode_append(C.byref(desc), b, b, b, C.byref(kv), 2, C.byref(casc), b, None, b, 1 << 24, None)
    if name == "steps":
        step = (ra.rc_decode_step * 1)()
        step[0].q = step[0].out = step[0].len = b
        step[0].max_len = 16
        return L.attn_decode_steps(C.byref(desc), C.byref(kv), 2, C.byref(casc), step, 1, b, 1 << 24, None, None)
    return L.attn_decode(C.byref(desc), b, C.byref(kv), 2, C.byref(casc), b, None, b, 1 << 24, None)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", BAD)
@pytest.mark.parametrize("name", ["extend", "cascade", "append", "steps"])
def test_refused(built, name, fmt, scale):
    if name == "append" and fmt != "bf16":
        assert call(name, fmt, scale) in (ra.RC_ERR_ARG, ra.RC_ERR_UNSUPPORTED)
    else:
        assert call(name, fmt, scale) == ra.RC_ERR_ARG
