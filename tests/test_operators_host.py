"""Refusals of kv_store_rope, attn_cross and the 4-bit pool: every call here
fails its checks on the host, before any CUDA call."""
from __future__ import annotations

import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


def fp4_tensors(n=64, hkv=8, d=128):
    codes = lambda: torch.zeros(n, hkv, d // 2, dtype=torch.uint8)
    scales = lambda: torch.zeros(n, hkv, d // 16, dtype=torch.uint8)
    return codes(), codes(), scales(), scales()


def fp4_pool(n=64, hkv=8, d=128):
    k, v, ks, vs = fp4_tensors(n, hkv, d)
    return ra.make_pool_desc(k, v, k_bscale=ks, v_bscale=vs)


def bf16_pool(n=64, hkv=8, d=128):
    return ra.make_pool_desc(torch.zeros(n, hkv, d, dtype=BF), torch.zeros(n, hkv, d, dtype=BF))


def test_rope_struct_matches_the_header(tmp_path):
    src = tmp_path / "layout.c"
    fields = [f for f, _ in ra.rc_rope_desc._fields_]
    lines = "".join(f'printf("%zu\\n", offsetof(rc_rope_desc, {f}));' for f in fields)
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "radixattn.h"\nint main(void){'
                   f'printf("%zu\\n", sizeof(rc_rope_desc));{lines}printf("%d\\n", RC_KV_FP4);return 0;}}\n')
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    assert got == [C.sizeof(ra.rc_rope_desc)] + [getattr(ra.rc_rope_desc, f).offset for f in fields] + [ra.RC_KV_FP4]


def test_fp4_pool_descriptor():
    d = fp4_pool()
    assert (d.n_slots, d.kv_heads, d.head_dim_k, d.head_dim_v, d.kv_fp8) == (64, 8, 128, 128, ra.RC_KV_FP4)
    assert bf16_pool().kv_fp8 == 0
    k, v, ks, vs = fp4_tensors()
    bad = [dict(k_bscale=ks), dict(v_bscale=vs), dict(k_bscale=ks, v_bscale=vs[:, :, :4]),
           dict(k_bscale=ks, v_bscale=vs.float()), dict(k_bscale=ks, v_bscale=vs, mla=True, head_dim_v=512),
           dict(k_bscale=ks, v_bscale=vs, k_scale=torch.zeros(64, 8), v_scale=torch.zeros(64, 8)),
           dict(k_bscale=ks, v_bscale=torch.zeros(64, 8, 16, dtype=torch.uint8)[..., ::2])]
    for kw in bad:
        with pytest.raises(ValueError):
            ra.make_pool_desc(k, v, **kw)
    with pytest.raises(ValueError):
        ra.make_pool_desc(k, v[:32].contiguous(), k_bscale=ks, v_bscale=vs[:32].contiguous())


def call_rope(pool, rope, n=4, hkv=8, d=128, hq=32, k_off=0, **over):
    """kv_store_rope through the C ABI with host pointers: only its checks may run."""
    buf = torch.zeros(1 << 16, dtype=BF)
    base = (buf.data_ptr() + 255) // 256 * 256
    a = dict(slots=base, positions=base, k=base + k_off, ks=hkv * d, v=base, vs=hkv * d, n=n, q=base, qs=hq * d, hq=hq,
             qo=base, qos=hq * d, table=None, pos=None)
    a.update(over)
    return ra.lib().kv_store_rope(C.byref(pool) if pool is not None else None,
                                  C.byref(rope) if rope is not None else None, a["slots"], a["positions"], a["k"],
                                  a["ks"], a["v"], a["vs"], a["n"], a["q"], a["qs"], a["hq"], a["qo"], a["qos"],
                                  a["table"], a["pos"], None)


def rope_desc(rot=128, offset=0, max_pos=16):
    return ra.make_rope_desc(ra.rope_table(max_pos, rot, device="cpu"), offset=offset)


def test_kv_store_rope_refusals(built):
    A, U = ra.RC_ERR_ARG, ra.RC_ERR_UNSUPPORTED
    r = rope_desc()
    assert call_rope(None, r) == A and call_rope(bf16_pool(), None) == A
    assert call_rope(bf16_pool(), r, n=-1) == A
    assert call_rope(bf16_pool(), r, n=0) == ra.RC_OK
    for missing in ("slots", "positions", "k", "v", "q", "qo"):
        assert call_rope(bf16_pool(), r, **{missing: None}) == A, missing
    assert call_rope(bf16_pool(), r, table=256) == A
    assert call_rope(bf16_pool(), r, k_off=2) == A                # not 16-byte aligned
    assert call_rope(bf16_pool(), r, ks=1028) == A and call_rope(bf16_pool(), r, vs=-8) == A
    assert call_rope(bf16_pool(), r, qs=4100) == A and call_rope(bf16_pool(), r, qos=4088) == A   # rows overlap
    assert call_rope(bf16_pool(), r, hq=0) == A
    for rot, off, want in ((16, 0, U), (48, 0, U), (64, 8, U), (128, 16, A), (160, 0, A), (64, -16, A)):
        assert call_rope(bf16_pool(), rope_desc(rot, off)) == want, (rot, off)
    assert call_rope(bf16_pool(d=96), rope_desc(64), d=96) == U
    fp8 = ra.make_pool_desc(*[torch.zeros(64, 8, 64, dtype=torch.uint8)] * 2, k_scale=torch.zeros(64, 8),
                            v_scale=torch.zeros(64, 8))
    assert call_rope(fp8, rope_desc(64), d=64) == U
    latent = ra.make_pool_desc(torch.zeros(64, 512, dtype=BF), None, mla=True, head_dim_v=448)
    assert call_rope(latent, rope_desc(64, 448), hkv=1, d=512, v=None) == U
    p = fp4_pool()
    p.k_bscale = None
    assert call_rope(p, r) == A
    assert call_rope(fp4_pool(d=256), rope_desc(), d=256) == U


def test_kv_store_rope_binding_checks_shapes(built):
    pool, r = bf16_pool(), rope_desc()
    k = torch.zeros(4, 8, 128, dtype=BF)
    q = torch.zeros(4, 32, 128, dtype=BF)
    slots = torch.arange(4, dtype=torch.int32)
    wide = torch.zeros(4, 48, 128, dtype=BF)
    good = dict(slots=slots, positions=slots, k_new=k, v_new=k, q=q, q_out=torch.zeros_like(q))
    bad = [dict(k_new=k[:3]), dict(k_new=k.float()), dict(k_new=k[:, :4]), dict(v_new=k[..., :64]),
           dict(k_new=k.transpose(1, 2)), dict(q_out=q[:, :16].contiguous()), dict(positions=slots[:3]),
           dict(slots=slots.long()), dict(slots=slots[None]), dict(table=slots.float()), dict(table_pos=slots[:3]),
           dict(positions=slots.repeat_interleave(2)[::2]), dict(q=None), dict(q=q[0], q_out=None), dict(q=q[:, :0], q_out=q[:, :0]), dict(q_out=torch.zeros(1, 32, 128, dtype=BF).expand(4, 32, 128)),
           dict(k_new=torch.zeros(4, 128, 8, dtype=BF).transpose(1, 2))]
    for kw in bad:
        with pytest.raises(ValueError):
            ra.kv_store_rope(pool, r, **{**good, **kw})
    # host tensors in a good layout (here slices of one projection's output) are refused for where they are
    with pytest.raises((ValueError, RuntimeError)):
        ra.kv_store_rope(pool, r, slots, slots, wide[:, 32:40], wide[:, 40:], wide[:, :32], torch.zeros_like(q))
    with pytest.raises(ValueError):
        ra.make_rope_desc(torch.zeros(4, 128, dtype=BF))
    with pytest.raises(ValueError):
        ra.make_rope_desc(torch.zeros(4, 256)[:, ::2])


def call_cross(pool, hq=32, batch=2, max_q=16, max_len=64, ws=None, ws_bytes=0, scale=0.1, **over):
    buf = torch.zeros(1 << 14, dtype=BF)
    base = (buf.data_ptr() + 255) // 256 * 256
    desc = ra.make_attn_desc(pool, hq, scale) if pool is not None else None
    a = dict(q=base, qo=base, out=base, slots=base, start=base, len=base)
    a.update(over)
    kv = ra.rc_kv_table(slots=a["slots"], start=a["start"], len=a["len"], max_len=max_len, table_len=128)
    return ra.lib().attn_cross(C.byref(desc) if desc is not None else None, a["q"], a["qo"], C.byref(kv), batch, max_q,
                               a["out"], None, ws, ws_bytes, None)


def test_attn_cross_refusals(built):
    A, U = ra.RC_ERR_ARG, ra.RC_ERR_UNSUPPORTED
    assert call_cross(None) == A
    assert call_cross(bf16_pool(), batch=-1) == A and call_cross(bf16_pool(), max_q=-1) == A
    assert call_cross(bf16_pool(), max_len=-1) == A
    for scale in (0.0, -0.1, float("nan")):
        assert call_cross(bf16_pool(), scale=scale) == A
    assert call_cross(bf16_pool(), batch=0) == ra.RC_OK and call_cross(bf16_pool(), max_q=0) == ra.RC_OK
    for missing in ("q", "qo", "out", "slots", "start", "len"):
        assert call_cross(bf16_pool(), **{missing: None}) == A, missing
    assert call_cross(bf16_pool(), hq=12) == A and call_cross(bf16_pool(), hq=24) == U
    assert call_cross(bf16_pool(hkv=1), hq=16) == U
    assert call_cross(bf16_pool(d=96)) == U
    latent = ra.make_pool_desc(torch.zeros(64, 576, dtype=BF), None, mla=True, head_dim_v=512)
    assert call_cross(latent) == U
    p = fp4_pool()
    p.v_bscale = None
    assert call_cross(p) == A
    # split keys need their workspace, of the stated size and alignment
    need = ra.attn_cross_workspace(ra.make_attn_desc(bf16_pool(), 32, 0.1), 1, 16, 4096)
    assert need > 0
    assert call_cross(bf16_pool(), batch=1, max_len=4096) == A
    assert call_cross(bf16_pool(), batch=1, max_len=4096, ws=256, ws_bytes=need - 1) == A
    assert call_cross(bf16_pool(), batch=1, max_len=4096, ws=264, ws_bytes=need) == A


def test_attn_cross_workspace(built):
    desc = ra.make_attn_desc(bf16_pool(), 32, 0.1)
    assert ra.attn_cross_workspace(desc, 64, 1024, 4096) == 0          # the grid fills the SMs
    assert ra.attn_cross_workspace(desc, 1, 1, 32) == 0                # nothing to split
    assert ra.attn_cross_workspace(desc, 0, 4, 64) == 0 and ra.attn_cross_workspace(desc, 4, 0, 64) == 0
    small = ra.attn_cross_workspace(desc, 1, 1, 4096)
    assert small >= 2 * 32 * 129 * 4
    n = C.c_size_t(0)
    assert ra.lib().attn_cross_workspace(None, 1, 1, 1, C.byref(n)) == ra.RC_ERR_ARG
    assert ra.lib().attn_cross_workspace(C.byref(desc), 1, -1, 1, C.byref(n)) == ra.RC_ERR_ARG
    assert ra.lib().attn_cross_workspace(C.byref(desc), 1, 1, 1, None) == ra.RC_ERR_ARG


def test_fp4_pool_refused_where_unsupported(built):
    """kv_store, decode (with the appended form) and extend check a 4-bit pool's layout and arrays."""
    L, A, U = ra.lib(), ra.RC_ERR_ARG, ra.RC_ERR_UNSUPPORTED
    buf = torch.zeros(1 << 14, dtype=BF)
    b = (buf.data_ptr() + 255) // 256 * 256

    def decode(pool, k_new=None, q=b, hq=32, out=None, scale=0.1, casc=None):
        d = ra.make_attn_desc(pool, hq, scale)
        kv = ra.rc_kv_table(slots=b, start=b, len=b, max_len=16, table_len=64)
        if k_new:
            return L.attn_decode_append(C.byref(d), q, k_new, k_new, C.byref(kv), 2, None, b, None, b, 1 << 24, None)
        return L.attn_decode(C.byref(d), q, C.byref(kv), 2, casc, out or b, None, b, 1 << 24, None)

    def extend(pool, q=b, hq=32, scale=0.1):
        d = ra.make_attn_desc(pool, hq, scale)
        kv = ra.rc_kv_table(slots=b, start=b, len=b, max_len=16, table_len=64)
        return L.attn_extend(C.byref(d), q, b, C.byref(kv), 2, 8, b, None, None, 0, None)

    store = lambda pool, v=b, k=b: L.kv_store(C.byref(pool), b, k, v, 2, None, None, None)
    no_scale, odd, deep = fp4_pool(), fp4_pool(), fp4_pool(d=256)
    no_scale.k_bscale = None
    odd.v_bscale = odd.v_bscale + 8
    for call in (decode, extend, store):
        assert call(no_scale) == A and call(odd) == A and call(deep) == U, call
    casc = ra.rc_cascade(n_seg=1, total_seg_rows=2, max_seg_rows=2, max_seg_len=8, seg_slots=b, seg_indptr=b,
                         seg_row_indptr=b, seg_rows=b, req_seg_indptr=b, req_seg_pos=b)
    nan = float("nan")
    for scale in (0.0, -0.1, nan):
        assert extend(fp4_pool(), scale=scale) == A and decode(fp4_pool(), scale=scale, casc=C.byref(casc)) == A
    assert decode(fp4_pool(), scale=nan) == A
    empty = fp4_pool()
    empty.n_slots = 0
    assert decode(empty) == A and extend(empty) == A and store(empty) == A
    assert decode(fp4_pool(), k_new=b) == U          # appended keys: kv_store, then attn_decode
    assert decode(fp4_pool(), q=b + 2) == A and extend(fp4_pool(), q=b + 2) == A
    assert decode(fp4_pool(), out=b + 8) == A
    assert decode(fp4_pool(), hq=24) == U
    assert store(fp4_pool(), v=None) == A and store(fp4_pool(), k=b + 8) == A
