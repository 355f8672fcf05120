"""Calls with a workspace sized once, for the largest max_len, as a decode loop
has it: each gives the bits of a call with a workspace of its own."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra
from tests.test_gpu_operators import BF, Pool, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,B,first,last", [("bf16", 64, 250, 262), ("fp8", 64, 250, 262), ("bf16", 40, 380, 388),
                                              ("fp4", 64, 90, 100), ("latent", 64, 1214, 1218)])
def test_decode_steps(cuda, fmt, B, first, last):
    hq, hkv, d = (128, 1, 576) if fmt == "latent" else (32, 8, 128)
    n_slots = B * last
    g = torch.Generator().manual_seed(1)
    if fmt == "latent":
        err = torch.zeros(1, dtype=torch.int32, device=cuda)
        pool = ra.make_pool_desc(torch.randn(n_slots, d, generator=g).to(BF).to(cuda), None, err, mla=True, head_dim_v=512)
    else:
        p = Pool(fmt, n_slots, hkv, d, cuda, 2)
        pool, err = p.desc, p.err
    desc = ra.make_attn_desc(pool, hq, 1.0 / np.sqrt(d))
    table = torch.arange(n_slots, dtype=torch.int32, device=cuda)
    start = torch.arange(B, dtype=torch.int32, device=cuda) * last
    q = rand(g, B, hq, d)
    dv = 512 if fmt == "latent" else d
    lens = {m: torch.tensor([max(1, m - 3 * (i % 9)) for i in range(B)], dtype=torch.int32, device=cuda)
            for m in range(first, last + 1)}
    own = {}
    for m in lens:
        kv = ra.make_kv_table(table, start, lens[m], m)
        ws = torch.full((ra.attn_decode_workspace(desc, B, m),), 0xFF, dtype=torch.uint8, device=cuda)
        own[m] = torch.zeros(B, hq, dv, dtype=BF, device=cuda)
        ra.attn_decode(desc, q, kv, B, own[m], None, ws)
    ws = torch.full((ra.attn_decode_workspace(desc, B, last),), 0xFF, dtype=torch.uint8, device=cuda)
    outs = {m: torch.zeros_like(own[m]) for m in lens}
    ra.attn_decode_steps(desc, ra.make_kv_table(table, start, lens[first], first), B,
                         [dict(q=q, out=outs[m], len=lens[m], max_len=m) for m in lens], ws)
    assert ra.rc_sync(err) == ra.RC_OK
    assert all(torch.equal(outs[m], own[m]) for m in lens)


@pytest.mark.parametrize("fmt,max_q", [("bf16", 1), ("bf16", 40), ("fp8", 16), ("fp4", 1), ("fp4", 40)])
def test_cross(cuda, fmt, max_q):
    hq, hkv, d, B = 32, 8, 128, 3
    pool = Pool(fmt, 2000, hkv, d, cuda, 2)
    desc = ra.make_attn_desc(pool.desc, hq, 0.09)
    table = torch.arange(2000, dtype=torch.int32, device=cuda)
    to = lambda *a: torch.tensor(a, dtype=torch.int32, device=cuda)
    q = rand(torch.Generator().manual_seed(1), B * max_q, hq, d)
    qo = to(*[i * max_q for i in range(B + 1)])
    ws = torch.full((ra.attn_cross_workspace(desc, B, max_q, 1500),), 0xFF, dtype=torch.uint8, device=cuda)
    for m in (1500, 1025, 641, 640, 300, 129, 64, 1):
        kv = ra.make_kv_table(table, to(0, 100, 400), to(m, max(1, m - 70), m // 2), m)
        a, b = torch.zeros_like(q), torch.zeros_like(q)
        ra.attn_cross(desc, q, qo, kv, B, max_q, a, None, ws)
        own = torch.full((max(256, ra.attn_cross_workspace(desc, B, max_q, m)),), 0xFF, dtype=torch.uint8, device=cuda)
        ra.attn_cross(desc, q, qo, kv, B, max_q, b, None, own)
        assert ra.rc_sync(pool.err) == ra.RC_OK and torch.equal(a, b)
