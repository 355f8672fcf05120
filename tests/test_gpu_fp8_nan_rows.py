"""An E4M3 row of NaNs (and zeros beside them) reads back as NaN, not as zeros:
kv_store and kv_store_rope, and the attention that reads it."""
from __future__ import annotations

import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra
from tests.test_gpu_operators import BF, Pool, rand

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.mark.parametrize("rope", [False, True])
def test_rows_of_nan_and_zeros(cuda, rope):
    hq, hkv, d, n = 8, 2, 128, 300
    g = torch.Generator().manual_seed(1)
    k, v = rand(g, n, hkv, d), rand(g, n, hkv, d)
    k[40, 0] = NAN                                  # all NaN
    k[50, 1], v[60, 1], v[70, 0] = 0, 0, 0
    k[50, 1, 7], v[60, 1, 9] = -NAN, NAN            # a NaN among zeros
    v[80, 0, 3] = NAN                               # among others: the others keep their codes
    v[90, 1, ::2] = -0.0
    v[90, 1, 1::2] = 0.0
    pool = Pool("fp8", n, hkv, d, cuda, 3)
    slots = torch.arange(n, dtype=torch.int32, device=cuda)
    if rope:
        desc = ra.make_rope_desc(ra.rope_table(4, d, device=cuda))
        ra.kv_store_rope(pool.desc, desc, slots, torch.zeros_like(slots), k, v)
    else:
        ra.kv_store(pool.desc, slots, k, v)
    assert ra.rc_sync(pool.err) == ra.RC_OK
    kd = pool.k.view(torch.float8_e4m3fn).float() * pool.ks[..., None]
    vd = pool.v.view(torch.float8_e4m3fn).float() * pool.vs[..., None]
    if rope:      # at angle 0 a NaN still reaches its pair (NaN * 0)
        want_k = torch.isnan(k)
        want_k |= want_k.roll(d // 2, -1)
    else:
        want_k = torch.isnan(k)
    assert torch.equal(torch.isnan(kd), want_k) and torch.equal(torch.isnan(vd), torch.isnan(v))
    assert int(pool.v[70, 0].max()) == 0 and int(pool.v[90, 1].max()) == 0      # zeros: zero codes, scale 0
    assert float(pool.vs[70, 0]) == 0 and float(pool.vs[90, 1]) == 0
    # who reads them: 4 query heads per KV head, rows of 100 keys
    start = torch.tensor([0, 100, 200], dtype=torch.int32, device=cuda)
    length = torch.tensor([100, 100, 100], dtype=torch.int32, device=cuda)
    desc, kv = ra.make_attn_desc(pool.desc, hq, 0.1), ra.make_kv_table(slots, start, length, 100)
    q = rand(g, 3, hq, d)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=cuda)
    qo = torch.arange(4, dtype=torch.int32, device=cuda)
    for call in ("decode", "extend", "cross"):
        out = torch.zeros(3, hq, d, dtype=BF, device=cuda)
        if call == "decode":
            ra.attn_decode(desc, q, kv, 3, out, None, ws)
        elif call == "extend":
            ra.attn_extend(desc, q, qo, kv, 3, 1, out)
        else:
            ra.attn_cross(desc, q, qo, kv, 3, 1, out, None, ws)
        assert ra.rc_sync(pool.err) == ra.RC_OK
        assert bool(torch.isnan(out[0]).all()) and bool(torch.isfinite(out[1:]).all()), call   # K rows 40 and 50
    k[40, 0], k[50, 1] = 1, 1
    ra.kv_store(pool.desc, slots, k, v)
    for call in ("decode", "cross"):
        out = torch.zeros(3, hq, d, dtype=BF, device=cuda)
        if call == "decode":
            ra.attn_decode(desc, q, kv, 3, out, None, ws)
        else:
            ra.attn_cross(desc, q, qo, kv, 3, 1, out, None, ws)
        assert ra.rc_sync(pool.err) == ra.RC_OK
        nan = torch.isnan(out)
        want = torch.zeros_like(nan)
        want[0, 4:, 9], want[0, :4, 3] = True, True          # the values' own columns
        assert torch.equal(nan, want), call
