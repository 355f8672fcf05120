"""kv_store_rope and attn_cross refuse a descriptor, table or tensor that is not
on the current device, before anything is launched."""
from __future__ import annotations

import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra
from tests.test_gpu_operators import BF, Pool, rand

pytestmark = pytest.mark.gpu


def host_pool(fmt):
    k = torch.zeros(64, 8, 128, dtype=BF)
    if fmt == "bf16":
        return ra.make_pool_desc(k, k.clone())
    c, s = torch.zeros(64, 8, 64, dtype=torch.uint8), torch.zeros(64, 8, 8, dtype=torch.uint8)
    return ra.make_pool_desc(c, c.clone(), k_bscale=s, v_bscale=s.clone())


def test_kv_store_rope(cuda):
    pool = Pool("bf16", 64, 8, 128, cuda, 1)
    here = ra.make_rope_desc(ra.rope_table(16, 128, device=cuda))
    k = rand(torch.Generator().manual_seed(1), 4, 8, 128)
    ids = torch.arange(4, dtype=torch.int32, device=cuda)
    mixed = ra.make_pool_desc(pool.k, pool.v.cpu())
    before = pool.k.clone()
    for p, r, slots in ((pool.desc, ra.make_rope_desc(ra.rope_table(16, 128, device="cpu")), ids),
                        (host_pool("bf16"), here, ids), (host_pool("fp4"), here, ids), (mixed, here, ids),
                        (pool.desc, here, ids.cpu())):
        with pytest.raises(ValueError, match="device"):
            ra.kv_store_rope(p, r, slots, ids, k, k)
    torch.cuda.synchronize()
    assert torch.equal(pool.k, before)
    ra.kv_store_rope(pool.desc, here, ids, ids, k, k)
    assert ra.rc_sync(pool.err) == ra.RC_OK


def test_attn_cross(cuda):
    pool = Pool("bf16", 64, 8, 128, cuda, 1)
    ids = torch.arange(64, dtype=torch.int32, device=cuda)
    to = lambda *a: torch.tensor(a, dtype=torch.int32, device=cuda)
    q = rand(torch.Generator().manual_seed(1), 2, 8, 128)
    desc, qo = ra.make_attn_desc(pool.desc, 8, 0.1), to(0, 1, 2)
    kv = ra.make_kv_table(ids, to(0, 32), to(20, 10), 20)
    out = torch.full_like(q, 3.0)
    for d, t, x in ((ra.make_attn_desc(host_pool("bf16"), 8, 0.1), kv, q), (ra.make_attn_desc(host_pool("fp4"), 8, 0.1), kv, q),
                    (desc, ra.make_kv_table(ids.cpu(), to(0, 32), to(20, 10), 20), q),
                    (desc, ra.make_kv_table(ids, to(0, 32).cpu(), to(20, 10), 20), q),
                    (desc, ra.make_kv_table(ids, to(0, 32), to(20, 10).cpu(), 20), q), (desc, kv, q.cpu())):
        with pytest.raises(ValueError, match="device"):
            ra.attn_cross(d, x, qo, t, 2, 1, out)
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())
    ra.attn_cross(desc, q, qo, kv, 2, 1, out)
    assert ra.rc_sync(pool.err) == ra.RC_OK
