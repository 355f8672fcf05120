"""DeviceEngine hands attn_extend the workspace with which a 4-bit pool's small
batches over long prefixes are split over the SMs."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra
from radixattention_prefix_shared_tree_gb300.driver import DeviceEngine
from tests.test_gpu_operators import BF, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("prefix,new", [(4000, 8), (100, 8), (4000, 900)])
def test_extend_as_the_library_plans_it(cuda, fmt, prefix, new):
    sh = SimpleNamespace(q_heads=32, kv_heads=8, head_dim_k=128, head_dim_v=128, mla=False, scale=0.09)
    n, B = prefix + new, 2
    eng = DeviceEngine(sh, 2 * n, device=cuda, kv_fp8=fmt == "fp8", kv_fp4=fmt == "fp4")
    g = torch.Generator().manual_seed(3)
    slots = torch.arange(2 * n, dtype=torch.int32, device=cuda)
    eng.store(slots, rand(g, 2 * n, 8, 128), rand(g, 2 * n, 8, 128))
    q = rand(g, B * new, 32, 128)
    to = lambda *a: torch.tensor(a, dtype=torch.int32, device=cuda)
    lay = SimpleNamespace(extend_table=ra.make_kv_table(slots, to(0, n), to(n, n), n), qo_indptr=to(0, new, 2 * new),
                          batch_size=B, max_q=new)
    out, lse = torch.empty_like(q), torch.empty(B * new, 32, device=cuda)
    before = eng.launches
    eng.extend(lay, q, out, lse)
    size = ra.attn_extend_workspace(eng.desc, B, new, n)
    assert (size > 0) == (fmt == "fp4" and prefix == 4000 and new == 8)
    want, want_lse = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(size, dtype=torch.uint8, device=cuda) if size else None
    ra.attn_extend(eng.desc, q, lay.qo_indptr, lay.extend_table, B, new, want, want_lse, ws)
    assert ra.rc_sync(eng.err) == ra.RC_OK
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert eng.launches - before == (2 if size else 1)
