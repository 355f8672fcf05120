"""The 128-head latent kernel around its ring of four 32-key stages: every
count of tiles from one to beyond two laps, each stage's last use followed at
once by another CTA on the same SM; whole rows and rows in chunks."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import radixattention_prefix_shared_tree_gb300 as ra
from tests import tolerance as tol
from tests.test_gpu_operators import BF, bits, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_len,batch", [(256, 400), (2600, 300)])
def test_every_tile_count(cuda, max_len, batch):
    """Rows of 1..9 tiles (also one key short of them), whole in the first batch, cut into chunks in the second;
    several CTAs one after another on every SM.  The same bits twice."""
    hq, n_slots = 128, 3000
    lens = [min(max_len, max(1, 32 * (1 + i % 9) - (i // 9) % 2)) for i in range(batch)]
    lens[-1] = max_len
    g = torch.Generator().manual_seed(batch)
    pool = torch.randn(n_slots, 576, generator=g).to(BF).to(cuda)
    err = torch.zeros(1, dtype=torch.int32, device=cuda)
    scale = 1.0 / 24.0
    desc = ra.make_attn_desc(ra.make_pool_desc(pool, None, err, mla=True, head_dim_v=512), hq, scale)
    rng = np.random.default_rng(batch)
    rows = [rng.choice(n_slots, size=n, replace=False).astype(np.int32) for n in lens]
    to = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=cuda)
    kv = ra.make_kv_table(to(np.concatenate(rows)), to(np.concatenate([[0], np.cumsum(lens)[:-1]])), to(lens), max_len)
    q = rand(g, batch, hq, 576)
    ws = torch.empty(ra.attn_decode_workspace(desc, batch, max_len), dtype=torch.uint8, device=cuda)
    outs = []
    for _ in range(2):
        out = torch.zeros(batch, hq, 512, dtype=BF, device=cuda)
        lse = torch.zeros(batch, hq, dtype=torch.float32, device=cuda)
        ra.attn_decode(desc, q, kv, batch, out, lse, ws)
        assert ra.rc_sync(err) == ra.RC_OK
        outs.append((out, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    pick = list(range(18)) + [batch - 1]
    kb, qb = bits(pool).reshape(n_slots, -1), bits(q)
    for b in pick:
        k = np.ascontiguousarray(kb[rows[b]])
        v = np.ascontiguousarray(k[:, :512])
        n = np.full(1, lens[b], np.int64)
        args = (np.ascontiguousarray(qb[b:b + 1]).reshape(1, -1), k, v, np.zeros(1, np.int64), n, hq, 1, 576, 512, scale)
        ref, ref_lse = oracle.attention(*args)
        a_abs, _ = oracle.attention(args[0], k, tol.abs_bits(v), *args[3:])
        got = outs[0][0][b].float().cpu().numpy().reshape(ref.shape)
        tol.check_values(got, ref, a_abs, label=f"{lens[b]} keys")
        tol.check_lse(outs[0][1][b].cpu().numpy().reshape(ref_lse.shape), ref_lse)
