"""Slot ids outside the pool, alone, through every attention call and pool
format: the call is flagged and the key reads as zeros; ids behind a row's end
are not looked at."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra
from oracle import fp4_oracle as f4
from tests.test_gpu_operators import BF, Pool, check, f32, rand

pytestmark = pytest.mark.gpu

HQ, HKV, D, N_SLOTS = 8, 2, 128, 1300
LENS = [130, 1000, 70]
START = [0, 200, 1210]           # room to grow behind every row: entries that nobody may read


def run_call(call, cuda, pool, flat, qo, q, max_len=1000):
    """One call over the three rows of `flat`; (status, out, lse)."""
    to = lambda *a: torch.tensor(a, dtype=torch.int32, device=cuda)
    desc = ra.make_attn_desc(pool.desc, HQ, 0.1)
    kv = ra.make_kv_table(flat, to(*START), to(*LENS), max_len)
    out, lse = torch.zeros_like(q), torch.zeros(len(q), HQ, dtype=torch.float32, device=cuda)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=cuda)
    max_q = len(q) // 3
    if call == "decode":
        ra.attn_decode(desc, q, kv, 3, out, lse, ws)
    elif call == "cascade":      # the middle row's first 800 keys as a segment of its own
        seg = flat[200:1000].contiguous()
        casc = ra.make_cascade(seg, to(0, 800), to(0, 1), to(1), to(0, 0, 1, 1), to(0), max_seg_rows=1, max_seg_len=800)
        kv = ra.make_kv_table(flat, to(0, 1000, 1210), to(130, 200, 70), 200)
        ra.attn_decode(desc, q, kv, 3, out, lse, ws, cascade=casc)
    elif call == "extend":
        ra.attn_extend(desc, q, qo, kv, 3, max_q, out, lse)
    elif call == "extend split":
        ra.attn_extend(desc, q, qo, kv, 3, max_q, out, lse, ws)
    else:
        ra.attn_cross(desc, q, qo, kv, 3, max_q, out, lse, ws)
    return ra.rc_sync(pool.err), out, lse


CALLS = [("decode", 1), ("cascade", 1), ("extend", 8), ("extend split", 8), ("extend", 60), ("cross", 1), ("cross", 40)]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("call,nq", CALLS)
def test_one_bad_slot_is_flagged_and_reads_as_zeros(cuda, call, nq, fmt):
    pool = Pool(fmt, N_SLOTS, HKV, D, cuda, 31)
    g = torch.Generator().manual_seed(3)
    flat = torch.full((1300,), -1, dtype=torch.int32)
    perm = torch.randperm(N_SLOTS, generator=g).to(torch.int32)
    for s, n in zip(START, LENS):
        flat[s:s + n] = perm[s:s + n]
    flat = flat.to(cuda)
    q = rand(g, 3 * nq, HQ, D)
    qo = torch.arange(4, dtype=torch.int32, device=cuda) * nq
    status, want, _ = run_call(call, cuda, pool, flat, qo, q)
    assert status == ra.RC_OK                     # the -1 entries lie behind the rows' ends
    k, v = pool.values()
    k, v = np.concatenate([k, np.zeros_like(k[:1])]), np.concatenate([v, np.zeros_like(v[:1])])
    # in the middle row: its first keys, one for each of three groups of eight; keys of later tiles and chunks; the last
    for at in (0, 9, 17, 70, 333, 700, 999):
        if call in ("extend", "extend split") and at == 999:
            at = 999 - nq                          # a key that all of the row's tokens see
        for bad in (-1, N_SLOTS):
            rows = flat.clone()
            rows[200 + at] = bad
            status, out, lse = run_call(call, cuda, pool, rows, qo, q)
            assert status == ra.RC_ERR_DEVICE, (at, bad)
            assert torch.equal(out[:nq], want[:nq]) and torch.equal(out[2 * nq:], want[2 * nq:])
        if at in (9, 700):
            ids = rows[200:1200].cpu().numpy().astype(np.int64)     # the slot behind the pool holds zeros
            lim = [1000 - nq + i + 1 for i in range(nq)] if call.startswith("extend") else None
            ref = f4.attention(f32(q[nq:2 * nq]).astype(np.float64), k, v, [ids] * nq, HQ, HKV, float(np.float32(0.1)), lim)
            check(out[nq:2 * nq], lse[nq:2 * nq], ref, pool.u_p, label=f"{call} {fmt} key {at}")
