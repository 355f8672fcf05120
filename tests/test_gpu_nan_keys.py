"""A NaN key makes the outputs that read it NaN with an lse of +infinity, in
every form of attention and every pool format; other rows and heads stay as
they were, bit for bit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra
from tests.test_gpu_operators import BF, Pool, rand

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _poison(pool, slot, head):
    if pool.fmt == "bf16":
        pool.k[slot, head, 5] = NAN
    elif pool.fmt == "fp8":
        pool.ks[slot, head] = NAN
    else:
        pool.ks[slot, head, 3] = 255


def _expect(before, after, hit):
    (out0, lse0), (out, lse) = before, after
    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isposinf(lse[hit]).all())
    assert torch.equal(out[~hit], out0[~hit]) and torch.equal(lse[~hit], lse0[~hit])


@pytest.mark.parametrize("fmt,append", [("bf16", False), ("bf16", True), ("fp8", False), ("fp4", False)])
@pytest.mark.parametrize("lens", [[1500, 1400, 700], [60, 50, 33], [200 + (i * 37) % 100 for i in range(700)]])
def test_decode(cuda, fmt, lens, append):
    """Rows in several chunks, in one, and enough rows for a warp each; the appended form (bf16 pools) too."""
    hq, hkv, d, B = 8, 2, 128, len(lens)
    n_slots = sum(lens)
    pool = Pool(fmt, n_slots, hkv, d, cuda, 11)
    table = torch.arange(n_slots, dtype=torch.int32, device=cuda)      # no slot in two rows
    start = torch.tensor(np.concatenate([[0], np.cumsum(lens)[:-1]]), dtype=torch.int32, device=cuda)
    length = torch.tensor(lens, dtype=torch.int32, device=cuda)
    g = torch.Generator().manual_seed(2)
    q = rand(g, B, hq, d)
    new = [rand(g, B, hkv, d) for _ in range(2)]
    desc = ra.make_attn_desc(pool.desc, hq, 0.1)
    kv = ra.make_kv_table(table, start, length, max(lens))
    ws = torch.empty(ra.attn_decode_workspace(desc, B, max(lens)), dtype=torch.uint8, device=cuda)

    def run():
        out, lse = torch.zeros_like(q), torch.zeros(B, hq, dtype=torch.float32, device=cuda)
        if append:
            ra.attn_decode_append(desc, q, *new, kv, B, out, lse, ws)
        else:
            ra.attn_decode(desc, q, kv, B, out, lse, ws)
        assert ra.rc_sync(pool.err) == ra.RC_OK
        return out, lse

    clean = run()
    _poison(pool, int(start[1]) + 7, 1)
    hit = torch.zeros(B, hq, dtype=torch.bool, device=cuda)
    hit[1, 4:] = True
    _expect(clean, run(), hit)
    if append:      # the new key itself
        new[0][0, 0, 9] = NAN
        hit[0, :4] = True
        _expect(clean, run(), hit)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("B", [6, 700])
@pytest.mark.parametrize("where", ["segment", "row"])
def test_decode_with_a_cascade(cuda, fmt, B, where):
    """The NaN in a shared segment (all rows below it) or in one row's own part; rows 3.. are under the segment."""
    hq, hkv, d, shared, own = 8, 2, 128, 700, 90
    pool = Pool(fmt, shared + own * B, hkv, d, cuda, 5)
    to = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=cuda)
    seg = to(range(shared))
    table = to(range(shared, shared + own * B))
    q = rand(torch.Generator().manual_seed(2), B, hq, d)
    under = list(range(3, B))
    indptr = [0] * 4 + list(range(1, B - 2))
    casc = ra.make_cascade(seg, to([0, shared]), to([0, len(under)]), to(under), to(indptr), to(range(len(under))),
                           max_seg_rows=len(under), max_seg_len=shared)
    desc = ra.make_attn_desc(pool.desc, hq, 0.1)
    kv = ra.make_kv_table(table, to(np.arange(B) * own), to([own] * B), own)
    ws = torch.empty(ra.attn_decode_workspace(desc, B, own, casc), dtype=torch.uint8, device=cuda)

    def run():
        out, lse = torch.zeros_like(q), torch.zeros(B, hq, dtype=torch.float32, device=cuda)
        ra.attn_decode(desc, q, kv, B, out, lse, ws, cascade=casc)
        assert ra.rc_sync(pool.err) == ra.RC_OK
        return out, lse

    clean = run()
    hit = torch.zeros(B, hq, dtype=torch.bool, device=cuda)
    if where == "segment":
        _poison(pool, 400, 0)
        hit[3:, :4] = True
    else:
        _poison(pool, shared + own * 4 + 70, 0)
        hit[4, :4] = True
    _expect(clean, run(), hit)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("nq", [5, 300])
def test_extend(cuda, fmt, nq):
    """The tokens that see the key; those before it do not."""
    hq, hkv, d, lens = 8, 2, 128, [900, 700, 400]
    pool = Pool(fmt, sum(lens), hkv, d, cuda, 11)
    to = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=cuda)
    start = np.concatenate([[0], np.cumsum(lens)[:-1]])
    kv = ra.make_kv_table(to(range(sum(lens))), to(start), to(lens), 900)
    q = rand(torch.Generator().manual_seed(2), 3 * nq, hq, d)
    qo = to(np.arange(4) * nq)
    desc = ra.make_attn_desc(pool.desc, hq, 0.1)

    def run():
        out, lse = torch.zeros_like(q), torch.zeros(3 * nq, hq, dtype=torch.float32, device=cuda)
        ra.attn_extend(desc, q, qo, kv, 3, nq, out, lse)
        assert ra.rc_sync(pool.err) == ra.RC_OK
        return out, lse

    clean = run()
    _poison(pool, 900 + 300, 1)                       # row 1: a key of its prefix
    _poison(pool, 1600 + 400 - nq + 2, 0)             # row 2: its third new token
    hit = torch.zeros(3 * nq, hq, dtype=torch.bool, device=cuda)
    hit[nq:2 * nq, 4:] = True
    hit[2 * nq + 2:, :4] = True
    _expect(clean, run(), hit)


@pytest.mark.parametrize("hq", [128, 16])
@pytest.mark.parametrize("lens", [[3000, 2500, 64], [100, 90, 33]])
def test_decode_latent(cuda, hq, lens):
    """Both latent kernels, rows in several chunks and in one: every head reads the key."""
    n_slots, B = sum(lens), len(lens)
    g = torch.Generator().manual_seed(4)
    pool_t = torch.randn(n_slots, 576, generator=g).to(BF).to(cuda)
    err = torch.zeros(1, dtype=torch.int32, device=cuda)
    desc = ra.make_attn_desc(ra.make_pool_desc(pool_t, None, err, mla=True, head_dim_v=512), hq, 1.0 / 24.0)
    to = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=cuda)
    start = np.concatenate([[0], np.cumsum(lens)[:-1]])
    kv = ra.make_kv_table(to(range(n_slots)), to(start), to(lens), max(lens))
    q = rand(g, B, hq, 576)
    ws = torch.empty(ra.attn_decode_workspace(desc, B, max(lens)), dtype=torch.uint8, device=cuda)

    def run():
        out = torch.zeros(B, hq, 512, dtype=BF, device=cuda)
        lse = torch.zeros(B, hq, dtype=torch.float32, device=cuda)
        ra.attn_decode(desc, q, kv, B, out, lse, ws)
        assert ra.rc_sync(err) == ra.RC_OK
        return out, lse

    clean = run()
    pool_t[int(start[1]) + 40, 570] = NAN             # a rotary column: in the scores only
    hit = torch.zeros(B, hq, dtype=torch.bool, device=cuda)
    hit[1] = True
    _expect(clean, run(), hit)
