"""Calls large enough for the forms of kv_load and of the appends that take several units or passes a thread.

Which form a call takes depends on its size and on the GPU's SMs, so sizes are
derived from both, on either side of each border.  Bars: bit for bit, against the
oracle's definition (kv_load) and against the same tokens appended a few at a time
(by the form for few tokens, which the other tests compare with the oracle).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra
from oracle import fp4_oracle as f4
from tests.test_gpu_pool_rows import BF, LOADS, bits, f32, held, make_pool

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("fmt,hkv,d", LOADS)
@pytest.mark.parametrize("extra", [0, 8, 16])
def test_kv_load_two_units_a_thread(cuda, fmt, hkv, d, extra):
    """Up to sms x 2,048 units of 16 values a thread takes one, beyond two."""
    g = torch.Generator(device=cuda).manual_seed(d + extra)
    n_slots, row, sides = 700, hkv * d, 1 if fmt == "latent" else 2
    pool, arrays, err = make_pool(fmt, n_slots, hkv, d, cuda)
    spread = torch.exp(3 * torch.randn(n_slots, hkv, 1, generator=g, device=cuda))
    k, v = ((torch.randn(n_slots, hkv, d, generator=g, device=cuda) * spread).to(BF) for _ in range(2))
    ra.kv_store(pool, torch.arange(n_slots, dtype=torch.int32, device=cuda), k, None if fmt == "latent" else v)
    want = [torch.from_numpy(x.reshape(n_slots, row).view(np.int16)).to(cuda) for x in held(fmt, arrays)]
    one = sms() * 2048 * 16 // (sides * row)       # the most tokens at one unit a thread
    for n, only in ((one, None), (one + 1, None), (one + 37, None), (sides * one + 1, 0), (sides * one + 5, sides - 1)):
        slots = torch.randint(0, n_slots, (n,), generator=g, device=cuda).to(torch.int32)
        out = [torch.full((n, row + extra), 7.0, dtype=BF, device=cuda) for _ in range(sides)]
        got = [x[:, :row].unflatten(1, (hkv, d)) if only in (None, i) else None for i, x in enumerate(out)]
        ra.kv_load(pool, slots, got[0], got[1] if sides == 2 else None)
        assert ra.rc_sync(err) == ra.RC_OK
        for x, y, ref in zip(out, got, want):
            if y is None:
                assert bool((x == 7).all())
            else:
                assert torch.equal(x[:, :row].view(torch.int16), ref[slots.long()]) and bool((x[:, row:] == 7).all())


def test_kv_load_two_units_a_thread_bad_slots(cuda):
    """Slots outside the pool among many: zeros and the error flag."""
    pool, arrays, err = make_pool("fp8", 50, 2, 128, cuda)
    k = torch.randn(50, 2, 128, device=cuda).to(BF)
    ra.kv_store(pool, torch.arange(50, dtype=torch.int32, device=cuda), k, k)
    n = sms() * 2048 // 32 + 11
    slots = (torch.arange(n, device=cuda) % 50).to(torch.int32)
    bad = torch.tensor([0, 31, n // 2, n - 2, n - 1], device=cuda)
    slots[bad] = torch.tensor([-1, 50, 2 ** 31 - 1, -2 ** 31, 51], dtype=torch.int32, device=cuda)
    ko, vo = (torch.full((n, 2, 128), 7.0, dtype=BF, device=cuda) for _ in range(2))
    ra.kv_load(pool, slots, ko, vo)
    assert ra.rc_sync(err) == ra.RC_ERR_DEVICE
    want = torch.from_numpy(held("fp8", arrays)[0].view(np.int16)).to(cuda)
    good = torch.ones(n, dtype=torch.bool, device=cuda)
    good[bad] = False
    assert bool((ko[bad] == 0).all()) and bool((vo[bad] == 0).all())
    assert torch.equal(ko[good].view(torch.int16), want[slots[good].long()])


APPENDS = [  # format, Hq, Hkv, d, rotated (0: stored as it is), offset, interleaved, axes' pairs
    ("bf16", 32, 8, 128, 128, 0, False, None), ("bf16", 32, 8, 128, 128, 0, True, [24, 20, 20]),
    ("fp8", 32, 8, 128, 64, 32, True, None), ("fp8", 32, 8, 128, 128, 0, False, [16, 24, 24]),
    ("fp4", 32, 8, 128, 128, 0, False, None), ("fp4", 32, 8, 128, 128, 0, True, [40, 24]),
    ("bf16", 64, 8, 128, 128, 0, False, None), ("fp8", 64, 8, 128, 128, 0, False, None), ("fp4", 64, 8, 128, 128, 0, True, None),
    ("bf16", 16, 8, 64, 64, 0, False, None), ("bf16", 32, 8, 64, 32, 16, True, None), ("fp4", 16, 8, 64, 64, 0, False, None),
    ("bf16", 7, 3, 64, 64, 0, False, None), ("fp4", 0, 8, 128, 0, 0, False, None), ("fp4", 0, 4, 64, 0, 0, False, None),
    ("fp4", 0, 32, 128, 0, 0, False, None),
    ("latent", 16, 1, 576, 64, 512, False, None), ("latent", 16, 1, 576, 64, 512, True, [12, 10, 10]),
    ("latent", 128, 1, 576, 64, 512, True, None), ("latent", 128, 1, 576, 576, 0, False, [100, 88, 50, 50]),
]


@pytest.mark.parametrize("fmt,hq,hkv,d,rot,off,inter,sections", APPENDS)
def test_appends_of_many_tokens(cuda, fmt, hq, hkv, d, rot, off, inter, sections):
    """Above 64 passes (32 units of 16 values) an SM a warp takes several passes of its token: how many depends on
    how many warps the GPU holds (16 to 24 an SM), so sizes lie around whole waves of 4, 6 and 12 passes a warp."""
    rows = hq + (1 if fmt == "latent" else 2 * hkv)
    passes = (rows * d // 16 + 31) // 32
    few = 64 * sms() // passes                  # the most tokens at a pass a warp
    sizes = {few, few + 1, few + few // 3}
    for a_warp in (4, 6, 12):
        for warps in (16, 20, 24):
            for waves in (1, 2):
                n = waves * warps * sms() // -(-passes // a_warp)
                sizes |= {n, n + 1}
    sizes = sorted(n for n in sizes if few <= n <= 4 * few)
    most = sizes[-1]
    g = torch.Generator(device=cuda).manual_seed(rows + d)
    k, v = (torch.randn(most, hkv, d, generator=g, device=cuda).to(BF) for _ in range(2))
    q = torch.randn(most, hq, d, generator=g, device=cuda).to(BF) if hq else None
    axis = ra.rope_axes(sections, True) if sections else None
    table = ra.rope_table(400, rot, device=cuda) if rot else None
    rope = ra.make_rope_desc(table, inter, off, pair_axis=axis) if rot else None
    pos = torch.randint(0, 400, (len(sections) if sections else 1, most), generator=g, device=cuda).to(torch.int32)
    n_slots = most + 9
    perm = torch.randperm(n_slots, generator=g, device=cuda).to(torch.int32)

    def append(pool, a, b, q_out):
        if rope is None:
            return ra.kv_store(pool, perm[a:b], k[a:b], v[a:b])
        p = pos[:, a:b].contiguous() if sections else pos[0, a:b]
        ra.kv_store_rope(pool, rope, perm[a:b], p, k[a:b], None if fmt == "latent" else v[a:b], q[a:b], q_out[a:b])

    want_pool, want, err = make_pool(fmt, n_slots, hkv, d, cuda, fill=3)
    want_q = torch.zeros_like(q) if hq else None
    for a in range(0, most, few):
        append(want_pool, a, min(a + few, most), want_q)
    assert ra.rc_sync(err) == ra.RC_OK
    if rot:     # some of those tokens against the oracle's rotation
        some = torch.randint(0, most, (50,), generator=g, device=cuda)
        at = pos.long()[torch.tensor(axis, device=cuda)].t()[some] if sections else pos[0].long()[some][:, None]
        cols = torch.arange(rot // 2, device=cuda)
        own = torch.cat([table[at, cols], table[at, cols + rot // 2]], 1).cpu().numpy()
        assert np.array_equal(bits(want_q[some]), f4.bf16_round(f4.rotate(f32(q[some]), own, np.arange(50), off, inter)))
    for n in sizes:
        pool, arrays, err = make_pool(fmt, n_slots, hkv, d, cuda, fill=3)
        q_out = torch.zeros_like(q) if hq else None
        append(pool, 0, n, q_out)
        assert ra.rc_sync(err) == ra.RC_OK
        at, rest = perm[:n].long(), perm[n:].long()
        for x, y in zip(arrays, want):
            assert torch.equal(x[at], y[at]) and bool((x[rest] == 3).all()), n
        if hq:
            assert torch.equal(q_out[:n], want_q[:n]) and not bool(q_out[n:].any()), n
