"""kv_store_rope, the 4-bit pool and attn_cross on the GPU against their oracle.

Bars.  Stored rows and rotated queries: bit for bit against the fp32 definition
(every operation rounded once), and against the 64-bit formula within half a
bf16 step plus the fp32 operations' 2^-24 each.  Attention: tests/tolerance.py
with P rounded to f16 for the 4-bit and E4M3 pools, to bf16 for bf16 pools; the
4-bit pool's values are exact in f16, so its error is P's and the output's
rounding like the others'.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra
from oracle import fp4_oracle as f4
from oracle import fp8_oracle as f8
from synth import hashgen as hg
from tests import tolerance as tol

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def f32(t):
    return t.float().cpu().numpy()


def rand(gen, *shape, dev="cuda"):
    return torch.randn(*shape, generator=gen, dtype=torch.float32).to(BF).to(dev)


class Pool:
    """A pool of the given format, every slot filled by kv_store (or by hand in bf16), and its values."""

    def __init__(self, fmt, n_slots, hkv, d, dev, seed, gain=1.0):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.err = fmt, torch.zeros(1, dtype=torch.int32, device=dev)
        k, v = (torch.randn(n_slots, hkv, d, generator=g) * gain).to(BF).to(dev), rand(g, n_slots, hkv, d, dev=dev)
        self.src_k, self.src_v = k, v
        if fmt == "bf16":
            self.k, self.v = k, v
            self.desc = ra.make_pool_desc(k, v, self.err)
            return
        w = d // 2 if fmt == "fp4" else d
        self.k, self.v = (torch.zeros(n_slots, hkv, w, dtype=torch.uint8, device=dev) for _ in range(2))
        if fmt == "fp4":
            self.ks, self.vs = (torch.zeros(n_slots, hkv, d // 16, dtype=torch.uint8, device=dev) for _ in range(2))
            self.desc = ra.make_pool_desc(self.k, self.v, self.err, k_bscale=self.ks, v_bscale=self.vs)
        else:
            self.ks, self.vs = (torch.zeros(n_slots, hkv, dtype=torch.float32, device=dev) for _ in range(2))
            self.desc = ra.make_pool_desc(self.k, self.v, self.err, k_scale=self.ks, v_scale=self.vs)
        ra.kv_store(self.desc, torch.arange(n_slots, dtype=torch.int32, device=dev), k, v)
        assert ra.rc_sync(self.err) == ra.RC_OK

    def values(self):
        if self.fmt == "bf16":
            return f32(self.k).astype(np.float64), f32(self.v).astype(np.float64)
        de = f4.dequantize if self.fmt == "fp4" else f8.dequantize
        return tuple(de(c.cpu().numpy(), s.cpu().numpy()) for c, s in ((self.k, self.ks), (self.v, self.vs)))

    @property
    def u_p(self):
        return tol.U_BF16 if self.fmt == "bf16" else tol.U_F16


def check(out, lse, ref, u_p, label="out"):
    o, l, a = ref
    tol.check_values(hg.bf16_bits_to_f32(bits(out)), o, a, u_p=u_p, label=label)
    if lse is not None:
        got = lse.cpu().numpy()
        empty = np.isneginf(l)
        assert np.array_equal(np.isneginf(got), empty)
        tol.check_lse(got[~empty], l[~empty])


def tables(lens, n_slots, seed, dev, shared=0):
    rng = np.random.default_rng(seed)
    perm = rng.permutation(n_slots)
    rows, at = [], shared
    for n in lens:
        own = rng.choice(n_slots, size=max(n - shared, 0), replace=False)
        rows.append(np.concatenate([perm[:min(shared, n)], own]).astype(np.int32))
    starts = np.concatenate([[0], np.cumsum([len(r) for r in rows])[:-1]]).astype(np.int32)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)
    flat = np.concatenate(rows) if sum(lens) else np.zeros(1, np.int32)
    return rows, to(flat), to(starts), to(lens)


# ---------------------------------------------------------------- kv_store, 4 bits
@pytest.mark.parametrize("d,hkv", [(128, 8), (64, 3), (128, 1)])
def test_kv_store_fp4_bit_exact(cuda, d, hkv):
    n, n_slots = 517, 700
    g = torch.Generator().manual_seed(d + hkv)
    spread = torch.exp(4 * torch.randn(n, hkv, 1, generator=g))
    k = (torch.randn(n, hkv, d, generator=g) * spread).to(BF)
    v = torch.randn(n, hkv, d, generator=g).to(BF)
    k[0] = 0
    k[1, :, :16] = 0
    k[2, :, 3], k[3, :, 17], k[4, :, d - 1] = float("inf"), float("nan"), 3e38
    k[5] = 2.0 ** -20
    v[6] = 0.25 * torch.arange(d).to(BF) % 8          # many ties
    k, v = k.to(cuda), v.to(cuda)
    err = torch.zeros(1, dtype=torch.int32, device=cuda)
    pk, pv = (torch.full((n_slots, hkv, d // 2), 7, dtype=torch.uint8, device=cuda) for _ in range(2))
    sk, sv = (torch.full((n_slots, hkv, d // 16), 9, dtype=torch.uint8, device=cuda) for _ in range(2))
    pool = ra.make_pool_desc(pk, pv, err, k_bscale=sk, v_bscale=sv)
    slots = torch.randperm(n_slots, generator=g)[:n].to(torch.int32).to(cuda)
    table, pos = torch.full((n,), -1, dtype=torch.int32, device=cuda), torch.arange(n, dtype=torch.int32, device=cuda)
    ra.kv_store(pool, slots, k, v, table, pos)
    assert ra.rc_sync(err) == ra.RC_OK
    at = slots.long()
    for codes, scales, src in ((pk, sk, k), (pv, sv, v)):
        c_ref, s_ref = f4.quantize(f32(src))
        assert np.array_equal(scales[at].cpu().numpy(), s_ref)
        assert np.array_equal(codes[at].cpu().numpy(), c_ref)
    rest = torch.ones(n_slots, dtype=torch.bool, device=cuda)
    rest[at] = False
    assert bool((pk[rest] == 7).all()) and bool((sv[rest] == 9).all())       # other slots untouched
    assert torch.equal(table, slots)
    before = pk.clone()
    bad = slots.clone()
    bad[3], bad[9] = n_slots, -1
    ra.kv_store(pool, bad, v, k)
    assert ra.rc_sync(err) == ra.RC_ERR_DEVICE
    assert torch.equal(pk[at[3]], before[at[3]]) and torch.equal(pk[at[9]], before[at[9]])
    assert np.array_equal(pk[at[10:]].cpu().numpy(), f4.quantize(f32(v[10:]))[0])


# ---------------------------------------------------------------- kv_store_rope
ROPE_CASES = [
    # pool, hq, hkv, d, rot, offset, interleaved, n, strided
    ("bf16", 32, 8, 128, 128, 0, False, 77, True),
    ("bf16", 32, 8, 128, 64, 0, True, 1, True),
    ("bf16", 4, 4, 64, 64, 0, False, 33, False),
    ("bf16", 5, 1, 64, 32, 32, True, 260, True),
    ("bf16", 8, 8, 128, 96, 16, False, 19, True),
    ("bf16", 3, 2, 128, 32, 96, False, 3001, False),
    ("fp8", 32, 8, 128, 128, 0, False, 50, True),
    ("fp8", 8, 2, 128, 64, 64, True, 7, False),
    ("fp4", 32, 8, 128, 128, 0, False, 51, True),
    ("fp4", 16, 4, 128, 64, 0, True, 9, True),
    ("fp4", 8, 8, 64, 64, 0, False, 400, False),
    ("fp4", 2, 1, 64, 32, 16, False, 13, True),
    ("latent", 16, 1, 576, 64, 512, True, 21, False),
    ("latent", 128, 1, 576, 64, 512, False, 5, True),
]


@pytest.mark.parametrize("fmt,hq,hkv,d,rot,off,inter,n,strided", ROPE_CASES)
def test_kv_store_rope_bit_exact(cuda, fmt, hq, hkv, d, rot, off, inter, n, strided):
    g = torch.Generator().manual_seed(n + d)
    max_pos, n_slots = 40_000, n + 50
    vd = 0 if fmt == "latent" else d
    fused = torch.randn(n, hq * d + hkv * d + hkv * vd + 8, generator=g).to(BF).to(cuda)
    q, k, v = fused[:, :-8].split([hq * d, hkv * d, hkv * vd], 1)
    q, k = q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d))
    v = v.unflatten(1, (hkv, d)) if vd else None
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous() if vd else None
    cs = ra.rope_table(max_pos, rot, device=cuda)
    rope = ra.make_rope_desc(cs, interleaved=inter, offset=off)
    slots = torch.randperm(n_slots, generator=g)[:n].to(torch.int32).to(cuda)
    pos = torch.randint(0, max_pos, (n,), generator=g).to(torch.int32).to(cuda)
    pos[0] = max_pos - 1
    err = torch.zeros(1, dtype=torch.int32, device=cuda)
    w = {"bf16": d, "fp8": d, "fp4": d // 2, "latent": d}[fmt]
    dt = torch.uint8 if fmt in ("fp8", "fp4") else BF
    kw = {}
    if fmt == "latent":
        pk, pv = torch.zeros(n_slots, d, dtype=dt, device=cuda), None
        kw = dict(mla=True, head_dim_v=512)
    else:
        pk, pv = (torch.zeros(n_slots, hkv, w, dtype=dt, device=cuda) for _ in range(2))
    if fmt == "fp8":
        kw = {f"{x}_scale": torch.zeros(n_slots, hkv, device=cuda) for x in "kv"}
    if fmt == "fp4":
        kw = {f"{x}_bscale": torch.zeros(n_slots, hkv, d // 16, dtype=torch.uint8, device=cuda) for x in "kv"}
    pool = ra.make_pool_desc(pk, pv, err, **kw)
    q_out = torch.zeros(n, hq, d, dtype=BF, device=cuda)
    table, tpos = torch.full((n,), -1, dtype=torch.int32, device=cuda), torch.arange(n, dtype=torch.int32, device=cuda)
    before = fused.clone()
    ra.kv_store_rope(pool, rope, slots, pos, k, v, q, q_out, table, tpos)
    assert ra.rc_sync(err) == ra.RC_OK
    assert torch.equal(fused, before) and torch.equal(table, slots)
    t, p, at = cs.cpu().numpy(), pos.cpu().numpy(), slots.long()
    kr, qr = f4.rotate(f32(k), t, p, off, inter), f4.rotate(f32(q), t, p, off, inter)
    assert np.array_equal(bits(q_out), f4.bf16_round(qr))
    # against the 64-bit formula: half a bf16 step, and three fp32 roundings of terms up to |a| + |b|
    q64 = f4.rotate64(f32(q), t, p, off, inter)
    got = hg.bf16_bits_to_f32(bits(q_out)).astype(np.float64)
    slack = 3 * 2.0 ** -24 * 2 * np.abs(f32(q)).max()
    assert (np.abs(got - q64) <= tol.bf16_ulp(np.abs(q64) + slack) / 2 + slack).all()
    if fmt == "latent":
        assert np.array_equal(bits(pk[at]), f4.bf16_round(kr[:, 0]))
    elif fmt == "bf16":
        assert np.array_equal(bits(pk[at]), f4.bf16_round(kr)) and torch.equal(pv[at], v)
    else:
        for codes, name, x in ((pk, "k", kr), (pv, "v", f32(v))):
            got_c = codes[at].cpu().numpy()
            if fmt == "fp4":
                c_ref, s_ref = f4.quantize(x)
                assert np.array_equal(kw[name + "_bscale"][at].cpu().numpy(), s_ref)
                assert np.array_equal(got_c, c_ref)
            else:   # the FP8 oracle's definition on fp32 rows
                scale = (np.abs(x).max(-1) / np.float32(448)).astype(np.float32)
                c_ref = f8.encode((x / scale[..., None]).astype(np.float32).astype(np.float64))
                assert np.array_equal(kw[name + "_scale"][at].cpu().numpy(), scale)
                strip = lambda c: np.where((c & 0x7F) == 0, 0, c)
                assert np.array_equal(strip(got_c), strip(c_ref))
    # in place: the same queries, and nothing else of the projection's output moves
    ra.kv_store_rope(pool, rope, slots, pos, k, v, q)
    assert ra.rc_sync(err) == ra.RC_OK
    assert torch.equal(q, q_out)
    if strided:
        assert torch.equal(fused[:, hq * d:], before[:, hq * d:])


def test_kv_store_rope_at_position_zero_is_kv_store(cuda):
    """Angle 0 turns nothing: the rows are kv_store's, for every pool."""
    g = torch.Generator().manual_seed(5)
    k, v = rand(g, 90, 8, 128), rand(g, 90, 8, 128)
    slots = torch.randperm(90, generator=g).to(torch.int32).to(cuda)
    rope = ra.make_rope_desc(ra.rope_table(4, 128, device=cuda))
    zero = torch.zeros(90, dtype=torch.int32, device=cuda)
    for fmt in ("bf16", "fp8", "fp4"):
        a, b = Pool(fmt, 90, 8, 128, cuda, 1), Pool(fmt, 90, 8, 128, cuda, 2)
        ra.kv_store(a.desc, slots, k, v)
        ra.kv_store_rope(b.desc, rope, slots, zero, k, v)
        assert ra.rc_sync(a.err) == ra.RC_OK and ra.rc_sync(b.err) == ra.RC_OK
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v), fmt
        if fmt != "bf16":
            assert torch.equal(a.ks, b.ks) and torch.equal(a.vs, b.vs), fmt


def test_kv_store_rope_bad_slots_and_positions(cuda):
    g = torch.Generator().manual_seed(6)
    n = 40
    k, v, q = rand(g, n, 8, 128), rand(g, n, 8, 128), rand(g, n, 32, 128)
    rope = ra.make_rope_desc(ra.rope_table(100, 128, device=cuda))
    for fmt in ("bf16", "fp4"):
        p = Pool(fmt, 64, 8, 128, cuda, 3)
        before_k, before_v = p.k.clone(), p.v.clone()
        slots, pos = torch.arange(n, dtype=torch.int32, device=cuda), torch.arange(n, dtype=torch.int32, device=cuda)
        slots[2], slots[5], pos[7], pos[9] = 64, -3, 100, -1
        out = torch.full_like(q, 7.0)
        table, tp = torch.full((n,), -1, dtype=torch.int32, device=cuda), torch.arange(n, dtype=torch.int32, device=cuda)
        ra.kv_store_rope(p.desc, rope, slots, pos, k, v, q, out, table, tp)
        assert ra.rc_sync(p.err) == ra.RC_ERR_DEVICE
        for i in (2, 5, 7, 9):
            assert torch.equal(p.k[i], before_k[i]) and torch.equal(p.v[i], before_v[i]) and int(table[i]) == -1
        assert not torch.equal(p.k[3], before_k[3]) and int(table[3]) == 3
        ref = f4.bf16_round(f4.rotate(f32(q), rope._keep[0].cpu().numpy(), np.clip(pos.cpu().numpy(), 0, 99), 0, False))
        good = [i for i in range(n) if i not in (7, 9)]
        assert np.array_equal(bits(out)[good], ref[good])
        assert bool((out[7] == 7.0).all()) and bool((out[9] == 7.0).all())
        # no tokens, and no queries
        none = torch.zeros(0, dtype=torch.int32, device=cuda)
        ra.kv_store_rope(p.desc, rope, none, none, k[:0], v[:0], q[:0], out[:0])
        ra.kv_store_rope(p.desc, rope, pos[10:11], pos[10:11], k[:1], v[:1])
        assert ra.rc_sync(p.err) == ra.RC_OK


# ---------------------------------------------------------------- attention, 4 bits
DECODE_CASES = [
    # hq, hkv, d, lens
    (32, 8, 128, [1, 17, 64, 200, 1000, 2500, 4097, 0]),
    (64, 8, 128, [5, 129, 2817]),
    (16, 8, 128, [700, 33, 31, 32, 95, 96, 97]),
    (8, 8, 128, [1, 1024]),
    (4, 4, 64, [1, 2, 63, 64, 65, 130, 0, 33]),
    (16, 2, 64, [3000, 15, 16]),
    (8, 4, 64, [511]),
    (8, 2, 64, [1, 700]),
    (32, 8, 128, [48 + (i * 37) % 150 for i in range(160)]),      # one warp per (row, head): the fused epilogue
    (4, 4, 64, [1 + (i * 53) % 200 for i in range(320)]),
]


@pytest.mark.parametrize("hq,hkv,d,lens", DECODE_CASES)
def test_decode_fp4_vs_oracle(cuda, hq, hkv, d, lens):
    n_slots, B = 6000, len(lens)
    pool = Pool("fp4", n_slots, hkv, d, cuda, hq + d)
    rows, table, start, length = tables(lens, n_slots, 3, cuda)
    q = rand(torch.Generator().manual_seed(2), B, hq, d)
    scale = 1.0 / np.sqrt(d)
    desc = ra.make_attn_desc(pool.desc, hq, scale)
    kv = ra.make_kv_table(table, start, length, max(lens))
    ws = torch.empty(ra.attn_decode_workspace(desc, B, max(lens)), dtype=torch.uint8, device=cuda)
    out = torch.full((B + 1, hq, d), 5.0, dtype=BF, device=cuda)
    lse = torch.empty(B, hq, dtype=torch.float32, device=cuda)
    ra.attn_decode(desc, q, kv, B, out[:B], lse, ws)
    assert ra.rc_sync(pool.err) == ra.RC_OK
    k, v = pool.values()
    check(out[:B], lse, f4.attention(f32(q).astype(np.float64), k, v, rows, hq, hkv, scale), pool.u_p)
    assert bool((out[B] == 5.0).all())
    # the library's own scratch: the same kernels on the same plan
    again = torch.empty_like(out[:B])
    if ra.attn_decode_static(desc, q, kv, B, again) == ra.RC_OK:
        assert torch.equal(again, out[:B])


@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_decode_fp4_scales_that_are_not_positive(cuda, scale):
    """A negative scale prefers the smallest products; zero gives the keys' mean."""
    hq, hkv, d, lens = 16, 4, 128, [1, 40, 333, 700]
    pool = Pool("fp4", 2000, hkv, d, cuda, 21)
    rows, table, start, length = tables(lens, 2000, 3, cuda)
    q = rand(torch.Generator().manual_seed(2), len(lens), hq, d)
    desc = ra.make_attn_desc(pool.desc, hq, scale)
    ws = torch.empty(max(ra.attn_decode_workspace(desc, len(lens), 700), 256), dtype=torch.uint8, device=cuda)
    out, lse = torch.empty_like(q), torch.empty(len(lens), hq, dtype=torch.float32, device=cuda)
    ra.attn_decode(desc, q, ra.make_kv_table(table, start, length, 700), len(lens), out, lse, ws)
    assert ra.rc_sync(pool.err) == ra.RC_OK
    k, v = pool.values()
    check(out, lse, f4.attention(f32(q).astype(np.float64), k, v, rows, hq, hkv, float(np.float32(scale))), pool.u_p)


def test_decode_fp4_large_and_small_values(cuda):
    """Rows spread over e^(+-6) in size: peaked softmax, outputs of many units (the mean bar grows with them)."""
    hq, hkv, d, lens = 32, 8, 128, [1, 40, 333, 2049]
    n_slots, B = 4000, len(lens)
    pool = Pool("fp4", n_slots, hkv, d, cuda, 9)
    g = torch.Generator().manual_seed(4)
    k = (torch.randn(n_slots, hkv, d, generator=g) * torch.exp(2 * torch.randn(n_slots, hkv, 1, generator=g))).to(BF).to(cuda)
    v = (torch.randn(n_slots, hkv, d, generator=g) * torch.exp(3 * torch.randn(n_slots, hkv, 1, generator=g))).to(BF).to(cuda)
    ra.kv_store(pool.desc, torch.arange(n_slots, dtype=torch.int32, device=cuda), k, v)
    rows, table, start, length = tables(lens, n_slots, 3, cuda)
    q = rand(g, B, hq, d)
    desc = ra.make_attn_desc(pool.desc, hq, 0.08)
    kv = ra.make_kv_table(table, start, length, max(lens))
    ws = torch.empty(ra.attn_decode_workspace(desc, B, max(lens)), dtype=torch.uint8, device=cuda)
    out, lse = torch.empty(B, hq, d, dtype=BF, device=cuda), torch.empty(B, hq, device=cuda)
    ra.attn_decode(desc, q, kv, B, out, lse, ws)
    assert ra.rc_sync(pool.err) == ra.RC_OK
    kd, vd = pool.values()
    ref, rl, a = f4.attention(f32(q).astype(np.float64), kd, vd, rows, hq, hkv, float(np.float32(0.08)))
    got = hg.bf16_bits_to_f32(bits(out)).astype(np.float64)
    tol.check_values(got, ref, a, u_p=pool.u_p, mean=tol.MEAN_ABS + tol.bf16_ulp(ref).mean() / 4, label="magnitudes")
    # scores are fp32 sums of d products and reach |lse|: 2^-23 d relative at most
    tol.check_lse(lse.cpu().numpy(), rl, tol.LSE_ABS + 2.0 ** -23 * d * np.abs(rl).max())


def test_decode_fp4_nan_blocks_and_bad_slots(cuda):
    """A non-finite block makes the outputs that read it NaN, and no others; one behind a row's end is not read."""
    hq, hkv, d = 8, 2, 128
    pool = Pool("fp4", 300, hkv, d, cuda, 1)
    lens = [100, 90, 65]
    flat = torch.arange(300, dtype=torch.int32, device=cuda)
    start = torch.tensor([0, 100, 200], dtype=torch.int32, device=cuda)
    length = torch.tensor(lens, dtype=torch.int32, device=cuda)
    pool.ks[150, 1] = 255                  # row 1, KV head 1: every score of the head
    pool.vs[40, 0, 2] = 255                # row 0, KV head 0: columns 32..47
    pool.ks[195], pool.vs[299] = 255, 255  # behind the ends of rows 1 and 2
    q = rand(torch.Generator().manual_seed(2), 3, hq, d)
    desc = ra.make_attn_desc(pool.desc, hq, 0.1)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=cuda)
    qo = torch.arange(4, dtype=torch.int32, device=cuda)
    for call in ("decode", "cross", "extend"):
        out = torch.zeros(3, hq, d, dtype=BF, device=cuda)
        kv = ra.make_kv_table(flat, start, length, 100)
        if call == "decode":
            ra.attn_decode(desc, q, kv, 3, out, None, ws)
        elif call == "cross":
            ra.attn_cross(desc, q, qo, kv, 3, 1, out, None, ws)
        else:
            ra.attn_extend(desc, q, qo, kv, 3, 1, out, None, ws)
        assert ra.rc_sync(pool.err) == ra.RC_OK
        nan = torch.isnan(out).cpu().numpy()
        want = np.zeros_like(nan)
        want[0, :4, 32:48] = True
        want[1, 4:] = True
        assert np.array_equal(nan, want), call
    bad = flat.clone()
    bad[10], bad[210] = 300, -1
    kv = ra.make_kv_table(bad, start, length, 100)
    ra.attn_decode(desc, q, kv, 3, out, None, ws)
    assert ra.rc_sync(pool.err) == ra.RC_ERR_DEVICE
    ra.attn_cross(desc, q, qo, kv, 3, 1, out, None, ws)
    assert ra.rc_sync(pool.err) == ra.RC_ERR_DEVICE


@pytest.mark.parametrize("call,fmt,nq", [("decode", "fp4", 1), ("extend", "fp4", 8), ("extend", "fp4", 300),
                                         ("cross", "bf16", 1), ("cross", "fp8", 1), ("cross", "fp4", 1),
                                         ("cross", "bf16", 40), ("cross", "fp8", 40), ("cross", "fp4", 40)])
def test_nan_key_of_a_split_row(cuda, call, fmt, nq):
    """A NaN key in one part of a row's keys: NaN for the heads that read it, lse +infinity, the rest as without it."""
    hq, hkv, d = 8, 2, 128
    pool = Pool(fmt, 4000, hkv, d, cuda, 11)
    lens = [1500, 1400, 700]
    rows, table, start, length = tables(lens, 4000, 5, cuda)
    rows[1] = np.arange(100, 1500, dtype=np.int32)       # row 1's keys are no other row's
    others = np.concatenate([np.arange(100), np.arange(1500, 4000)]).astype(np.int32)
    rows[0], rows[2] = others[:1500], others[1500:2200]
    table = torch.from_numpy(np.concatenate(rows)).to(cuda)
    q = rand(torch.Generator().manual_seed(2), 3 * nq, hq, d)
    qo = torch.arange(4, dtype=torch.int32, device=cuda) * nq
    desc = ra.make_attn_desc(pool.desc, hq, 0.1)
    kv = ra.make_kv_table(table, start, length, 1500)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=cuda)

    def run():
        out, lse = torch.zeros_like(q), torch.zeros(3 * nq, hq, dtype=torch.float32, device=cuda)
        if call == "decode":
            ra.attn_decode(desc, q, kv, 3, out, lse, ws)
        elif call == "cross":
            ra.attn_cross(desc, q, qo, kv, 3, nq, out, lse, ws)
        else:
            ra.attn_extend(desc, q, qo, kv, 3, nq, out, lse, ws)
        assert ra.rc_sync(pool.err) == ra.RC_OK
        return out, lse

    clean, clean_lse = run()
    slot = int(rows[1][300])
    if fmt == "bf16":
        pool.k[slot, 1, 5] = float("nan")
    elif fmt == "fp8":
        pool.ks[slot, 1] = float("nan")
    else:
        pool.ks[slot, 1, 3] = 255
    out, lse = run()
    hit = torch.zeros(3 * nq, hq, dtype=torch.bool, device=cuda)
    hit[nq:2 * nq, 4:] = True
    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isposinf(lse[hit]).all())
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (64, 8, 128), (4, 4, 64)])
def test_cascade_fp4_vs_oracle(cuda, hq, hkv, d):
    """A shared segment read once for all rows, on both grids, equals the flat rows' oracle."""
    n_slots, B, shared = 9000, 40, 700
    pool = Pool("fp4", n_slots, hkv, d, cuda, 99 + hq)
    lens = [shared + 1 + (i * 31) % 150 for i in range(B)]
    rows, table, start, length = tables(lens, n_slots, 5, cuda, shared=shared)
    q = rand(torch.Generator().manual_seed(7), B, hq, d)
    scale = 1.0 / np.sqrt(d)
    desc = ra.make_attn_desc(pool.desc, hq, scale)
    T = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=cuda)
    args = [T(rows[0][:shared]), T([0, shared]), T([0, B]), T(range(B)), T(range(B + 1)), T(range(B))]
    k, v = pool.values()
    ref = f4.attention(f32(q).astype(np.float64), k, v, rows, hq, hkv, scale)
    kv = ra.make_kv_table(table, start + shared, length - shared, max(lens) - shared)
    for host in (False, True):
        more = dict(host_seg_indptr=np.array([0, shared]), host_seg_row_indptr=np.array([0, B])) if host else {}
        casc = ra.make_cascade(*args, max_seg_rows=B, max_seg_len=shared, **more)
        ws = torch.empty(ra.attn_decode_workspace(desc, B, kv.max_len, casc), dtype=torch.uint8, device=cuda)
        out, lse = torch.empty(B, hq, d, dtype=BF, device=cuda), torch.empty(B, hq, device=cuda)
        ra.attn_decode(desc, q, kv, B, out, lse, ws, cascade=casc)
        assert ra.rc_sync(pool.err) == ra.RC_OK
        check(out, lse, ref, pool.u_p, label=f"cascade host={host}")


@pytest.mark.parametrize("hq,hkv,d,reqs", [
    (32, 8, 128, [(1792, 40), (0, 17), (100, 130), (1792, 64), (0, 1)]),
    (64, 8, 128, [(1000, 33), (300, 8), (0, 200)]),
    (8, 8, 128, [(63, 65)]),
    (16, 8, 64, [(32, 9), (0, 70), (5, 64), (700, 3)]),
    (4, 4, 64, [(0, 300)]),
    (8, 1, 64, [(129, 40)]),
])
def test_extend_fp4_vs_oracle(cuda, hq, hkv, d, reqs):
    n_slots = 4000
    pool = Pool("fp4", n_slots, hkv, d, cuda, 7 * hq)
    lens, ns = [p + n for p, n in reqs], [n for _, n in reqs]
    rows, table, start, length = tables(lens, n_slots, 5, cuda)
    T = sum(ns)
    q = rand(torch.Generator().manual_seed(4), T, hq, d)
    qo = torch.tensor(np.concatenate([[0], np.cumsum(ns)]), dtype=torch.int32, device=cuda)
    scale = 1.0 / np.sqrt(d)
    desc = ra.make_attn_desc(pool.desc, hq, scale)
    kv = ra.make_kv_table(table, start, length, max(lens))
    out = torch.full((T + 2, hq, d), 3.0, dtype=BF, device=cuda)
    lse = torch.empty(T, hq, device=cuda)
    ra.attn_extend(desc, q, qo, kv, len(reqs), max(ns), out[:T], lse)
    assert ra.rc_sync(pool.err) == ra.RC_OK
    row_of = [rows[b] for b, n in enumerate(ns) for _ in range(n)]
    lim = [p + i + 1 for p, n in reqs for i in range(n)]
    k, v = pool.values()
    ref = f4.attention(f32(q).astype(np.float64), k, v, row_of, hq, hkv, scale, lim)
    check(out[:T], lse, ref, pool.u_p)
    # with the workspace that splits the keys; what it held before is not read
    size = ra.attn_extend_workspace(desc, len(reqs), max(ns), max(lens))
    ws = torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device=cuda)
    ra.attn_extend(desc, q, qo, kv, len(reqs), max(ns), out[:T], lse, ws)
    assert ra.rc_sync(pool.err) == ra.RC_OK
    check(out[:T], lse, ref, pool.u_p, label="split")
    assert bool((out[T:] == 3.0).all())


def test_extend_fp4_split_covers_few_and_refuses_long_rows(cuda):
    """Small batches with long prefixes are split (both head_dims), and then a row above max_len or with too many
    tokens is flagged and left out; unsplit calls ignore the bound."""
    for hq, hkv, d in ((8, 2, 128), (4, 4, 64)):
        pool = Pool("fp4", 4000, hkv, d, cuda, 4)
        desc = ra.make_attn_desc(pool.desc, hq, 0.1)
        flat = torch.randperm(4000, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(cuda)
        to = lambda *a: torch.tensor(a, dtype=torch.int32, device=cuda)
        lens, ns = [1900, 700, 33], [5, 70, 33]
        size = ra.attn_extend_workspace(desc, 3, 70, 1900)
        assert size > 0
        ws = torch.empty(size, dtype=torch.uint8, device=cuda)
        q = rand(torch.Generator().manual_seed(2), 108, hq, d)
        qo, start = to(0, 5, 75, 108), to(0, 1900, 2600)

        def run(length, max_q=70, w=ws):
            out = torch.full((108, hq, d), 3.0, dtype=BF, device=cuda)
            ra.attn_extend(desc, q, qo, ra.make_kv_table(flat, start, to(*length), 1900), 3, max_q, out, None, w)
            return ra.rc_sync(pool.err), out

        ok, want = run(lens)
        assert ok == ra.RC_OK
        rows = flat.cpu().numpy()
        row_of = [rows[s:s + n] for s, n, k in zip((0, 1900, 2600), lens, ns) for _ in range(k)]
        lim = [n - k + i + 1 for n, k in zip(lens, ns) for i in range(k)]
        k, v = pool.values()
        check(want, None, f4.attention(f32(q).astype(np.float64), k, v, row_of, hq, hkv, float(np.float32(0.1)), lim),
              pool.u_p)
        st, got = run([1901, 700, 33])
        assert st == ra.RC_ERR_DEVICE and bool((got[:5] == 0).all()) and torch.equal(got[5:], want[5:])
        assert run([1901, 700, 33], w=None)[0] == ra.RC_OK
        st, got = run(lens, max_q=69)
        assert st == ra.RC_ERR_DEVICE and bool((got[5:75] == 3.0).all()) and torch.equal(got[:5], want[:5])


# ---------------------------------------------------------------- attn_cross
CROSS_CASES = [
    # pool, hq, hkv, d, tokens per row, keys per row
    ("bf16", 16, 16, 64, [1, 1, 1, 1], [1500, 1, 0, 77]),            # few columns, split keys
    ("bf16", 32, 8, 128, [2, 0, 1, 2], [700, 50, 64, 33]),
    ("bf16", 8, 8, 128, [8, 3, 5], [129, 0, 2000]),
    ("bf16", 4, 4, 64, [1 + i % 7 for i in range(330)], [(i * 29) % 90 for i in range(330)]),   # fused
    ("bf16", 32, 8, 128, [70, 1, 0, 33], [1500, 64, 10, 0]),         # many columns, split keys
    ("bf16", 16, 8, 128, [300, 17], [65, 1000]),
    ("bf16", 4, 4, 64, [260] * 40, [100 + i for i in range(40)]),    # the grid fills the SMs
    ("bf16", 8, 1, 64, [2], [3000]),
    ("bf16", 64, 8, 128, [1] * 3, [513, 3, 64]),
    ("fp8", 32, 8, 128, [2, 1], [900, 31]),
    ("fp8", 32, 8, 128, [50, 9], [900, 0]),
    ("fp4", 64, 8, 128, [1, 1, 1], [900, 0, 31]),
    ("fp4", 8, 8, 64, [8, 0, 7], [33, 5, 2000]),
    ("fp4", 4, 4, 64, [1 + i % 7 for i in range(330)], [(i * 29) % 90 for i in range(330)]),
    ("fp4", 32, 8, 128, [130, 64], [4095, 257]),
    ("fp4", 16, 8, 64, [40, 1], [100, 64]),
]


@pytest.mark.parametrize("fmt,hq,hkv,d,ns,lens", CROSS_CASES)
def test_cross_vs_oracle(cuda, fmt, hq, hkv, d, ns, lens):
    n_slots, B, T = 5000, len(ns), sum(ns)
    pool = Pool(fmt, n_slots, hkv, d, cuda, hq + 3 * d)
    rows, table, start, length = tables(lens, n_slots, 3, cuda)
    q = rand(torch.Generator().manual_seed(2), T, hq, d)
    qo = torch.tensor(np.concatenate([[0], np.cumsum(ns)]), dtype=torch.int32, device=cuda)
    scale = 1.0 / np.sqrt(d)
    desc = ra.make_attn_desc(pool.desc, hq, scale)
    kv = ra.make_kv_table(table, start, length, max(lens))
    size = ra.attn_cross_workspace(desc, B, max(ns), max(lens))
    ws = torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device=cuda)     # NaNs, were they read
    out = torch.full((T + 3, hq, d), 3.0, dtype=BF, device=cuda)
    lse = torch.empty(T, hq, device=cuda)
    ra.attn_cross(desc, q, qo, kv, B, max(ns), out[:T], lse, ws[:size] if size else None)
    assert ra.rc_sync(pool.err) == ra.RC_OK
    pick = list(range(T)) if T <= 400 else list(range(0, T, T // 300))
    row_of = [rows[b] for b, n in enumerate(ns) for _ in range(n)]
    k, v = pool.values()
    ref = f4.attention(f32(q).astype(np.float64)[pick], k, v, [row_of[i] for i in pick], hq, hkv, scale)
    check(out[pick], lse[pick], ref, pool.u_p)
    assert bool((out[T:] == 3.0).all())
    first = out.clone()
    ra.attn_cross(desc, q, qo, kv, B, max(ns), out[:T], None, ws[:size] if size else None)   # no lse; same result
    assert ra.rc_sync(pool.err) == ra.RC_OK and torch.equal(out, first)


@pytest.mark.parametrize("max_q", [2, 64])
@pytest.mark.parametrize("batch,max_len", [(3, 200), (3, 2000)])
def test_cross_refuses_rows_outside_its_bounds(cuda, max_q, batch, max_len):
    """A row with too many tokens is left alone, one whose keys are outside the table or above max_len reads as
    empty; both are flagged and the others computed."""
    hq = hkv = 4
    d = 64
    pool = Pool("bf16", 3000, hkv, d, cuda, 1)
    desc = ra.make_attn_desc(pool.desc, hq, 0.1)
    flat = torch.randperm(3000, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(cuda)
    to = lambda *a: torch.tensor(a, dtype=torch.int32, device=cuda)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=cuda)
    size = ra.attn_cross_workspace(desc, batch, max_q, max_len)

    def run(qo, start, length):
        T = int(qo[-1])
        q = rand(torch.Generator().manual_seed(2), T, hq, d)
        out = torch.full((T, hq, d), 3.0, dtype=BF, device=cuda)
        kv = ra.make_kv_table(flat, start, length, max_len)
        ra.attn_cross(desc, q, qo, kv, batch, max_q, out, None, ws[:size])
        return ra.rc_sync(pool.err), out

    ok, want = run(to(0, 2, 3, 4), to(0, 20, 40), to(20, 20, max_len))
    assert ok == ra.RC_OK
    st, got = run(to(0, 2, 3, 4), to(0, 2990, 40), to(20, 20, max_len))       # past the table
    assert st == ra.RC_ERR_DEVICE and torch.equal(got[:2], want[:2]) and torch.equal(got[3:], want[3:])
    assert bool((got[2] == 0).all())
    for row in (to(0, -1, 40), to(0, 20, 40)):
        st, got = run(to(0, 2, 3, 4), row, to(20, max_len + 1 if int(row[1]) > 0 else 20, max_len))
        assert st == ra.RC_ERR_DEVICE and bool((got[2] == 0).all()) and torch.equal(got[:2], want[:2])
    st, got = run(to(0, 2, 3 + max_q, 4 + max_q), to(0, 20, 40), to(20, 20, max_len))   # row 1: max_q + 1 tokens
    assert st == ra.RC_ERR_DEVICE and torch.equal(got[:2], want[:2]) and bool((got[2:3 + max_q] == 3.0).all())


def test_cross_one_row_per_key_equals_decode(cuda):
    """A row of one token is attn_decode's row."""
    hq, hkv, d, lens = 32, 8, 128, [900, 17, 64, 2000]
    for fmt in ("bf16", "fp8", "fp4"):
        pool = Pool(fmt, 4000, hkv, d, cuda, 3)
        rows, table, start, length = tables(lens, 4000, 1, cuda)
        desc = ra.make_attn_desc(pool.desc, hq, 0.09)
        kv = ra.make_kv_table(table, start, length, 2000)
        q = rand(torch.Generator().manual_seed(2), 4, hq, d)
        a, b = (torch.empty(4, hq, d, dtype=BF, device=cuda) for _ in range(2))
        ws = torch.empty(ra.attn_decode_workspace(desc, 4, 2000), dtype=torch.uint8, device=cuda)
        wc = torch.empty(ra.attn_cross_workspace(desc, 4, 1, 2000), dtype=torch.uint8, device=cuda)
        ra.attn_decode(desc, q, kv, 4, a, None, ws)
        ra.attn_cross(desc, q, torch.arange(5, dtype=torch.int32, device=cuda), kv, 4, 1, b, None, wc)
        assert ra.rc_sync(pool.err) == ra.RC_OK
        # The two calls may split the keys differently, and each chunk rounds its P against a reference of its own: an
        # output moves by up to u_P A + fp32 slack + half a bf16 step on either side, so each is held to the exact
        # value by that bound (tolerance.bound) and not to the other by one step.
        k, v = pool.values()
        ref = f4.attention(f32(q).astype(np.float64), k, v, rows, hq, hkv, float(np.float32(0.09)))
        check(a, None, ref, pool.u_p, label="decode")
        check(b, None, ref, pool.u_p, label="cross")


def test_pool_offsets_beyond_32_bits(cuda):
    """Slots whose byte offsets pass 2^32 in a pool of nine million: stored with rotation, read by every call."""
    n_slots, hq, hkv, d = 9_000_000, 16, 8, 128
    assert n_slots * hkv * d // 2 > 1 << 32
    err = torch.zeros(1, dtype=torch.int32, device=cuda)
    k, v = (torch.zeros(n_slots, hkv, d // 2, dtype=torch.uint8, device=cuda) for _ in range(2))
    ks, vs = (torch.zeros(n_slots, hkv, d // 16, dtype=torch.uint8, device=cuda) for _ in range(2))
    pool = ra.make_pool_desc(k, v, err, k_bscale=ks, v_bscale=vs)
    g = torch.Generator().manual_seed(3)
    n = 300
    slots = (n_slots - 1 - torch.randperm(500_000, generator=g)[:n]).to(torch.int32).to(cuda)
    pos = torch.arange(n, dtype=torch.int32, device=cuda)
    kn, vn, q = rand(g, n, hkv, d), rand(g, n, hkv, d), rand(g, n, hq, d)
    cs = ra.rope_table(n, d, device=cuda)
    qr = torch.empty_like(q)
    ra.kv_store_rope(pool, ra.make_rope_desc(cs), slots, pos, kn, vn, q, qr)
    t, p = cs.cpu().numpy(), pos.cpu().numpy()
    kd = f4.dequantize(*f4.quantize(f4.rotate(f32(kn), t, p, 0, False)))
    vd = f4.dequantize(*f4.quantize(f32(vn)))
    desc = ra.make_attn_desc(pool, hq, 0.09)
    one = lambda *a: torch.tensor(a, dtype=torch.int32, device=cuda)
    kv = ra.make_kv_table(slots, one(0), one(n), n)
    size = max(ra.attn_decode_workspace(desc, 1, n), ra.attn_cross_workspace(desc, 1, 40, n), 256)
    ws = torch.empty(size, dtype=torch.uint8, device=cuda)
    rows = [np.arange(n)] * n
    qx = f32(qr).astype(np.float64)
    ref = f4.attention(qx, kd, vd, rows, hq, hkv, float(np.float32(0.09)), p + 1)
    full = f4.attention(qx[-40:], kd, vd, rows[:40], hq, hkv, float(np.float32(0.09)))
    out = torch.empty_like(q)
    ra.attn_extend(desc, qr, one(0, n), kv, 1, n, out)
    check(out, None, ref, tol.U_F16, label="extend")
    ra.attn_decode(desc, qr[-1:], kv, 1, out[-1:], None, ws)
    check(out[-1:], None, [x[-1:] for x in ref], tol.U_F16, label="decode")
    ra.attn_cross(desc, qr[-40:], one(0, 40), kv, 1, 40, out[-40:], None, ws)
    check(out[-40:], None, full, tol.U_F16, label="cross")
    ra.attn_cross(desc, qr[-1:], one(0, 1), kv, 1, 1, out[-1:], None, ws)
    check(out[-1:], None, [x[-1:] for x in full], tol.U_F16, label="cross of one")
    assert ra.rc_sync(err) == ra.RC_OK
    assert int(k[:1000].max()) == 0


# ---------------------------------------------------------------- together
def _serve(cuda, fmt, graph):
    """Prefill and decode steps of a small batch with positions, then cross attention over an encoder's states, all
    through the pool; returns outputs and their exact values."""
    hq, hkv, d, B, steps = 16, 4, 128, 3, 4
    prompt, enc = [37, 5, 64], [150, 1, 33]
    n_slots = 600
    g = torch.Generator().manual_seed(8)
    pool = Pool(fmt, n_slots, hkv, d, cuda, 3)
    err = pool.err
    total = [p + steps for p in prompt]
    perm = torch.randperm(n_slots, generator=g).to(torch.int32)
    slot_rows = list(perm[:sum(total)].split(total))
    enc_rows = list(perm[sum(total):sum(total) + sum(enc)].split(enc))
    T = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device=cuda)
    table, start = torch.cat(slot_rows).to(cuda), T(np.concatenate([[0], np.cumsum(total)[:-1]]))
    etable, estart, elen = torch.cat(enc_rows).to(cuda), T(np.concatenate([[0], np.cumsum(enc)[:-1]])), T(enc)
    cs = ra.rope_table(200, d, device=cuda)
    rope = ra.make_rope_desc(cs)
    scale = 1.0 / np.sqrt(d)
    desc = ra.make_attn_desc(pool.desc, hq, scale)
    ek, ev = rand(g, sum(enc), hkv, d), rand(g, sum(enc), hkv, d)
    width = (hq + 2 * hkv) * d
    proj = [rand(g, sum(prompt), width)] + [rand(g, B, width) for _ in range(steps)]
    pos = [T(np.concatenate([np.arange(p) for p in prompt]))] + [T([p + i for p in prompt]) for i in range(steps)]
    slots = [torch.cat([r[:p] for r, p in zip(slot_rows, prompt)]).to(cuda)] + \
            [torch.stack([r[p + i] for r, p in zip(slot_rows, prompt)]).to(cuda) for i in range(steps)]
    lens = [T(prompt)] + [T([p + i + 1 for p in prompt]) for i in range(steps)]
    qo, qo1 = T(np.concatenate([[0], np.cumsum(prompt)])), T(range(B + 1))
    qr = [torch.empty(x.shape[0], hq, d, dtype=BF, device=cuda) for x in proj]
    own, cross = [torch.empty_like(x) for x in qr], [torch.empty_like(x) for x in qr]
    ws = torch.empty(max(ra.attn_decode_workspace(desc, B, max(total)), 256), dtype=torch.uint8, device=cuda)
    wc = torch.empty(max(ra.attn_cross_workspace(desc, B, max(prompt), max(enc)),
                         ra.attn_cross_workspace(desc, B, 1, max(enc)), 256), dtype=torch.uint8, device=cuda)
    ekv = ra.make_kv_table(etable, estart, elen, max(enc))

    def all_steps():
        ra.kv_store(pool.desc, etable, ek, ev)
        for i, x in enumerate(proj):
            q, k, v = (t.unflatten(1, (-1, d)) for t in x.split([hq * d, hkv * d, hkv * d], 1))
            ra.kv_store_rope(pool.desc, rope, slots[i], pos[i], k, v, q, qr[i])
            kv = ra.make_kv_table(table, start, lens[i], max(total))
            if i == 0:
                ra.attn_extend(desc, qr[0], qo, kv, B, max(prompt), own[0])
                ra.attn_cross(desc, qr[0], qo, ekv, B, max(prompt), cross[0], None, wc)
            else:
                ra.attn_decode(desc, qr[i], kv, B, own[i], None, ws)
                ra.attn_cross(desc, qr[i], qo1, ekv, B, 1, cross[i], None, wc)

    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            all_steps()      # once before the capture
        torch.cuda.current_stream().wait_stream(side)
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            all_steps()
        for t in own + cross + qr:
            t.zero_()
        for t in proj:       # other inputs than the captured run's
            t.copy_(rand(g, *t.shape))
        cg.replay()
    else:
        all_steps()
    assert ra.rc_sync(err) == ra.RC_OK
    # the oracle: rotated, held as the pool holds it, attended
    t = cs.cpu().numpy()
    hold = {"bf16": lambda x: hg.bf16_bits_to_f32(f4.bf16_round(x)).astype(np.float64),
            "fp4": lambda x: f4.dequantize(*f4.quantize(x))}[fmt]
    ks, vs, refs = [[] for _ in range(B)], [[] for _ in range(B)], []
    eks, evs = hold(f32(ek)), hold(f32(ev))
    eoff = np.concatenate([[0], np.cumsum(enc)])
    for i, x in enumerate(proj):
        q, k, v = (a.unflatten(1, (-1, d)) for a in x.split([hq * d, hkv * d, hkv * d], 1))
        p = pos[i].cpu().numpy()
        kr, vr = hold(f4.rotate(f32(k), t, p, 0, False)), hold(f32(v))
        qx = hg.bf16_bits_to_f32(f4.bf16_round(f4.rotate(f32(q), t, p, 0, False))).astype(np.float64)
        of = np.repeat(np.arange(B), prompt if i == 0 else [1] * B)
        for r, b in enumerate(of):
            ks[b].append(kr[r])
            vs[b].append(vr[r])
        off = np.concatenate([[0], np.cumsum([len(y) for y in ks])])
        K, V = np.stack(sum(ks, [])), np.stack(sum(vs, []))
        a = f4.attention(qx, K, V, [np.arange(off[b], off[b + 1]) for b in of], hq, hkv, scale, p + 1)
        c = f4.attention(qx, eks, evs, [np.arange(eoff[b], eoff[b + 1]) for b in of], hq, hkv, scale)
        refs.append((a, c))
    return pool, own, cross, refs


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_prefill_decode_and_cross_together(cuda, fmt, graph):
    pool, own, cross, refs = _serve(cuda, fmt, graph)
    for i, (a, c) in enumerate(refs):
        check(own[i], None, a, pool.u_p, label=f"step {i}")
        check(cross[i], None, c, pool.u_p, label=f"cross {i}")


def test_decode_steps_store_into_an_fp4_pool(cuda):
    """attn_decode_steps with store_slots equals kv_store and attn_decode call by call."""
    hq, hkv, d, B = 32, 8, 128, 5
    lens = [70, 1, 33, 200, 129]
    rows, table, start, length = tables([n + 3 for n in lens], 2000, 4, cuda)
    g = torch.Generator().manual_seed(1)
    T = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=cuda)
    steps = []
    for i in range(3):
        steps.append(dict(q=rand(g, B, hq, d), k_new=rand(g, B, hkv, d), v_new=rand(g, B, hkv, d),
                          store_slots=T([r[n + i] for r, n in zip(rows, lens)]), len=T([n + i + 1 for n in lens]),
                          max_len=max(lens) + i + 1))
    outs = []
    for whole in (True, False):
        pool = Pool("fp4", 2000, hkv, d, cuda, 2)
        desc = ra.make_attn_desc(pool.desc, hq, 0.09)
        kv = ra.make_kv_table(table, start, length, max(lens) + 3)
        ws = torch.empty(ra.attn_decode_workspace(desc, B, max(lens) + 3), dtype=torch.uint8, device=cuda)
        o = [torch.empty(B, hq, d, dtype=BF, device=cuda) for _ in range(3)]
        if whole:
            ra.attn_decode_steps(desc, kv, B, [dict(s, out=o[i]) for i, s in enumerate(steps)], ws)
        else:
            for i, s in enumerate(steps):
                ra.kv_store(pool.desc, s["store_slots"], s["k_new"], s["v_new"])
                ra.attn_decode(desc, s["q"], ra.make_kv_table(table, start, s["len"], s["max_len"]), B, o[i], None, ws)
        assert ra.rc_sync(pool.err) == ra.RC_OK
        outs.append(o)
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_two_streams_with_their_own_workspaces(cuda):
    """Cross and decode calls that overlap on two streams give what they give alone."""
    hq, hkv, d, lens = 16, 8, 128, [3000, 1500]
    pool = Pool("fp4", 4000, hkv, d, cuda, 2)
    rows, table, start, length = tables(lens, 4000, 4, cuda)
    desc = ra.make_attn_desc(pool.desc, hq, 0.09)
    kv = ra.make_kv_table(table, start, length, 3000)
    q = rand(torch.Generator().manual_seed(1), 40, hq, d)
    qo = torch.tensor([0, 20, 40], dtype=torch.int32, device=cuda)

    def call(stream=None, n=1):
        o, c = torch.zeros(2, hq, d, dtype=BF, device=cuda), torch.zeros(40, hq, d, dtype=BF, device=cuda)
        ws = torch.empty(ra.attn_decode_workspace(desc, 2, 3000), dtype=torch.uint8, device=cuda)
        wc = torch.empty(ra.attn_cross_workspace(desc, 2, 20, 3000), dtype=torch.uint8, device=cuda)
        torch.cuda.synchronize()
        for _ in range(n):
            ra.attn_decode(desc, q[:2], kv, 2, o, None, ws, stream=stream)
            ra.attn_cross(desc, q, qo, kv, 2, 20, c, None, wc, stream=stream)
        return o, c, ws, wc

    alone = call()
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [call(s, 20) for s in streams]
    torch.cuda.synchronize()
    assert ra.rc_sync(pool.err) == ra.RC_OK
    for x in both:
        assert torch.equal(x[0], alone[0]) and torch.equal(x[1], alone[1])


@pytest.mark.parametrize("cascade", [True, False])
def test_few_shot_workload_over_a_4_bit_pool(cuda, cascade):
    """The few-shot workload (reduced) through the scheduler and the engine: prefill over the cached examples, decode
    steps storing each new token; sampled requests against the oracle on the oracle's own quantisation."""
    from radixattention_prefix_shared_tree_gb300 import workloads as wl
    from radixattention_prefix_shared_tree_gb300.driver import DeviceEngine
    from synth import traces
    from synth.model import SynthModel
    tr = traces.few_shot(n_questions=40, max_new=5)
    sh = tr.shape
    model = SynthModel(sh, tr.seed, tr.vocab, device=cuda)
    eng = DeviceEngine(sh, 1 << 16, device=cuda, kv_fp4=True)
    runner = wl.Runner(ra.RadixCache(1 << 16), model, eng, policy=ra.RC_LPM, cascade=cascade, collect=True)
    reqs = wl.run_few_shot(runner, tr)
    assert ra.rc_sync(eng.err) == ra.RC_OK
    assert runner.last_layout.use_cascade == cascade
    for r in reqs[::6]:
        h = model.hashes(r.rid)
        pos, out, lse = runner.extend_out[r.rid]
        pos, out, lse = list(pos), [out], [lse]
        for p, o, l in runner.decode_out[r.rid]:
            pos.append(p)
            out.append(o[None])
            lse.append(l[None])
        n = max(pos) + 1
        held = [f4.dequantize(*f4.quantize(hg.bf16_bits_to_f32(hg.gen_values(h[:n], kind, sh.kv_heads, sh.head_dim_k)
                                                               .reshape(n, sh.kv_heads, -1))))
                for kind in (hg.KIND_K, hg.KIND_V)]
        q = hg.bf16_bits_to_f32(hg.gen_values(h[np.asarray(pos)], hg.KIND_Q, sh.q_heads, sh.head_dim_k)
                                .reshape(len(pos), sh.q_heads, -1)).astype(np.float64)
        ref, rl, a = f4.attention(q, *held, [np.arange(p + 1) for p in pos], sh.q_heads, sh.kv_heads, sh.scale)
        got = hg.bf16_bits_to_f32(np.concatenate([np.asarray(o).reshape(-1, sh.q_heads, sh.head_dim_v) for o in out]))
        tol.check_values(got, ref, a, u_p=tol.U_F16, label="fp4 workload")
        tol.check_lse(np.concatenate([np.asarray(l).reshape(-1, sh.q_heads) for l in lse]), rl)
