"""E4M3 pools whose V rows are small, large, or both: the products' weights
(softmax weight times V scale, in f16) keep their bits whatever the scales.

Bar.  tests/tolerance.py's derived terms without its flat 1e-2, plus f16's
subnormals: the weights are held in a unit of the largest V scale that a CTA or
warp has met, which is at least 2^2 in it, so a weight that falls below f16's
normal numbers is off by at most 2^-25 of that unit, 2^-27 of the largest scale.
Over n keys of codes up to 448 and a softmax sum of at least 1 that is
n 2^-27 max|V| at most.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra
from oracle import fp4_oracle as f4
from synth import hashgen as hg
from tests import tolerance as tol
from tests.test_gpu_operators import BF, Pool, bits, f32, rand

pytestmark = pytest.mark.gpu

HQ, HKV, D = 8, 2, 128

# V's size by key position in a row, from 0 to 1
GAINS = {
    "1e-3": lambda x: np.full_like(x, 1e-3),
    "1e-5": lambda x: np.full_like(x, 1e-5),
    "1e-20": lambda x: np.full_like(x, 1e-20),
    "1e5": lambda x: np.full_like(x, 1e5),
    "1e20": lambda x: np.full_like(x, 1e20),
    "rising": lambda x: 10.0 ** (8 * x - 6),
    "falling": lambda x: 10.0 ** (2 - 8 * x),
    "zeros, then ones": lambda x: (x >= 0.5).astype(np.float64),
    "one large": lambda x: np.where(x == x[len(x) // 3], 1e3, 1e-1),
}


def make(cuda, gain, lens):
    """Rows of consecutive slots whose V grows or shrinks along the row."""
    n = sum(lens)
    pool = Pool("fp8", n, HKV, D, cuda, 17)
    size = np.concatenate([GAINS[gain](np.linspace(0, 1, k) if k > 1 else np.ones(1)) for k in lens])
    g = torch.Generator().manual_seed(6)
    v = (torch.randn(n, HKV, D, generator=g) * torch.from_numpy(size).float()[:, None, None]).to(BF).to(cuda)
    ra.kv_store(pool.desc, torch.arange(n, dtype=torch.int32, device=cuda), pool.src_k, v)
    to = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=cuda)
    start = np.concatenate([[0], np.cumsum(lens)[:-1]])
    rows = [np.arange(s, s + k) for s, k in zip(start, lens)]
    return pool, rows, to(range(n)), to(start), to(lens)


def check_relative(out, ref, vmax, n):
    o, _, a = ref
    got = hg.bf16_bits_to_f32(bits(out)).astype(np.float64)
    e = tol.U_F16 * a + tol.FP32_SLACK * (a + np.abs(o)) + n * 2.0 ** -27 * vmax
    bound = e + tol.bf16_ulp(np.abs(o) + e) / 2
    err = np.abs(got - o)
    assert np.isfinite(got).all()
    assert (err <= bound).all(), f"max err/bound {(err / bound).max():.3g}"


@pytest.mark.parametrize("gain", list(GAINS))
@pytest.mark.parametrize("call", ["decode split", "decode whole", "cascade", "extend", "cross 1", "cross 40"])
def test_v_rows_of_any_size(cuda, call, gain):
    lens = [60, 64, 33, 1] if call == "decode whole" else [1500, 700, 64, 1]
    pool, rows, table, start, length = make(cuda, gain, lens)
    B, nq = len(lens), {"extend": 1, "cross 40": 40}.get(call, 1)
    scale = 0.09
    q = rand(torch.Generator().manual_seed(2), B * nq, HQ, D)
    qo = torch.arange(B + 1, dtype=torch.int32, device=cuda) * nq
    desc = ra.make_attn_desc(pool.desc, HQ, scale)
    kv = ra.make_kv_table(table, start, length, max(lens))
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=cuda)
    out = torch.empty_like(q)
    if call.startswith("decode"):
        ra.attn_decode(desc, q, kv, B, out, None, ws)
    elif call == "cascade":     # row 0's first 1,400 keys as a segment of its own
        to = lambda *a: torch.tensor(a, dtype=torch.int32, device=cuda)
        casc = ra.make_cascade(table[:1400].contiguous(), to(0, 1400), to(0, 1), to(0), to(0, 1, 1, 1, 1), to(0),
                               max_seg_rows=1, max_seg_len=1400)
        kv = ra.make_kv_table(table, to(1400, 1500, 2200, 2264), to(100, 700, 64, 1), 700)
        ra.attn_decode(desc, q, kv, B, out, None, ws, cascade=casc)
    elif call == "extend":
        ra.attn_extend(desc, q, qo, kv, B, nq, out)
    else:
        ra.attn_cross(desc, q, qo, kv, B, nq, out, None, ws)
    assert ra.rc_sync(pool.err) == ra.RC_OK
    k, v = pool.values()
    row_of = [rows[b] for b in range(B) for _ in range(nq)]
    ref = f4.attention(f32(q).astype(np.float64), k, v, row_of, HQ, HKV, float(np.float32(scale)))
    vmax = np.array([np.abs(v[r]).max() for r in row_of])[:, None, None]
    n = np.array([len(r) for r in row_of])[:, None, None]
    check_relative(out, ref, vmax, n)
