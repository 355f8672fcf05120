"""Calls at the edge of what the header allows: the largest bounds, unused axes, very many prompts."""
from __future__ import annotations

import subprocess
import sys

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra
from oracle import fp4_oracle as f4
from radixattention_prefix_shared_tree_gb300 import workloads as wl
from radixattention_prefix_shared_tree_gb300.driver import DeviceEngine
from synth import hashgen as hg
from synth.model import SynthModel
from tests import tolerance as tol
from tests.conftest import ROOT
from tests.test_gpu_generation import shape_of, values
from tests.test_gpu_pool_rows import make_pool

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("w", [2, 6, 11, 32])
def test_reorder_without_a_bound_on_columns(cuda, w):
    """max_cols up to the largest whole number: the grid follows the table."""
    b, room, cols = 3, 40, 25
    table = torch.arange(b * w * room, dtype=torch.int32, device=cuda)
    start = (torch.arange(b * w, dtype=torch.int32, device=cuda) * room).view(b, w)
    first = torch.full((b,), 5, dtype=torch.int32, device=cuda)
    par = torch.arange(w, dtype=torch.int32, device=cuda).flip(0).repeat(b, 1).contiguous()
    want = table.clone().view(b, w, room)
    want[:, :, 5:5 + cols] = want[:, :, 5:5 + cols].flip(1)
    for bound in (cols, 2 ** 31 - 1, 2 ** 31 - 128, 2 ** 31 - 600):
        out, err = table.clone(), torch.zeros(1, dtype=torch.int32, device=cuda)
        ra.beam_reorder(out, start, first, first + cols, par, bound, err=err)
        assert ra.rc_sync(err) == ra.RC_OK
        assert torch.equal(out.view(b, w, room), want)
    # more columns than the table has entries is more than any bound
    out = table.clone()
    ra.beam_reorder(out, start, first, first + b * w * room + 1, par, 2 ** 31 - 1, err=err)
    assert ra.rc_sync(err) == ra.RC_ERR_DEVICE and torch.equal(out, table)
    # an empty table: rows without columns are fine, others are not in it
    zero = torch.zeros_like(start)
    for last, st in ((first, ra.RC_OK), (first + 1, ra.RC_ERR_DEVICE)):
        torch.cuda.synchronize()
        got = ra.lib().beam_reorder(out.data_ptr(), out.data_ptr(), 0, zero.data_ptr(), first.data_ptr(), last.data_ptr(),
                                    par.data_ptr(), b, w, 2 ** 31 - 1, err.data_ptr(), None)
        assert got == ra.RC_OK and ra.rc_sync(err) == st
    assert torch.equal(out, table)


@pytest.mark.parametrize("sections", [[32, 32, 0], [64, 0, 0], [20, 0, 44, 0]])
@pytest.mark.parametrize("n", [1, 300])
def test_positions_on_an_axis_that_no_pair_turns_by(cuda, sections, n):
    """A model of three axes whose last section is empty passes its [3, n] positions; the last row has no effect."""
    g = torch.Generator(device=cuda).manual_seed(n)
    axis = ra.rope_axes(sections)
    used, rope = max(axis) + 1, ra.make_rope_desc(ra.rope_table(50, 128, device=cuda), pair_axis=axis)
    pos = torch.randint(0, 50, (len(sections), n), generator=g, device=cuda).to(torch.int32)
    pos[used:] = -7
    k, v = (torch.randn(n, 2, 128, generator=g, device=cuda).to(BF) for _ in range(2))
    slots = torch.randperm(n, generator=g, device=cuda).to(torch.int32)
    got = []
    for p in (pos, pos[:used].contiguous() if used > 1 else pos[0]):
        pool, arrays, err = make_pool("bf16", n, 2, 128, cuda)
        ra.kv_store_rope(pool, rope, slots, p, k, v)
        assert ra.rc_sync(err) == ra.RC_OK
        got.append(arrays)
    assert all(torch.equal(a, b) for a, b in zip(*got)) and torch.equal(got[0][1][slots.long()], v)


def prompts_at_once(cuda, lens, hq, hkv, d, seed, err):
    g = torch.Generator(device=cuda).manual_seed(seed)
    n = int(lens.sum())
    q, k, v = (torch.randn(n, h, d, generator=g, device=cuda).to(BF) for h in (hq, hkv, hkv))
    ip = torch.cat([lens.new_zeros(1), lens]).cumsum(0).to(torch.int32).to(cuda)
    out, lse = torch.zeros_like(q), torch.zeros(n, hq, device=cuda)
    ra.attn_prompt(q, k, v, ip, 0.1, out, lse, err)
    return q, k, v, ip, out, lse


@pytest.mark.parametrize("batch,most,hq,hkv,d", [(1024, 2, 8, 2, 64), (1025, 700, 4, 2, 64), (2049, 3, 4, 4, 64),
                                                 (5000, 2, 4, 1, 128), (3000, 400, 8, 8, 64), (40, 5000, 8, 2, 128)])
def test_very_many_prompts(cuda, batch, most, hq, hkv, d):
    """Thousands of prompts of all lengths (none among them), one much longer: a prompt's rows do not depend on the
    others in its batch, so they are, bit for bit, those of the same prompts a few at a time."""
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, most + 1, (batch,), generator=g)
    lens[torch.rand(batch, generator=g) < 0.2] = 0
    lens[batch // 3] = 3001
    err = torch.zeros(1, dtype=torch.int32, device=cuda)
    q, k, v, ip, out, lse = prompts_at_once(cuda, lens, hq, hkv, d, batch, err)
    few_out, few_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for a in range(0, batch, 100):
        ra.attn_prompt(q, k, v, ip[a:a + 101], 0.1, few_out, few_lse, err)
    assert ra.rc_sync(err) == ra.RC_OK
    assert torch.equal(out, few_out) and torch.equal(lse, few_lse)
    assert bool((lse != 0).any(1).all())


def test_time_follows_the_number_of_prompts(cuda):
    """100,000 prompts of a token, then as many of none but a few: a prompt is looked for once a level (25 ms), not once
    a unit (3.4 ms for 5,000 prompts, and that grew with the square of their number)."""
    err = torch.zeros(1, dtype=torch.int32, device=cuda)
    for lens in (torch.ones(100_000, dtype=torch.int64), (torch.arange(100_000) % 5000 == 4999).long() * 700):
        prompts_at_once(cuda, lens, 8, 8, 64, 1, err)
        assert ra.rc_sync(err) == ra.RC_OK
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        q, k, v, ip, out, lse = prompts_at_once(cuda, lens, 8, 8, 64, 2, err)
        b.record()
        assert ra.rc_sync(err) == ra.RC_OK
        assert a.elapsed_time(b) < 200, "ms"
        if bool((lens == 1).all()):     # a token alone: its own value
            assert torch.equal(out, v)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("lens", [[400, 1, 77], [1300]])
def test_whole_prompts_over_pools_of_codes_vs_oracle(cuda, fmt, lens):
    """DeviceEngine.prompt against the oracle over the values that it reads back: the pool's own of 4 bits, those
    of an E4M3 pool rounded to bf16, with the softmax weights in bf16; extend over the same tokens against the
    pool's own values, with the weights in f16."""
    sh, pool = shape_of(), 4000
    model = SynthModel(sh, 5, 500, device=cuda)
    for whole in (True, False):
        eng = DeviceEngine(sh, pool, cuda, kv_fp8=fmt == "fp8", kv_fp4=fmt == "fp4")
        runner = wl.Runner(ra.RadixCache(pool), model, eng, collect=True, whole_prompts=whole)
        reqs = [runner.request((np.arange(n) * (i + 3) % 500).astype(np.int32), 1) for i, n in enumerate(lens)]
        runner.serve(reqs)
        assert ra.rc_sync(eng.err) == ra.RC_OK
        for r in reqs:
            h = hg.prefix_hashes(r.prompt, model.seed)
            q = hg.bf16_bits_to_f32(hg.gen_values(h, hg.KIND_Q, sh.q_heads, sh.head_dim_k)).astype(np.float64)
            kv = values(fmt, eng, sh, h)
            if whole:
                kv = [hg.bf16_bits_to_f32(f4.bf16_round(x.astype(np.float32))).astype(np.float64) for x in kv]
            o, t, a = f4.attention(q, *kv, [np.arange(i + 1) for i in range(len(h))], sh.q_heads, sh.kv_heads, sh.scale)
            _, out, lse = runner.extend_out[r.rid]
            tol.check_values(hg.bf16_bits_to_f32(out).astype(np.float64), o, a, u_p=tol.U_BF16 if whole else tol.U_F16)
            tol.check_lse(lse, t)


@pytest.mark.parametrize("hkv,d,n", [(4, 128, 64), (3, 64, 5000)])
def test_rows_of_4_bits_move_between_pools(cuda, hkv, d, n):
    """Rows of a 4-bit pool, read back and stored in another, are the same codes and scales: their values are exact in
    bf16, and the largest of a block is 6 scales (a scale of four bits is within 2^-4 of amax / 6, so that amax is at
    least 5.6 of them and its code 6), so that the block gets its scale again.  Zeros of either sign and blocks
    with a NaN likewise.  (Blocks below 6 x 2^-14, whose scales go in steps of 2^-17, need not.)"""
    g = torch.Generator(device=cuda).manual_seed(n)
    src, had, err = make_pool("fp4", n, hkv, d, cuda)
    spread = torch.exp2(torch.randint(-8, 9, (n, hkv, 1), generator=g, device=cuda).float())
    k, v = ((torch.randn(n, hkv, d, generator=g, device=cuda) * spread).to(BF) for _ in range(2))
    k[1], k[2], k[3, :, 5] = 0.0, -0.0, float("nan")
    every = torch.randperm(n, generator=g, device=cuda).to(torch.int32)
    ra.kv_store(src, every, k, v)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    ra.kv_load(src, every, ko, vo)
    dst, got, err2 = make_pool("fp4", n, hkv, d, cuda, fill=7)
    ra.kv_store(dst, every, ko, vo)
    assert ra.rc_sync(err) == ra.RC_OK and ra.rc_sync(err2) == ra.RC_OK
    assert all(torch.equal(a, b) for a, b in zip(had, got))


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("v,gain", [(500, 4.0), (7142, 1.0), (32_000, 4.0), (130_001, 1.0)])
def test_select_scores_before_their_rounding(cuda, v, gain, f32):
    """A beam's score and its best logit that all but cancel the log-sum-exp leave the latter's error: at most 2^-20.
    Terms are off by 2^-22 (ex2) and, from their arguments' rounding, by ln 2 |y| 2^-24 where y is the exponent (8 on
    the weighted average here: 2^-21.5), a thread's eight terms at a time by 3 x 2^-24, its factor by 2^-23 (9.2e-7
    in all), and what the calls of one row and of all rows differ by is at most twice that."""
    g = torch.Generator(device=cuda).manual_seed(v)
    x = (torch.randn(96, 1, v, generator=g, device=cuda) * gain).to(torch.float32 if f32 else BF)
    lse, top = torch.logsumexp(x.double(), -1), x.double().max(-1).values
    s = (lse - top).float()
    exact = s.double() + top - lse

    def best(a, b):
        out = torch.empty(b - a, 1, device=cuda)
        tok, par = (torch.empty(b - a, 1, dtype=torch.int32, device=cuda) for _ in range(2))
        ra.beam_select(x[a:b], s[a:b], out, tok, par)
        return out.double()

    every, alone = best(0, 96), torch.cat([best(i, i + 1) for i in range(96)])
    assert (every - exact).abs().max().item() <= 2.0 ** -20
    assert (alone - exact).abs().max().item() <= 2.0 ** -20
    assert (every - alone).abs().max().item() <= 2.0 ** -19


FIRST_CALLS = """
import torch
import radixattention_prefix_shared_tree_gb300 as ra
BF, dev = torch.bfloat16, torch.device("cuda")
n, ints = {n}, dict(dtype=torch.int32, device=dev)
k, v, q = (torch.randn(n, h, 128, device=dev).to(BF) for h in (8, 8, 32))
pools = [[torch.zeros(n, 8, 128, dtype=BF, device=dev) for _ in range(2)] for _ in range(2)]
descs, rope = [ra.make_pool_desc(*p) for p in pools], ra.make_rope_desc(ra.rope_table(n, 128, device=dev))
at, ip = torch.arange(n, **ints), torch.arange(0, n + 1, max(n // {prompts}, 1), **ints)
outs = [[torch.zeros_like(x) for x in (q, k, v, q)] for _ in range(2)]


def calls(desc, o):
    ra.kv_store_rope(desc, rope, at, at, k, v, q, o[0])
    ra.kv_load(desc, at, o[1], o[2])
    ra.attn_prompt(o[0], o[1], o[2], ip, 0.1, o[3])


torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    calls(descs[0], outs[0])
g.replay()
calls(descs[1], outs[1])
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(*outs)) and bool(outs[0][3].any())
"""


@pytest.mark.parametrize("n,prompts", [(1, 1), (1100, 1100), (4001, 3)])
def test_first_calls_of_a_process_are_captured(cuda, n, prompts):
    """What a call asks the driver about its kernels the first time may be asked while a graph is captured."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(n=n, prompts=prompts)], capture_output=True, text=True,
                       timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
