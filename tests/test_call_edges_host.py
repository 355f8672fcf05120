"""Refusals of calls at the edge of what the header allows; every call here ends at its
checks on the host, before any CUDA call."""
from __future__ import annotations

from types import SimpleNamespace

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra
from radixattention_prefix_shared_tree_gb300.driver import BeamBatch
from tests.test_more_operators_host import call_load, call_prompt, pool

BF = torch.bfloat16
A, OK = ra.RC_ERR_ARG, ra.RC_OK


def pools():
    """A pool of every kind with its arrays' names and sizes in bytes."""
    n, h, d = 64, 8, 128
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    yield pool(n, h, d), dict(k=n * h * d * 2, v=n * h * d * 2)
    yield ra.make_pool_desc(torch.zeros(n, 576, dtype=BF), None, mla=True, head_dim_v=512), dict(k=n * 576 * 2)
    yield (ra.make_pool_desc(u8(n, h, d), u8(n, h, d), k_scale=torch.zeros(n, h), v_scale=torch.zeros(n, h)),
           dict(k=n * h * d, v=n * h * d, k_scale=n * h * 4, v_scale=n * h * 4))
    yield (ra.make_pool_desc(u8(n, h, d // 2), u8(n, h, d // 2), k_bscale=u8(n, h, d // 16), v_bscale=u8(n, h, d // 16)),
           dict(k=n * h * d // 2, v=n * h * d // 2, k_bscale=n * h * d // 16, v_bscale=n * h * d // 16))


def test_kv_load_into_its_own_pool_is_refused(built):
    for p, sizes in pools():
        latent = bool(p.mla)
        row = 576 if latent else 1024
        far = 1 << 40          # (addresses only)
        base = dict(slots=far, n=4, k=far + (1 << 20), ks=row, v=None if latent else far + (2 << 20), vs=row)
        ends = [(getattr(p, name), size) for name, size in sizes.items()] + [(far, 16)]
        for at, size in ends:
            for out in ("k",) if latent else ("k", "v"):
                for to in (at, at + size - 16, at - 4 * row * 2 + 16):
                    to -= to % 16
                    assert call_load(p, **{**base, out: to}) == A, (sizes, out)
                # a stride that steps over the array's start: its last row's end is inside
                assert call_load(p, **{**base, out: at - at % 16 - 3 * 2 * row * 2, out + "s": 2 * row}) == A
            assert call_load(p, **{**base, "n": 0, "k": at - at % 16}) == OK      # nothing is written



def test_attn_prompt_results_over_inputs_are_refused(built):
    step = 1 << 20      # (addresses only; the arrays below are smaller)
    far = {n: (1 << 40) + i * step for i, n in enumerate(("q", "k", "v", "ip", "out", "lse"))}
    size = dict(q=4 * 4096 * 2, k=4 * 1024 * 2, v=4 * 1024 * 2, ip=8, out=4 * 4096 * 2)
    for name, nbytes in size.items():
        for to in (far[name], far[name] + nbytes - 4, far[name] - 4 * 32 * 4 + 4):
            assert call_prompt(**{**far, "batch": 1, "lse": to}) == A, name
    for to in (far["ip"], far["ip"] - 4 * 4096 * 2 + 16):
        assert call_prompt(**{**far, "batch": 1, "out": to}) == A


@pytest.mark.parametrize("sections", [[32, 32, 0], [64, 0, 0], [64], [32, 0, 32, 0]])
def test_positions_may_have_axes_that_no_pair_turns_by(built, sections):
    rope = ra.make_rope_desc(ra.rope_table(16, 128, device="cpu"), pair_axis=ra.rope_axes(sections))
    k, s = torch.zeros(4, 8, 128, dtype=BF), torch.zeros(4, dtype=torch.int32)

    def refusal(pos):
        with pytest.raises((ValueError, RuntimeError)) as e:     # (at the latest because these tensors are the host's)
            ra.kv_store_rope(pool(), rope, s, pos, k, k)
        return "expected a contiguous int32" in str(e.value)

    used = max(a for a, n in enumerate(sections) if n) + 1
    for axes in range(1, 6):
        assert refusal(torch.zeros(axes, 4, dtype=torch.int32)) == (not used <= axes <= 4), axes
    assert refusal(s) == (used > 1)
    assert refusal(torch.zeros(4, 3, dtype=torch.int32)) and refusal(torch.zeros(1, 3, 4, dtype=torch.int32))


def test_attn_prompt_refuses_more_prompts_than_it_goes_through(built):
    assert call_prompt(batch=(1 << 20) + 1) == ra.RC_ERR_UNSUPPORTED
    assert call_prompt(batch=1 << 20, n=0) == OK


def test_beam_batch_refuses_a_table_past_32_bits(built):
    """Latent rows have no shared segments, so that every beam's row names its whole prompt."""
    eng = SimpleNamespace(shape=SimpleNamespace(mla=True), torch=torch)
    n = 2 ** 31 // 32 - 4     # (slots without memory of their own)
    r = SimpleNamespace(rid=0, prompt_len=n, slots=np.broadcast_to(np.int32(0), (n + 32 * 4,)))
    with pytest.raises(ValueError, match="1 x 32 rows"):
        BeamBatch(eng, [r], 32, 4)
