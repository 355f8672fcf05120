"""A workspace sized for the largest max_len serves every smaller one (CPU: the
queries alone), as attn_decode_steps and the engine's decode loop need."""
from __future__ import annotations

import pytest
import torch

import radixattention_prefix_shared_tree_gb300 as ra

BF = torch.bfloat16
BOUNDS = sorted({m + d for m in (0, 32, 64, 96, 128, 192, 256, 320, 384, 512, 640, 1024, 1500, 2048, 4096, 5119)
                 for d in (-1, 0, 1) if m + d > 0} | set(range(7, 6000, 119)) | {40_000, 131_071})


def attn_desc(fmt, hq, hkv, d):
    z = lambda *s, t=torch.uint8: torch.zeros(*s, dtype=t)
    if fmt == "latent":
        pool = ra.make_pool_desc(z(4, 576, t=BF), None, mla=True, head_dim_v=512)
    elif fmt == "bf16":
        pool = ra.make_pool_desc(z(4, hkv, d, t=BF), z(4, hkv, d, t=BF))
    elif fmt == "fp8":
        pool = ra.make_pool_desc(z(4, hkv, d), z(4, hkv, d), k_scale=z(4, hkv, t=torch.float32),
                                 v_scale=z(4, hkv, t=torch.float32))
    else:
        pool = ra.make_pool_desc(z(4, hkv, d // 2), z(4, hkv, d // 2), k_bscale=z(4, hkv, d // 16),
                                 v_bscale=z(4, hkv, d // 16))
    return ra.make_attn_desc(pool, hq, 0.1)


def assert_never_falls(size_of):
    sizes = [size_of(m) for m in BOUNDS]
    fell = [(a, b, x, y) for a, b, x, y in zip(BOUNDS, BOUNDS[1:], sizes, sizes[1:]) if y < x]
    assert not fell, fell[:5]


LAYOUTS = [("bf16", 32, 8, 128), ("bf16", 4, 4, 64), ("bf16", 8, 1, 128), ("fp8", 32, 8, 128), ("fp4", 32, 8, 128),
           ("fp4", 8, 2, 64)]


@pytest.mark.parametrize("fmt,hq,hkv,d", LAYOUTS + [("latent", 128, 1, 576), ("latent", 16, 1, 576)])
@pytest.mark.parametrize("batch", [1, 3, 7, 40, 64, 100, 151, 256, 1000])
def test_decode(built, fmt, hq, hkv, d, batch):
    desc = attn_desc(fmt, hq, hkv, d)
    assert_never_falls(lambda m: ra.attn_decode_workspace(desc, batch, m))
    if fmt != "latent":
        casc = ra.rc_cascade(n_seg=2, max_seg_len=700, max_seg_rows=batch, total_seg_rows=batch + 1)
        assert_never_falls(lambda m: ra.attn_decode_workspace(desc, batch, m, casc))


def test_decode_across_the_boundaries_of_a_chunk(built):
    """64 rows need more at 256 keys than their exact plan at 257 holds, 40 rows at 384 than at 385."""
    desc = attn_desc("bf16", 32, 8, 128)
    for batch, a in ((64, 256), (40, 384)):
        assert ra.attn_decode_workspace(desc, batch, a + 1) >= ra.attn_decode_workspace(desc, batch, a)


@pytest.mark.parametrize("fmt,hq,hkv,d", LAYOUTS)
@pytest.mark.parametrize("batch,max_q", [(1, 1), (1, 16), (3, 2), (8, 1), (8, 3), (16, 100), (40, 1), (300, 2)])
def test_cross_and_extend(built, fmt, hq, hkv, d, batch, max_q):
    desc = attn_desc(fmt, hq, hkv, d)
    assert_never_falls(lambda m: ra.attn_cross_workspace(desc, batch, max_q, m))
    assert_never_falls(lambda m: ra.attn_extend_workspace(desc, batch, max_q, m))
