"""Oracle of the 4-bit KV pool and of the position rotation: test infrastructure.

Only ``tests/``, ``__graft_entry__.smoke()`` and ``bench.py``'s CPU-baseline
leg may import this module; it shares no code with the product library.

4-bit pool.  A (slot, head) row of d values is d/16 blocks of 16.  A block's
scale is an unsigned 8-bit float E (5 bits, bias 15), M (3 bits):
(1 + M/8) 2^(E-15), or M/8 2^-14 at E = 0; byte 0xff is a NaN.  An element is
an E2M1 code (sign, 2 exponent bits of bias 1, 1 mantissa bit: 0, 0.5, 1, 1.5,
2, 3, 4, 6) times its block's scale.  Quantisation: raw = amax / 6 (fp32
division rounded to nearest), at most 10240; scale = nearest scale value, ties
to the even byte; code = nearest E2M1 value of x / scale (fp32 division rounded
to nearest), ties to the even code, saturating at 6, keeping the sign; a scale
of 0 has zero codes; a block with an infinity or a NaN has scale byte 0xff and
zero codes.

Rotation.  Pairs (a, b) -> (a cos - b sin, b cos + a sin), each product and sum
rounded once in fp32 (``rotate``), or in 64 bits (``rotate64``).

Parity status: pinned by tests/test_fp4_oracle.py -- the formats' values
against f16 bit patterns, brute-force nearest-value search, the error bound, and
the rotation against complex multiplication.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MAX_SCALE = 10240.0


def scale_table() -> np.ndarray:
    """Value of every scale byte 0..255 (NaN and infinity as an f16 reads them), float64."""
    out = np.empty(256, np.float64)
    for b in range(256):
        e, m = b >> 3, b & 7
        if e == 31:
            out[b] = np.inf if m == 0 else np.nan
        elif e == 0:
            out[b] = m / 8 * 2.0 ** -14
        else:
            out[b] = (1 + m / 8) * 2.0 ** (e - 15)
    return out


def _nearest(values: np.ndarray, x: np.ndarray) -> np.ndarray:
    """Index of the nearest of ascending `values` to each x >= 0, ties to the even index."""
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo = hi - 1
    dl, dh = x - values[lo], values[hi] - x
    return np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))


def quantize(x) -> tuple:
    """fp32 rows [..., d] -> (codes uint8 [..., d/2], scale bytes uint8 [..., d/16])."""
    x = np.asarray(x, np.float32)
    b = x.reshape(*x.shape[:-1], -1, 16)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], np.float32(0), b)
    raw = np.minimum(np.abs(b).max(-1) / np.float32(6), np.float32(MAX_SCALE)).astype(np.float32)
    table = scale_table()[:248]
    byte = _nearest(table, raw.astype(np.float64))
    s = table[byte].astype(np.float32)
    safe = np.where(s > 0, s, np.float32(1))
    q = np.where(s[..., None] > 0, (b / safe[..., None]).astype(np.float32), np.float32(0))
    code = _nearest(E2M1, np.minimum(np.abs(q).astype(np.float64), 6.0)) | (np.signbit(q).astype(np.int64) << 3)
    code = np.where((s > 0)[..., None], code, 0).reshape(x.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), np.where(bad, 255, byte).astype(np.uint8)


def dequantize(codes, scales) -> np.ndarray:
    """Values (float64) of codes [..., d/2] under scale bytes [..., d/16]."""
    c = np.asarray(codes, np.uint8)
    c = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1)
    v = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    with np.errstate(invalid="ignore"):
        return v * np.repeat(scale_table()[np.asarray(scales, np.uint8)], 16, axis=-1)


def _pairs(dim: int, rot: int, offset: int, interleaved: bool):
    j = np.arange(rot // 2)
    return (offset + 2 * j, offset + 2 * j + 1) if interleaved else (offset + j, offset + j + rot // 2)


def rotate(x, cos_sin, positions, offset: int, interleaved: bool) -> np.ndarray:
    """fp32 rows [n, heads, d] turned by their positions' angles, one rounding per operation."""
    y = np.array(x, np.float32)
    rot = cos_sin.shape[1]
    t = np.asarray(cos_sin, np.float32)[np.asarray(positions)]
    c, s = t[:, None, :rot // 2], t[:, None, rot // 2:]
    ia, ib = _pairs(y.shape[-1], rot, offset, interleaved)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
    y[..., ib] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return y


def rotate64(x, cos_sin, positions, offset: int, interleaved: bool) -> np.ndarray:
    """The same from the definition in 64 bits."""
    y = np.array(x, np.float64)
    rot = cos_sin.shape[1]
    t = np.asarray(cos_sin, np.float64)[np.asarray(positions)]
    ia, ib = _pairs(y.shape[-1], rot, offset, interleaved)
    z = (y[..., ia] + 1j * y[..., ib]) * (t[:, None, :rot // 2] + 1j * t[:, None, rot // 2:])
    y[..., ia], y[..., ib] = z.real, z.imag
    return y


def bf16_round(x) -> np.ndarray:
    """uint16 bits of fp32 values rounded to bf16 (nearest, ties to even; finite)."""
    u = np.asarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def attention(q, k, v, tok_of_row, q_heads, kv_heads, scale, lim=None):
    """Exact attention in double.  q [rows, Hq, D] values; k, v [tokens, Hkv, D]
    values, row r seeing tokens tok_of_row[r] (an index array; the first lim[r]
    of it).  A row without keys gives zeros and -inf.  Returns (out, lse, A), A the
    attention over |V|."""
    g = q_heads // kv_heads
    rows, D = q.shape[0], q.shape[2]
    out, a_abs = np.zeros((rows, q_heads, D)), np.zeros((rows, q_heads, D))
    lse = np.full((rows, q_heads), -np.inf)
    for r in range(rows):
        idx = tok_of_row[r] if lim is None else tok_of_row[r][:lim[r]]
        if len(idx) == 0:
            continue
        for h in range(kv_heads):
            s = (q[r, h * g:(h + 1) * g] @ k[idx, h].T) * scale
            m = s.max(-1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(-1, keepdims=True)
            out[r, h * g:(h + 1) * g] = (p / l) @ v[idx, h]
            a_abs[r, h * g:(h + 1) * g] = (p / l) @ np.abs(v[idx, h])
            lse[r, h * g:(h + 1) * g] = (m + np.log(l))[:, 0]
    return out, lse, a_abs
