"""Cases of the operators around the KV pool: appending rotated keys and values
(``kv_store_rope``), attention over a pool held in 4 bits (``attn_decode`` and
``attn_extend`` on it) and cross attention to an encoder's states in the pool
(``attn_cross``).

``run`` computes them from elementary torch operations in 32 bits, or, where
``own`` is true, through the package's entry points.

The 4-bit pool: each (slot, head) row of d values is d/16 blocks of 16; a
block holds one scale byte (5 exponent bits of bias 15 and 3 mantissa bits, no
sign: bits 14..7 of an f16) and 16 E2M1 codes, two per byte, the even element
in the low half.  A value is its code times its block's scale.
"""
import math

import numpy as np
import torch

own = False

RUN = 64        # slots of a row lie in runs of this many, as an allocator hands them out


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one request decoding alone: the append of its one token, all launch latency
        dict(name="append 1 token bf16", op="append", pool="bf16", hq=32, hkv=8, d=128, rot=128, inter=False,
             n=1, max_pos=8192, strided=True),
        # one decode step of a full batch into an E4M3 pool
        dict(name="append 256 tokens fp8", op="append", pool="fp8", hq=32, hkv=8, d=128, rot=128, inter=False,
             n=256, max_pos=8192, strided=True),
        # the prefill of a few-shot batch: 256 questions of 32..64 tokens and the shared examples
        dict(name="append 14001 tokens bf16", op="append", pool="bf16", hq=32, hkv=8, d=128, rot=64, inter=True,
             n=14001, max_pos=8192, strided=True),
        # latent rows: the last 64 of 576 columns are rotated, for the row and for 128 query heads
        dict(name="append 1023 latent rows", op="append", pool="latent", hq=128, hkv=1, d=576, rot=64, inter=True,
             n=1023, max_pos=32768, strided=False),
        # one request decoding over its own context
        dict(name="decode 1 x 4097 fp4", op="decode", pool="fp4", hq=32, hkv=8, d=128, batch=1, lo=4097, hi=4097,
             shared=0),
        # chat: a full decode batch whose contexts have grown to between 500 and 5,000 tokens
        dict(name="decode 256 x 512-5119 fp4", op="decode", pool="fp4", hq=32, hkv=8, d=128, batch=256, lo=512,
             hi=5119, shared=0),
        # agent tree: one whole decode step (append with rotation, then attention with the shared root as a segment)
        dict(name="step 64 agents fp4", op="step", pool="fp4", hq=64, hkv=8, d=128, rot=128, inter=False, batch=64,
             lo=2817, hi=3071, shared=2048, max_pos=8192),
        # a few long documents
        dict(name="decode 3 x 100k fp4", op="decode", pool="fp4", hq=32, hkv=8, d=128, batch=3, lo=65537, hi=131071,
             shared=0),
        # few-shot prefill: 256 questions over 1,792 shared tokens
        dict(name="extend 256 x 1792+32-64 fp4", op="extend", pool="fp4", hq=32, hkv=8, d=128, batch=256, lo=32, hi=64,
             prefix=1792, shared=1792),
        # decoding over an encoder's 1,500 states, a head for each
        dict(name="cross 32 x 1 x 1500 bf16", op="cross", pool="bf16", hq=16, hkv=16, d=64, batch=32, lo=1, hi=1,
             keys_lo=1500, keys_hi=1500),
        # prompts over an encoder's states of ragged lengths
        dict(name="cross 16 x 100-448 x 375-1500 bf16", op="cross", pool="bf16", hq=16, hkv=8, d=128, batch=16, lo=100,
             hi=448, keys_lo=375, keys_hi=1500),
        # long prompts over image tokens that the pool holds in 4 bits
        dict(name="cross 6 x 900-1024 x 4095 fp4", op="cross", pool="fp4", hq=32, hkv=8, d=128, batch=6, lo=900, hi=1024,
             keys_lo=4095, keys_hi=4095),
    ]


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "decode", "decode", "step", "extend", "cross", "cross"])
    hq, hkv = rng.choice([(32, 8), (64, 8), (16, 8), (8, 8), (16, 16), (32, 16)])
    d = rng.choice([64, 128, 128])
    if op == "append":
        pool = rng.choice(["bf16", "bf16", "fp8", "latent"])
        if pool == "latent":
            return dict(op=op, pool=pool, hq=rng.choice([16, 128]), hkv=1, d=576, rot=64, inter=rng.random() < 0.5,
                        n=_log_int(rng, 1, 1500), max_pos=32768, strided=rng.random() < 0.5)
        d = 128 if pool == "fp8" else d
        return dict(op=op, pool=pool, hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d // 2]), inter=rng.random() < 0.4,
                    n=_log_int(rng, 1, 12000), max_pos=8192, strided=rng.random() < 0.5)
    if op in ("decode", "step"):
        batch = _log_int(rng, 1, 256)
        hi = _log_int(rng, 1, min(131071, max(64, 600000 // batch)))
        lo = rng.randint(1, hi)
        c = dict(op=op, pool="fp4", hq=hq, hkv=hkv, d=d, batch=batch, lo=lo, hi=hi, shared=0)
        if op == "step":
            c.update(rot=rng.choice([d, d // 2]), inter=rng.random() < 0.4, max_pos=hi + 1)
            c["shared"] = lo // 2 if rng.random() < 0.5 else 0
        return c
    pool = "fp4" if op == "extend" else rng.choice(["bf16", "bf16", "fp8", "fp4"])
    d = 128 if pool == "fp8" else d
    batch, hi = _log_int(rng, 1, 64), _log_int(rng, 1, 1500)
    lo = rng.randint(max(1, hi // 4), hi)
    if op == "extend":
        prefix = _log_int(rng, 1, 6000)
        c = dict(op=op, pool=pool, hq=hq, hkv=hkv, d=d, batch=batch, lo=lo, hi=hi, prefix=prefix,
                 shared=prefix if rng.random() < 0.5 else 0)
    else:
        keys = _log_int(rng, 1, 6000)
        c = dict(op=op, pool=pool, hq=hq, hkv=hkv, d=d, batch=batch, lo=lo, hi=hi,
                 keys_lo=rng.randint(max(1, keys // 3), keys), keys_hi=keys)
    most = min(_cost(x) for x in listed() if x["name"].startswith(("extend", "cross 6")))
    while c["batch"] > 1 and _cost(c) > 0.8 * most:
        c["batch"] = (c["batch"] + 1) // 2
    return c


def _spread(n, lo, hi):
    """n whole numbers over lo..hi, the same for every seed."""
    return [lo + ((i * 2654435761 + 12345) % (1 << 32)) * (hi - lo + 1) // (1 << 32) for i in range(n)]


def _lengths(case):
    """Query tokens and keys of each row."""
    b = case["batch"]
    if case["op"] in ("decode", "step"):
        return [1] * b, _spread(b, case["lo"], case["hi"])
    new = _spread(b, case["lo"], case["hi"])
    if case["op"] == "extend":
        return new, [case["prefix"] + x for x in new]
    return new, _spread(b, case["keys_lo"], case["keys_hi"])


def _row_bytes(pool, d):
    """Bytes that one head's row of d values takes in the pool."""
    return {"bf16": 2 * d, "latent": 2 * d, "fp8": d + 4, "fp4": d // 2 + d // 16}[pool]


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    arrays = 1 if case["pool"] == "latent" else 2
    store = lambda n: n * (arrays * hkv * (2 * d + _row_bytes(case["pool"], d)) + hq * 4 * d + 4 * case["rot"] + 8)  # noqa: E731
    rotate = lambda n: 3 * n * (hq + hkv) * case["rot"]  # noqa: E731
    if case["op"] == "append":
        return {"bytes": store(case["n"]), "flops": rotate(case["n"])}
    new, keys = _lengths(case)
    shared = case.get("shared", 0)
    unique = sum(keys) - shared * (len(keys) - 1)
    if case["op"] == "extend":
        pairs = sum(n * (k - n) + n * (n + 1) // 2 for n, k in zip(new, keys))
    else:
        pairs = sum(n * k for n, k in zip(new, keys))
    out = {"bytes": unique * hkv * arrays * _row_bytes(case["pool"], d) + 4 * sum(keys) + sum(new) * hq * (4 * d + 4),
           "flops": 4 * d * hq * pairs}
    if case["op"] == "step":
        out["bytes"] += store(case["batch"]) - case["batch"] * hq * 2 * d
        out["flops"] += rotate(case["batch"])
    return out


# ------------------------------------------------------------------ the inputs
def _to_blocks(x):
    """Codes and scale bytes of rows [..., d] for the 4-bit pool."""
    x = x.float()
    blocks = x.unflatten(-1, (-1, 16))
    raw = (blocks.abs().amax(-1) / 6.0).clamp(max=10240.0)
    exponent = torch.frexp(raw)[1] - 1
    quantum = torch.ldexp(torch.ones_like(raw), exponent.clamp(min=-14) - 3)
    scale = torch.round(raw / quantum) * quantum
    q = torch.where(scale[..., None] > 0, blocks / scale[..., None], torch.zeros_like(blocks))
    a = q.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code.to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)
    code = code.flatten(-2)
    byte = (scale.half().view(torch.int16) >> 7).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte


def _from_blocks(codes, scales):
    """Values (fp32) of rows held as codes and scale bytes."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    m = (c & 7).float()
    v = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))     # 0 .5 1 1.5 2 3 4 6
    v = torch.where(c > 7, -v, v)
    s = (scales.to(torch.int16) << 7).view(torch.float16).float()
    return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _to_e4m3(x):
    """Codes (as float8) and scales of rows [..., 128] for the E4M3 pool."""
    x = x.float()
    scale = x.abs().amax(-1) / 448.0
    q = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
    return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _angles(max_pos, rot, dev):
    """cos | sin of every position, from 64-bit angles."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], -1).float().contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev, dtype=torch.float32)  # noqa: E731
    hq, hkv, d, pool = case["hq"], case["hkv"], case["d"], case["pool"]
    gain = torch.exp(0.3 * rnd(hkv, d))     # some channels of the keys are larger than others
    s = {"case": case, "err": torch.zeros(1, dtype=torch.int32, device=dev)}

    def new_rows(n):
        """K, V and Q of n new tokens: slices of one projection's output, or arrays of their own."""
        vd = 0 if pool == "latent" else d
        if case.get("strided", True):
            fused = torch.cat([rnd(n, hq, d).flatten(1), (rnd(n, hkv, d) * gain).flatten(1), rnd(n, hkv * vd)], 1)
            fused = fused.to(torch.bfloat16)
            q, k, v = fused.split([hq * d, hkv * d, hkv * vd], 1)
        else:
            q, k, v = rnd(n, hq * d).bfloat16(), (rnd(n, hkv, d) * gain).flatten(1).bfloat16(), rnd(n, hkv * vd).bfloat16()
        s["q"], s["k_new"] = q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d))
        s["v_new"] = v.unflatten(1, (hkv, d)) if vd else None
        s["q_out"] = torch.zeros(n, hq, d, dtype=torch.bfloat16, device=dev)
        s["table"] = _angles(case["max_pos"], case["rot"], dev)

    def fill(n_slots):
        """The pool, every slot in use."""
        k = (rnd(n_slots, hkv, d) * gain).bfloat16()
        v = rnd(n_slots, hkv, d).bfloat16() if pool != "latent" else None
        if pool == "fp4":
            (s["k"], s["k_bscale"]), (s["v"], s["v_bscale"]) = _to_blocks(k), _to_blocks(v)
        elif pool == "fp8":
            (s["k"], s["k_scale"]), (s["v"], s["v_scale"]) = _to_e4m3(k), _to_e4m3(v)
        elif pool == "latent":
            s["k"], s["v"] = k.reshape(n_slots, d), None
        else:
            s["k"], s["v"] = k, v

    if case["op"] == "append":
        n = case["n"]
        n_slots = n + n // 8 + 17
        new_rows(n)
        fill(n_slots)
        s["slots"] = torch.randperm(n_slots, generator=gen, device=dev)[:n].int()
        s["positions"] = torch.randint(0, case["max_pos"], (n,), generator=gen, device=dev).int()
        return s

    new, keys = _lengths(case)
    shared = case.get("shared", 0)
    runs = [-(-(k - shared) // RUN) for k in keys]
    first = -(-shared // RUN)
    n_runs = first + sum(runs)
    place = torch.randperm(n_runs, generator=gen, device=dev)
    slots = (place[:, None] * RUN + torch.arange(RUN, device=dev)).flatten()
    fill(n_runs * RUN)
    # the slot table: row b's keys are slots[start[b] : start[b] + len[b]], the shared ones first
    rows, at = [], first * RUN
    for k, r in zip(keys, runs):
        rows.append(torch.cat([slots[:shared], slots[at:at + k - shared]]))
        at += r * RUN
    starts = np.concatenate([[0], np.cumsum(keys)[:-1]]).astype(np.int32)
    to = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)  # noqa: E731
    s["rows"] = torch.cat(rows).int()
    s["start"], s["len"], s["max_len"] = to(starts), to(keys), max(keys)
    s["qo"], s["max_q"] = to(np.concatenate([[0], np.cumsum(new)])), max(new)
    total = sum(new)
    if case["op"] == "step":
        new_rows(total)
        s["positions"] = s["len"] - 1
        s["slots"] = torch.stack([r[-1] for r in rows]).int()
        if shared:      # the shared root is one segment of the cascade, read once for all rows
            s["seg"] = dict(slots=slots[:shared].int().contiguous(), indptr=to([0, shared]), row_indptr=to([0, total]),
                            rows=to(np.arange(total)), req_indptr=to(np.arange(total + 1)), req_pos=to(np.arange(total)))
            s["own_start"], s["own_len"] = s["start"] + shared, s["len"] - shared
    else:
        s["q"] = rnd(total, hq, d).bfloat16()
    s["out"] = torch.zeros(total, hq, d, dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.zeros(total, hq, dtype=torch.float32, device=dev)
    return s


# -------------------------------------------------------------- the plain form
def _rotated(x, table, positions, offset, rot, inter):
    """Rows [n, heads, d] with columns offset..offset+rot turned by their positions' angles, fp32."""
    x = x.float()
    c, sn = (t[:, None, :] for t in table[positions.long()].split(rot // 2, -1))
    part = x[..., offset:offset + rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if inter else part.split(rot // 2, -1)
    ya, yb = a * c - b * sn, b * c + a * sn
    part = torch.stack([ya, yb], -1).flatten(-2) if inter else torch.cat([ya, yb], -1)
    return torch.cat([x[..., :offset], part, x[..., offset + rot:]], -1)


def _append_plain(s):
    case = s["case"]
    pool, rot = case["pool"], case["rot"]
    offset = case["d"] - rot if pool == "latent" else 0
    k = _rotated(s["k_new"], s["table"], s["positions"], offset, rot, case["inter"])
    s["q_out"].copy_(_rotated(s["q"], s["table"], s["positions"], offset, rot, case["inter"]))
    at = s["slots"].long()
    if pool == "latent":
        s["k"][at] = k[:, 0].bfloat16()
    elif pool == "bf16":
        s["k"][at] = k.bfloat16()
        s["v"][at] = s["v_new"]
    elif pool == "fp8":
        for name, x in (("k", k), ("v", s["v_new"])):
            codes, scales = _to_e4m3(x)
            s[name].view(torch.uint8)[at] = codes.view(torch.uint8)
            s[name + "_scale"][at] = scales
    else:
        for name, x in (("k", k), ("v", s["v_new"])):
            s[name][at], s[name + "_bscale"][at] = _to_blocks(x)


def _values(s, name, at):
    """fp32 values of the pool's rows at the given slots."""
    pool = s["case"]["pool"]
    if pool == "fp4":
        return _from_blocks(s[name][at], s[name + "_bscale"][at])
    if pool == "fp8":
        return s[name].view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * s[name + "_scale"][at][..., None]
    return s[name][at].float()


def _attend_plain(s, q):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    dev = q.device
    b, g, lmax, nmax = len(s["len"]), hq // hkv, s["max_len"], s["max_q"]
    lens, qo = s["len"].long(), s["qo"].long()
    j = torch.arange(lmax, device=dev)
    live = j < lens[:, None]
    at = s["rows"].long()[torch.where(live, s["start"].long()[:, None] + j, 0)]
    k, v = (_values(s, n, at).transpose(1, 2) for n in ("k", "v"))                 # [b, hkv, lmax, d]
    i = torch.arange(nmax, device=dev)
    n_new = qo[1:] - qo[:-1]
    has = i < n_new[:, None]
    row = torch.where(has, qo[:-1, None] + i, 0)
    qp = q.float()[row].unflatten(2, (hkv, g)).permute(0, 2, 1, 3, 4).reshape(b, hkv, nmax * g, d)
    sc = torch.matmul(qp, k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).unflatten(2, (nmax, g))
    seen = live[:, None, :]
    if case["op"] == "extend":
        seen = seen & (j < (lens - n_new)[:, None, None] + i[:, None] + 1)
    sc.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (nmax, g)) / torch.where(l > 0, l, 1.0)
    lse = torch.where(l > 0, m + l.log(), -math.inf)[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(b, nmax, hq, d)
    lse = lse.permute(0, 2, 1, 3).reshape(b, nmax, hq)
    tok = torch.arange(len(q), device=dev)
    of = torch.searchsorted(qo[1:], tok, right=True)
    s["out"].copy_(o[of, tok - qo[of]])
    s["lse"].copy_(lse[of, tok - qo[of]])


# ------------------------------------------------------- the framework's calls
def _plan(s):
    """Descriptors and workspace of a state's buffers, made once."""
    import radixattention_prefix_shared_tree_gb300 as ra
    case = s["case"]
    p = {"ra": ra}
    raw = lambda t: t.view(torch.uint8) if t is not None and t.dtype == torch.float8_e4m3fn else t  # noqa: E731
    pool = ra.make_pool_desc(raw(s["k"]), raw(s["v"]), s["err"], mla=case["pool"] == "latent", head_dim_v=512,
                             k_scale=s.get("k_scale"), v_scale=s.get("v_scale"), k_bscale=s.get("k_bscale"),
                             v_bscale=s.get("v_bscale"))
    p["pool"] = pool
    if "table" in s:
        p["rope"] = ra.make_rope_desc(s["table"], interleaved=case["inter"],
                                      offset=case["d"] - case["rot"] if case["pool"] == "latent" else 0)
    if case["op"] == "append":
        return p
    b = case["batch"]
    p["desc"] = ra.make_attn_desc(pool, case["hq"], 1.0 / math.sqrt(case["d"]))
    p["casc"] = None
    start, length, max_len = s["start"], s["len"], s["max_len"]
    if "seg" in s:
        g, shared = s["seg"], case["shared"]
        p["casc"] = ra.make_cascade(g["slots"], g["indptr"], g["row_indptr"], g["rows"], g["req_indptr"], g["req_pos"],
                                    max_seg_rows=b, max_seg_len=shared, host_seg_indptr=np.array([0, shared]),
                                    host_seg_row_indptr=np.array([0, b]))
        start, length, max_len = s["own_start"], s["own_len"], s["max_len"] - shared
    p["kv"] = ra.make_kv_table(s["rows"], start, length, max_len)
    if case["op"] in ("decode", "step"):
        size = ra.attn_decode_workspace(p["desc"], b, max_len, p["casc"])
    elif case["op"] == "extend":
        size = ra.attn_extend_workspace(p["desc"], b, s["max_q"], max_len)
    else:
        size = ra.attn_cross_workspace(p["desc"], b, s["max_q"], max_len)
    p["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device=s["out"].device)
    return p


def _run_own(s):
    if "plan" not in s:
        s["plan"] = _plan(s)
    p, case = s["plan"], s["case"]
    ra, op = p["ra"], case["op"]
    if op in ("append", "step"):
        ra.kv_store_rope(p["pool"], p["rope"], s["slots"], s["positions"], s["k_new"], s["v_new"], s["q"], s["q_out"])
    if op == "step":
        ra.attn_decode(p["desc"], s["q_out"], p["kv"], case["batch"], s["out"], s["lse"], p["ws"], cascade=p["casc"])
    elif op == "decode":
        ra.attn_decode(p["desc"], s["q"], p["kv"], case["batch"], s["out"], s["lse"], p["ws"])
    elif op == "extend":
        ra.attn_extend(p["desc"], s["q"], s["qo"], p["kv"], case["batch"], s["max_q"], s["out"], s["lse"], p["ws"])
    elif op == "cross":
        ra.attn_cross(p["desc"], s["q"], s["qo"], p["kv"], case["batch"], s["max_q"], s["out"], s["lse"], p["ws"])


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        _run_own(s)
    else:
        if op in ("append", "step"):
            _append_plain(s)
        if op != "append":
            _attend_plain(s, s["q_out"] if op == "step" else s["q"])
    if op == "append":
        out = [s["q_out"], s["k"]] + ([s["v"]] if s["v"] is not None else [])
        return out + ([s["k_scale"], s["v_scale"]] if "k_scale" in s else [])
    return [s["out"], s["lse"]] + ([s["q_out"]] if op == "step" else [])


# ------------------------------------------------------- the definition, 64 bits
def _turn64(x, table, positions, offset, inter):
    """Each pair (a, b) as the complex number a + ib times cos + i sin."""
    x = x.double().clone()
    half = table.shape[1] // 2
    t = table.double()[positions.long()]
    w = torch.complex(t[:, :half], t[:, half:])[:, None, :]
    ia = offset + (torch.arange(half, device=x.device) * 2 if inter else torch.arange(half, device=x.device))
    ib = ia + (1 if inter else half)
    z = torch.complex(x[..., ia], x[..., ib]) * w
    x[..., ia], x[..., ib] = z.real, z.imag
    return x


def _value64(codes, scales):
    """E2M1 codes by their fields (2 exponent bits of bias 1, 1 mantissa bit) times 2^(E - 15) (1 + M / 8)."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    e, m = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).double()))
    mag = torch.where(c >= 8, -mag, mag)
    se, sm = (scales.long() >> 3), (scales.long() & 7).double() / 8
    sv = torch.where(se == 0, sm * 2.0 ** -14, (1 + sm) * torch.exp2((se - 15).double()))
    return mag * sv.repeat_interleave(16, -1)


def _nearest64(x):
    """Rows [..., d] as the 4-bit pool holds them: every value against the list of all that its block's scale allows."""
    b = x.reshape(*x.shape[:-1], -1, 16)
    grid = [m / 8 * 2.0 ** -14 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-14, 14) for m in range(8)]
    grid = [g for g in grid if g <= 10240.0]
    grid = grid[0::2] + grid[1::2]      # of two as near the even one, which the search meets first
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    sc = grid[(b.abs().amax(-1, keepdim=True) / 6 - grid).abs().argmin(-1)][..., None]
    lev = torch.tensor([0.0, 1.0, 2.0, 4.0, 0.5, 1.5, 3.0, 6.0], dtype=torch.float64, device=x.device)
    near = lev[(b.abs()[..., None] - sc[..., None] * lev).abs().argmin(-1)]
    return (near * sc * b.sign()).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op, pool = case["op"], case["pool"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    offset = d - case["rot"] if pool == "latent" else 0
    if op in ("append", "step"):
        k_rot = _turn64(s["k_new"], s["table"], s["positions"], offset, case["inter"])
        q_rot = _turn64(s["q"], s["table"], s["positions"], offset, case["inter"])
    if op == "append":
        at = s["slots"].long()
        if pool == "fp8":
            out = [q_rot, s["k"].double(), s["v"].double(), s["k_scale"].double(), s["v_scale"].double()]
            for j, x in ((1, k_rot), (2, s["v_new"].double())):
                sc = x.abs().amax(-1) / 448
                # the code's place between powers of two: 8 steps in each, down to 2^-6
                y = x / sc[..., None]
                step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                out[j][at] = torch.round(y / step) * step
                out[j + 2][at] = sc
            return out
        k = s["k"].double()
        k[at] = k_rot[:, 0] if pool == "latent" else k_rot
        if pool == "latent":
            return [q_rot, k]
        v = s["v"].double()
        v[at] = s["v_new"].double()
        return [q_rot, k, v]
    if pool == "fp4":
        k, v = _value64(s["k"], s["k_bscale"]), _value64(s["v"], s["v_bscale"])
    elif pool == "fp8":
        k, v = (s[n].double() * s[n + "_scale"].double()[..., None] for n in ("k", "v"))
    else:
        k, v = s["k"].double(), s["v"].double()
    q = s["q"].double()
    if op == "step":
        k[s["slots"].long()] = _nearest64(k_rot)
        v[s["slots"].long()] = _nearest64(s["v_new"].double())
        q = q_rot.bfloat16().double()       # the attention reads the rotated queries as they are held
    new, keys = _lengths(case)
    starts, qo = s["start"].tolist(), s["qo"].tolist()
    out = torch.empty(qo[-1], hq, d, dtype=torch.float64, device=q.device)
    lse = torch.empty(qo[-1], hq, dtype=torch.float64, device=q.device)
    for b, (n, length) in enumerate(zip(new, keys)):
        at = s["rows"][starts[b]:starts[b] + length].long()
        kb, vb = k[at], v[at]
        for h in range(hkv):
            g = slice(h * hq // hkv, (h + 1) * hq // hkv)
            sc = torch.einsum("nge,le->ngl", q[qo[b]:qo[b] + n, g], kb[:, h]) / math.sqrt(d)
            if op == "extend":
                at_pos = length - n + torch.arange(n, device=q.device)
                sc = sc + torch.where(torch.arange(length, device=q.device) > at_pos[:, None], -math.inf, 0.0)[:, None]
            t = torch.logsumexp(sc, -1)
            out[qo[b]:qo[b] + n, g] = torch.einsum("ngl,le->nge", torch.exp(sc - t[..., None]), vb[:, h])
            lse[qo[b]:qo[b] + n, g] = t
    return [out, lse] + ([q_rot] if op == "step" else [])
