"""Cases of the operators for a prompt's way through the pool and its answer:
attention over whole prompts (``attn_prompt``), appending with positions on
several axes (``kv_store_rope``), reading the pool back (``kv_load``), and beam
search (``beam_select``, ``beam_reorder``).

``run`` computes them from elementary torch operations in 32 bits (the beams'
scores in 64, since near scores decide what is chosen), or, where ``own`` is
true, through the package's entry points.

The 4-bit pool: each (slot, head) row of d values is d/16 blocks of 16; a block
holds one scale byte (bits 14..7 of an f16) and 16 E2M1 codes, two per byte, the
even element in the low half.  A value is its code times its block's scale.
"""
import math

import torch

own = False


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one short prompt of the smallest head layout: all launch latency
        dict(name="prompt 1 x 41 (4/4, 64)", op="prompt", hq=4, hkv=4, d=64, batch=1, lo=41, hi=41, strided=False),
        # the first turns of a full chat batch: nothing of them is cached yet
        dict(name="prompt 256 x 128-512", op="prompt", hq=32, hkv=8, d=128, batch=256, lo=128, hi=512, strided=True),
        # the root prompt of an agent tree, alone
        dict(name="prompt 1 x 2049 (64/8)", op="prompt", hq=64, hkv=8, d=128, batch=1, lo=2049, hi=2049, strided=True),
        # mid-sized prompts of a head for each, odd lengths
        dict(name="prompt 12 x 375-1500 (16/16, 64)", op="prompt", hq=16, hkv=16, d=64, batch=12, lo=375, hi=1500,
             strided=False),
        # a few long documents
        dict(name="prompt 3 x 9000-14000", op="prompt", hq=32, hkv=8, d=128, batch=3, lo=9000, hi=14000, strided=True),
        # one request decoding after an image: its one token, with a position on each of three axes
        dict(name="append 1 token, 3 axes", op="append", pool="bf16", hq=32, hkv=8, d=128, rot=128, inter=False, axes=3,
             spread=False, n=1, strided=True),
        # a batch of prompts, images and text, into a 4-bit pool, the axes taking turns over the pairs
        dict(name="append 9001 tokens, 3 axes fp4", op="append", pool="fp4", hq=32, hkv=8, d=128, rot=128, inter=False,
             axes=3, spread=True, n=9001, strided=True),
        # a cached prefix out of an E4M3 pool
        dict(name="load 1792 tokens fp8", op="load", pool="fp8", hkv=8, d=128, n=1792, strided=False),
        # long contexts leaving a 4-bit pool (for another pool, or another device)
        dict(name="load 60001 tokens fp4", op="load", pool="fp4", hkv=8, d=128, n=60001, strided=True),
        # one request with four beams
        dict(name="select 1 x 4 x 32000 bf16", op="select", batch=1, beams=4, vocab=32000, n_out=4, f32=False, masked=0.0,
             done=0.0, cols=0),
        # a full batch with eight beams, some finished; twice as many candidates are kept, for endings
        dict(name="select 64 x 8 x 32000 fp32", op="select", batch=64, beams=8, vocab=32000, n_out=16, f32=True,
             masked=0.0, done=0.1, cols=0),
        # one whole beam step with most of an odd vocabulary masked (a grammar): selection, then the slot rows and the
        # token histories follow their parents
        dict(name="step 200 x 4 x 32003, 2000 back", op="select", batch=200, beams=4, vocab=32003, n_out=4, f32=False,
             masked=0.9, done=0.1, cols=2000),
    ]


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "append", "load", "select", "select"])
    d = rng.choice([64, 128, 128])
    if op == "prompt":
        hq, hkv = rng.choice([(32, 8), (64, 8), (16, 16), (4, 4), (8, 1), (12, 4), (28, 4), (32, 2)])
        batch, hi = _log_int(rng, 1, 256), _log_int(rng, 1, 12000)
        c = dict(op=op, hq=hq, hkv=hkv, d=d, batch=batch, lo=rng.randint(0, hi), hi=hi, strided=rng.random() < 0.5)
        most = max(_cost(x) for x in listed() if x["op"] == "prompt")
        while _cost(c) > 0.8 * most:
            if c["batch"] > 1:
                c["batch"] = (c["batch"] + 1) // 2
            else:
                c["hi"] = c["hi"] * 3 // 4
                c["lo"] = min(c["lo"], c["hi"])
        return c
    if op == "append":
        pool = rng.choice(["bf16", "fp4", "fp8"])
        hq, hkv = rng.choice([(32, 8), (64, 8), (16, 16), (8, 1)])
        d = 128 if pool == "fp8" else d
        return dict(op=op, pool=pool, hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d // 2]), inter=rng.random() < 0.4,
                    axes=rng.randint(2, 4), spread=rng.random() < 0.5, n=_log_int(rng, 1, 8000),
                    strided=rng.random() < 0.5)
    if op == "load":
        pool = rng.choice(["bf16", "fp4", "fp8", "latent"])
        hkv = 1 if pool == "latent" else rng.choice([1, 4, 8, 16])
        d = 128 if pool == "fp8" else 576 if pool == "latent" else d
        return dict(op=op, pool=pool, hkv=hkv, d=d, n=_log_int(rng, 1, 40000), strided=rng.random() < 0.5)
    beams = rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
    vocab = _log_int(rng, 100, 130000)
    batch = max(1, min(_log_int(rng, 1, 256), 20_000_000 // (beams * vocab)))
    return dict(op=op, batch=batch, beams=beams, vocab=vocab, n_out=beams * rng.choice([1, 1, 2]), f32=rng.random() < 0.5,
                masked=rng.choice([0.0, 0.0, 0.5, 0.9]), done=rng.choice([0.0, 0.2]),
                cols=_log_int(rng, 1, 2000) if rng.random() < 0.4 else 0)


def _spread(n, lo, hi):
    """n whole numbers over lo..hi, the same for every seed."""
    return [lo + ((i * 2654435761 + 12345) % (1 << 32)) * (hi - lo + 1) // (1 << 32) for i in range(n)]


def _row_bytes(pool, d):
    """Bytes that one head's row of d values takes in the pool."""
    return {"bf16": 2 * d, "latent": 2 * d, "fp8": d + 4, "fp4": d // 2 + d // 16}[pool]


def work(case):
    op = case["op"]
    if op == "prompt":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        lens = _spread(case["batch"], case["lo"], case["hi"])
        return {"bytes": sum(lens) * (2 * d * (2 * hq + 2 * hkv) + 4 * hq) + 4 * len(lens) + 4,
                "flops": 4 * d * hq * sum(n * (n + 1) // 2 for n in lens)}
    if op == "append":
        hq, hkv, d, n = case["hq"], case["hkv"], case["d"], case["n"]
        return {"bytes": n * (2 * hkv * (2 * d + _row_bytes(case["pool"], d)) + hq * 4 * d + 4 * case["rot"] +
                              4 * case["axes"] + 4), "flops": 3 * n * (hq + hkv) * case["rot"]}
    if op == "load":
        arrays = 1 if case["pool"] == "latent" else 2
        return {"bytes": case["n"] * (arrays * case["hkv"] * (2 * case["d"] + _row_bytes(case["pool"], case["d"])) + 4),
                "flops": arrays * case["n"] * case["hkv"] * case["d"]}
    rows = case["batch"] * case["beams"]
    return {"bytes": rows * (case["vocab"] * (4 if case["f32"] else 2) + 5) + 13 * case["batch"] * case["n_out"] +
            2 * 2 * 4 * rows * case["cols"], "flops": 4 * rows * case["vocab"]}


# ------------------------------------------------------------------ the inputs
def _to_blocks(x):
    """Codes and scale bytes of rows [..., d] for the 4-bit pool."""
    x = x.float()
    blocks = x.unflatten(-1, (-1, 16))
    raw = (blocks.abs().amax(-1) / 6.0).clamp(max=10240.0)
    quantum = torch.ldexp(torch.ones_like(raw), (torch.frexp(raw)[1] - 1).clamp(min=-14) - 3)
    scale = torch.round(raw / quantum) * quantum
    q = torch.where(scale[..., None] > 0, blocks / scale[..., None], torch.zeros_like(blocks))
    a = q.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code.to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)).flatten(-2)
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
    scale = x.abs().amax(-1) / torch.tensor(448.0, device=x.device)
    q = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
    return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _angles(max_pos, rot, dev):
    """cos | sin of every position, from 64-bit angles."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], -1).float().contiguous()


def _pair_axis(case):
    """Axis of every rotated pair: runs of pairs, the first axis' a little longer, or the axes in turn."""
    pairs, axes = case["rot"] // 2, case["axes"]
    if case["spread"]:
        return [j % axes for j in range(pairs)]
    each = pairs // axes
    return [0] * (pairs - each * (axes - 1)) + [a for a in range(1, axes) for _ in range(each)]


def _positions(case, gen, dev):
    """[axes, n]: text, where all axes count alike, and images of 24 x 18 patches, where the later axes count rows and
    columns (a fourth counts frames)."""
    n, axes = case["n"], case["axes"]
    i = torch.arange(n, device=dev)
    start = torch.randint(0, 4000, (1,), generator=gen, device=dev)
    image = (i // 432) % 2 == 1
    k = i % 432
    pos = (start + i)[None].repeat(axes, 1)
    base = start + i - k
    for a, own_part in ((0, 0 * k), (1, k // 18), (2, k % 18), (3, k // 216)):
        if a < axes:
            pos[a] = torch.where(image, base + own_part, pos[a])
    return pos.int().contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev, dtype=torch.float32)  # noqa: E731
    s = {"case": case, "err": torch.zeros(1, dtype=torch.int32, device=dev)}
    op = case["op"]

    def rows_in(n, hq, hkv, d, gain):
        """Q, K and V of n tokens: slices of one projection's output, or arrays of their own."""
        parts = [rnd(n, hq * d).bfloat16(), (rnd(n, hkv, d) * gain).flatten(1).bfloat16(), rnd(n, hkv * d).bfloat16()]
        if case["strided"]:
            parts = torch.cat(parts, 1).split([hq * d, hkv * d, hkv * d], 1)
        return [x.unflatten(1, (h, d)) for x, h in zip(parts, (hq, hkv, hkv))]

    def pool_rows(n_slots, hkv, d, pool, gain):
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

    if op == "prompt":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        lens = _spread(case["batch"], case["lo"], case["hi"])
        n = sum(lens)
        s["lens"], s["scale"] = lens, 1.0 / math.sqrt(d)
        s["q"], s["k"], s["v"] = rows_in(n, hq, hkv, d, torch.exp(0.3 * rnd(hkv, d)))
        s["indptr"] = torch.tensor([0] + lens, device=dev).cumsum(0).int()
        s["out"] = torch.zeros(n, hq, d, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros(n, hq, dtype=torch.float32, device=dev)
        return s
    if op in ("append", "load"):
        n, hkv, d = case["n"], case["hkv"], case["d"]
        gain = torch.exp(0.3 * rnd(hkv, d))
        n_slots = n + n // 8 + 17
        pool_rows(n_slots, hkv, d, case["pool"], gain)
        s["slots"] = torch.randperm(n_slots, generator=gen, device=dev)[:n].int()
        if op == "append":
            s["q"], s["k_new"], s["v_new"] = rows_in(n, case["hq"], hkv, d, gain)
            s["q_out"] = torch.zeros(n, case["hq"], d, dtype=torch.bfloat16, device=dev)
            s["table"] = _angles(8192 + n, case["rot"], dev)
            s["positions"] = _positions(case, gen, dev)
        else:      # both halves of one buffer, or a buffer each
            arrays = 1 if case["pool"] == "latent" else 2
            wide = torch.zeros(n, arrays if case["strided"] else 1, hkv, d, dtype=torch.bfloat16, device=dev)
            s["k_out"] = wide[:, 0]
            s["v_out"] = None if arrays == 1 else wide[:, 1] if case["strided"] else torch.zeros_like(s["k_out"])
        return s
    b, w, vocab, n_out, cols = (case[k] for k in ("batch", "beams", "vocab", "n_out", "cols"))
    x = rnd(b, w, vocab).mul_(2.5)
    likely = torch.randint(0, vocab, (b, w, 12), generator=gen, device=dev)     # a few continuations stand out
    x.scatter_add_(2, likely, 3.0 + 4.0 * torch.rand(b, w, 12, generator=gen, device=dev))
    if case["masked"]:
        gone = torch.rand(b, 1, vocab, generator=gen, device=dev) < case["masked"]
        gone[:, :, :2] = False
        x.masked_fill_(gone, -math.inf)
    s["logits"] = x if case["f32"] else x.bfloat16()
    s["scores"] = (-2.0 - torch.rand(b, w, generator=gen, device=dev) * 12.0).sort(1, descending=True)[0].contiguous()
    s["end"] = 1
    s["done"] = (torch.rand(b, w, generator=gen, device=dev) < case["done"]).to(torch.uint8)
    s["out_scores"] = torch.zeros(b, n_out, dtype=torch.float32, device=dev)
    s["out_tokens"], s["out_parents"] = (torch.zeros(b, n_out, dtype=torch.int32, device=dev) for _ in range(2))
    s["out_done"] = torch.zeros(b, n_out, dtype=torch.uint8, device=dev)
    if cols:       # rows with room to grow: the beams' slot rows and their tokens so far
        room = cols + 64
        s["rows"], s["tokens"] = (torch.randint(0, 1 << 20, (b * w, room), generator=gen, device=dev).int() for _ in range(2))
        s["start"] = (torch.arange(b * w, device=dev).int() * room).view(b, w)
        last = torch.randint(cols // 2, cols, (b,), generator=gen, device=dev) + 1
        s["first"], s["last"] = (torch.zeros_like(last)).int(), last.int()
        s["new_rows"], s["new_tokens"] = s["rows"].clone(), s["tokens"].clone()
    return s


# -------------------------------------------------------------- the plain form
def _prompt_plain(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g, at = hq // hkv, 0
    for n in s["lens"]:
        heads = max(1, min(hkv, (1 << 29) // max(1, g * n * n)))
        later = torch.ones(n, n, dtype=torch.bool, device=s["q"].device).triu_(1)
        for h in range(0, hkv, heads):
            e = min(h + heads, hkv)
            q = s["q"][at:at + n, h * g:e * g].float().unflatten(1, (e - h, g)).permute(1, 2, 0, 3)     # [heads, g, n, d]
            k, v = (s[x][at:at + n, h:e].float().transpose(0, 1)[:, None] for x in ("k", "v"))         # [heads, 1, n, d]
            sc = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).masked_fill_(later, -math.inf)
            m = sc.amax(-1, keepdim=True) if n else sc.sum(-1, keepdim=True)
            p = sc.sub_(m).exp_()
            l = p.sum(-1, keepdim=True)
            o = torch.matmul(p, v) / l
            s["out"][at:at + n, h * g:e * g] = o.permute(2, 0, 1, 3).flatten(1, 2).bfloat16()
            s["lse"][at:at + n, h * g:e * g] = (m + l.log())[..., 0].permute(2, 0, 1).flatten(1, 2)
        at += n


def _rotated(x, case, table, positions):
    """Rows [n, heads, d], the first rot columns turned: pair j by the angle of its axis' position, fp32."""
    x, rot = x.float(), case["rot"]
    axis = torch.tensor(_pair_axis(case), device=x.device)
    at = positions.long()[axis].t()                                              # [n, pairs]
    j = torch.arange(rot // 2, device=x.device)
    c, sn = table[at, j][:, None, :], table[at, j + rot // 2][:, None, :]
    part = x[..., :rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if case["inter"] else part.split(rot // 2, -1)
    ya, yb = a * c - b * sn, b * c + a * sn
    part = torch.stack([ya, yb], -1).flatten(-2) if case["inter"] else torch.cat([ya, yb], -1)
    return torch.cat([part, x[..., rot:]], -1)


def _append_plain(s):
    case = s["case"]
    k = _rotated(s["k_new"], case, s["table"], s["positions"])
    s["q_out"].copy_(_rotated(s["q"], case, s["table"], s["positions"]))
    at = s["slots"].long()
    for name, x in (("k", k), ("v", s["v_new"].float())):
        if case["pool"] == "bf16":
            s[name][at] = x.bfloat16()
        elif case["pool"] == "fp8":
            codes, scales = _to_e4m3(x)
            s[name].view(torch.uint8)[at] = codes.view(torch.uint8)
            s[name + "_scale"][at] = scales
        else:
            s[name][at], s[name + "_bscale"][at] = _to_blocks(x)


def _load_plain(s):
    pool, at = s["case"]["pool"], s["slots"].long()
    for name in ("k", "v"):
        if s[name] is None:
            continue
        if pool == "fp4":
            x = _from_blocks(s[name][at], s[name + "_bscale"][at])
        elif pool == "fp8":
            x = s[name].view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * s[name + "_scale"][at][..., None]
        else:
            x = s[name][at].view(s["k_out"].shape)
        s[name + "_out"].copy_(x)


def _select_plain(s):
    case = s["case"]
    b, w, vocab, n_out = (case[k] for k in ("batch", "beams", "vocab", "n_out"))
    x = s["logits"].double()
    m = x.amax(-1, keepdim=True)
    lse = m + (x - m).exp().sum(-1, keepdim=True).log()
    score = x - lse + s["scores"].double()[..., None]
    stays = torch.full((vocab,), -math.inf, dtype=torch.float64, device=x.device)
    stays[s["end"]] = 0.0
    done = s["done"].bool()
    score = torch.where(done[..., None], s["scores"].double()[..., None] + stays, score).flatten(1)
    val, at = torch.sort(score, dim=1, descending=True, stable=True)
    val, at = val[:, :n_out], at[:, :n_out]
    some = val > -math.inf
    parents, tokens = torch.where(some, at // vocab, 0), torch.where(some, at % vocab, 0)
    s["out_scores"].copy_(val)
    s["out_tokens"].copy_(tokens)
    s["out_parents"].copy_(parents)
    s["out_done"].copy_(some & (done.gather(1, parents) | (tokens == s["end"])))
    if case["cols"]:
        col = torch.arange(s["rows"].shape[1], device=x.device)
        moves = ((col >= s["first"][:, None]) & (col < s["last"][:, None]))[:, None]             # [b, 1, room]
        frm = parents[:, :w, None].expand(b, w, len(col))
        for old, new in (("rows", "new_rows"), ("tokens", "new_tokens")):
            t = s[old].view(b, w, -1)
            s[new].view(b, w, -1).copy_(torch.where(moves, t.gather(1, frm), s[new].view(b, w, -1)))


# ------------------------------------------------------- the framework's calls
def _plan(s):
    """Descriptors of a state's buffers, made once."""
    import radixattention_prefix_shared_tree_gb300 as ra
    case = s["case"]
    p = {"ra": ra}
    if case["op"] in ("append", "load"):
        raw = lambda t: t.view(torch.uint8) if t is not None and t.dtype == torch.float8_e4m3fn else t  # noqa: E731
        p["pool"] = ra.make_pool_desc(raw(s["k"]), raw(s["v"]), s["err"], mla=case["pool"] == "latent", head_dim_v=512,
                                      k_scale=s.get("k_scale"), v_scale=s.get("v_scale"), k_bscale=s.get("k_bscale"),
                                      v_bscale=s.get("v_bscale"))
    if case["op"] == "append":
        p["rope"] = ra.make_rope_desc(s["table"], interleaved=case["inter"], pair_axis=_pair_axis(case))
    return p


def _run_own(s):
    if "plan" not in s:
        s["plan"] = _plan(s)
    p, case = s["plan"], s["case"]
    ra, op = p["ra"], case["op"]
    if op == "prompt":
        ra.attn_prompt(s["q"], s["k"], s["v"], s["indptr"], s["scale"], s["out"], s["lse"], err=s["err"])
    elif op == "append":
        ra.kv_store_rope(p["pool"], p["rope"], s["slots"], s["positions"], s["k_new"], s["v_new"], s["q"], s["q_out"])
    elif op == "load":
        ra.kv_load(p["pool"], s["slots"], s["k_out"], s["v_out"])
    else:
        ra.beam_select(s["logits"], s["scores"], s["out_scores"], s["out_tokens"], s["out_parents"], done=s["done"],
                       end_token=s["end"], out_done=s["out_done"], err=s["err"])
        if case["cols"]:
            parents = s["out_parents"] if case["n_out"] == case["beams"] else \
                s["out_parents"][:, :case["beams"]].contiguous()
            for old, new in (("rows", "new_rows"), ("tokens", "new_tokens")):
                ra.beam_reorder(s[old], s["start"], s["first"], s["last"], parents, case["cols"], out=s[new], err=s["err"])


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        _run_own(s)
    else:
        {"prompt": _prompt_plain, "append": _append_plain, "load": _load_plain, "select": _select_plain}[op](s)
    if op == "prompt":
        return [s["out"], s["lse"]]
    if op == "append":
        out = [s["q_out"]]
        for name in ("k", "v"):
            if "k_bscale" in s:
                out.append(_from_blocks(s[name], s[name + "_bscale"]).bfloat16())     # (at most six significant bits: exact)
            else:
                out += [s[name]] + ([s[name + "_scale"]] if "k_scale" in s else [])
        return out
    if op == "load":
        return [s["k_out"]] + ([s["v_out"]] if s["v_out"] is not None else [])
    out = [s["out_scores"], s["out_tokens"], s["out_parents"], s["out_done"]]
    return out + ([s["new_rows"], s["new_tokens"]] if s["case"]["cols"] else [])


# ------------------------------------------------------- the definition, 64 bits
def _turn64(x, case, table, positions):
    """Each pair (a, b) as the complex number a + ib times cos + i sin of its own axis' position."""
    x = x.double().clone()
    half = case["rot"] // 2
    t = table.double()
    for j, axis in enumerate(_pair_axis(case)):
        row = t[positions[axis].long()]
        ia, ib = (2 * j, 2 * j + 1) if case["inter"] else (j, j + half)
        z = torch.complex(x[..., ia], x[..., ib]) * torch.complex(row[:, j], row[:, j + half])[:, None]
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


def _exact_prompt(s):
    hq, hkv, d = (s["case"][k] for k in ("hq", "hkv", "d"))
    out = torch.empty(len(s["q"]), hq, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.empty(len(s["q"]), hq, dtype=torch.float64, device=s["q"].device)
    at = 0
    for n in s["lens"]:
        for h in range(hq if n else 0):
            k, v = (s[x][at:at + n, h * hkv // hq].double() for x in ("k", "v"))
            for i in range(0, n, 4096):      # a block of queries sees the keys up to its end
                e = min(i + 4096, n)
                sc = s["q"][at + i:at + e, h].double() @ k[:e].t() * s["scale"]
                sc += torch.full_like(sc, -math.inf).triu(i + 1)
                t = torch.logsumexp(sc, -1)
                out[at + i:at + e, h] = torch.exp(sc - t[:, None]) @ v[:e]
                lse[at + i:at + e, h] = t
        at += n
    return [out, lse]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prompt":
        return _exact_prompt(s)
    if op == "append":
        turned = [_turn64(s[x], case, s["table"], s["positions"]) for x in ("q", "k_new")] + [s["v_new"].double()]
        out, at = [turned[0]], s["slots"].long()
        for name, x in (("k", turned[1]), ("v", turned[2])):
            if case["pool"] == "fp4":
                # the plain definition of a block: its scale the nearest that the byte can hold, its values the nearest codes
                b = x.unflatten(-1, (-1, 16))
                raw = b.abs().amax(-1) / 6
                step = torch.exp2(torch.floor(torch.log2(raw.clamp(min=2.0 ** -14))) - 3)
                sc = (torch.round(raw / step) * step).clamp(max=10240.0)[..., None]
                y = torch.where(sc > 0, b / sc, 0.0).abs().clamp(max=6.0)
                part = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
                full = _value64(s[name], s[name + "_bscale"])
                full[at] = (torch.round(y / part) * part * sc * b.sign()).flatten(-2)
                out.append(full)
            elif case["pool"] == "fp8":
                codes, scale = s[name].double(), s[name + "_scale"].double()
                sc = x.abs().amax(-1) / 448
                y = x / sc[..., None]
                step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                codes[at], scale[at] = torch.round(y / step) * step, sc
                out += [codes, scale]
            else:
                full = s[name].double()
                full[at] = x
                out.append(full)
        return out
    if op == "load":
        at, out = s["slots"].long(), []
        for name in ("k", "v"):
            if s[name] is not None:
                if case["pool"] == "fp4":
                    out.append(_value64(s[name][at], s[name + "_bscale"][at]))
                elif case["pool"] == "fp8":
                    out.append(s[name].double()[at] * s[name + "_scale"].double()[at][..., None])
                else:
                    out.append(s[name][at].double().view(s["k_out"].shape))
        return out
    # every beam's best n_out alone, by repeated search for the largest, then the best of those
    w, vocab, n_out = case["beams"], case["vocab"], case["n_out"]
    x = s["logits"].double()
    free = x - torch.logsumexp(x, -1, keepdim=True)
    free[s["done"].bool()] = -math.inf
    free[..., s["end"]] = torch.where(s["done"].bool(), 0.0, free[..., s["end"]])
    score = (s["scores"].double()[..., None] + free).flatten(1)
    scores, tokens, parents = [], [], []
    index = torch.arange(w * vocab, device=x.device)
    for _ in range(n_out):
        best = score.amax(1, keepdim=True)
        at = torch.where(score == best, index, w * vocab).amin(1)      # the lowest index of the best
        live = best[:, 0] > -math.inf
        at = torch.where(live, at, 0)
        scores.append(best[:, 0])
        tokens.append(at % vocab)
        parents.append(at // vocab)
        score.scatter_(1, at[:, None], -math.inf)
    scores, tokens, parents = (torch.stack(y, 1) for y in (scores, tokens, parents))
    done = (scores > -math.inf) & (s["done"].bool().gather(1, parents) | (tokens == s["end"]))
    out = [scores, tokens.int(), parents.int(), done.to(torch.uint8)]
    if case["cols"]:
        for old in ("rows", "tokens"):
            new = s[old].view(-1, w, s[old].shape[1]).clone()
            for b, (a, e) in enumerate(zip(s["first"].tolist(), s["last"].tolist())):
                new[b, :, a:e] = s[old].view(new.shape)[b, parents[b, :w], a:e]
            out.append(new.view(s[old].shape))
    return out
