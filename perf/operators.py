"""Cases of the 4-bit KV cache operators and of the rotating append: their plain forms and the library's calls.

Three operators, used together by a serving loop:

* ``append``: the new tokens' keys (rotated by their positions) and values go into a KV cache, the queries are
  rotated on the way and come out in the fp32 layout that the attention calls take.  Caches: bf16, fp32, and 4-bit.
* ``attend``: decode attention over a 4-bit cache, for one query row or a few per sequence.
* ``read``: rows of a 4-bit cache as bf16 or fp32 values.

The 4-bit cache holds e2m1 codes with one e4m3 scale for sixteen consecutive channels of a token; a value is
code * scale * 2**exp.  It is laid out in blocks of sixteen tokens of one KV head, 18 * D bytes each:
K codes [16 tokens][D/2] (row t's 16-byte chunks swizzled), V codes [D][8] (two tokens a byte),
K scales [16][D/16], V scales [D/16][16].
"""

import math

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases
def listed():
    """What each stands for in real use is said beside it."""
    return [
        # one decode step of a served batch: every sequence brings a token (latency counts)
        {"name": "append_bf16_step", "op": "append", "cache": "bf16", "new": "bf16", "B": 64, "n": 1, "Hq": 32, "Hkv": 8,
         "D": 128, "cap": 512, "page": 16, "rot": 128, "interleaved": False, "ragged": False, "positions": False},
        # a whole prompt of one sequence goes into a contiguous cache
        {"name": "append_bf16_prompt", "op": "append", "cache": "bf16", "new": "bf16", "B": 1, "n": 8192, "Hq": 32,
         "Hkv": 8, "D": 128, "cap": 8192, "page": 0, "rot": 128, "interleaved": False, "ragged": False,
         "positions": False},
        # ragged windows with positions of their own (a tree of drafts), fp32 cache, neighbours rotated, half of the channels
        {"name": "append_f32_window", "op": "append", "cache": "f32", "new": "f32", "B": 6, "n": 37, "Hq": 12, "Hkv": 4,
         "D": 64, "cap": 320, "page": 0, "rot": 32, "interleaved": True, "ragged": True, "positions": True},
        # the decode step again, into pages of a 4-bit cache; the rows are read back
        {"name": "append_4bit_step", "op": "append", "cache": "4bit", "new": "bf16", "B": 96, "n": 1, "Hq": 32, "Hkv": 8,
         "D": 128, "cap": 512, "page": 16, "rot": 128, "interleaved": False, "ragged": False, "positions": False},
        # prompts of a padded batch into a 4-bit cache, half of the channels rotated; the rows are read back
        {"name": "append_4bit_prompt", "op": "append", "cache": "4bit", "new": "bf16", "B": 4, "n": 2048, "Hq": 32,
         "Hkv": 8, "D": 128, "cap": 4096, "page": 0, "rot": 64, "interleaved": False, "ragged": True,
         "positions": False},
        # the smallest decode: one short sequence (latency counts)
        {"name": "attend_tiny", "op": "attend", "B": 1, "nq": 1, "Hq": 4, "Hkv": 4, "D": 64, "lo": 1024, "hi": 1024,
         "page": 0},
        # one sequence of 128k tokens, grouped heads: the split over the long axis counts
        {"name": "attend_128k", "op": "attend", "B": 1, "nq": 1, "Hq": 32, "Hkv": 8, "D": 128, "lo": 131072,
         "hi": 131072, "page": 0},
        # a ragged batch in a padded contiguous cache
        {"name": "attend_ragged", "op": "attend", "B": 16, "nq": 1, "Hq": 32, "Hkv": 8, "D": 128, "lo": 1024,
         "hi": 16384, "page": 0},
        # a large served batch over scattered pages of sixteen tokens, eight heads a group
        {"name": "attend_paged", "op": "attend", "B": 64, "nq": 1, "Hq": 64, "Hkv": 8, "D": 128, "lo": 512,
         "hi": 16384, "page": 16},
        # a few drafted tokens verified at once, some sequences shorter than the window
        {"name": "attend_rows", "op": "attend", "B": 8, "nq": 4, "Hq": 32, "Hkv": 8, "D": 128, "lo": 2, "hi": 16384,
         "page": 16},
        # a long prefix read out as bf16, as the attention of a further prompt chunk needs it
        {"name": "read_prefix", "op": "read", "B": 1, "Hkv": 8, "D": 128, "lo": 32768, "hi": 32768, "page": 0,
         "out": "bf16"},
        # ragged sequences read out of pages in fp32
        {"name": "read_paged", "op": "read", "B": 8, "Hkv": 4, "D": 64, "lo": 33, "hi": 999, "page": 32, "out": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "read"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 8, 16])
    page = rng.choice([0, 16, 32, 48, 64])
    if op == "append":
        B = _log(rng, 1, 96)
        n = _log(rng, 1, max(1, min(2048, 4096 // B)))
        cap = -(-(n + _log(rng, 1, 512)) // 16) * 16
        return {"op": op, "cache": rng.choice(["bf16", "f32", "4bit", "4bit"]), "new": rng.choice(["bf16", "f32"]), "B": B,
                "n": n, "Hq": g * Hkv if g * Hkv <= 32 else Hkv, "Hkv": Hkv, "D": D, "cap": cap, "page": page,
                "rot": rng.choice([r for r in (0, 32, 64, 96, 128) if r <= D]), "interleaved": rng.random() < 0.4,
                "ragged": rng.random() < 0.5, "positions": rng.random() < 0.4}
    if op == "attend":
        B = _log(rng, 1, 32)
        nq = rng.choice([1, 1, 1, 2, 3, 5, 16])
        hi = _log(rng, 1, 262144 // (B * Hkv))
        return {"op": op, "B": B, "nq": nq, "Hq": g * Hkv, "Hkv": Hkv, "D": D, "lo": rng.choice([0, 1, max(1, hi // 2), hi]),
                "hi": hi, "page": page}
    B = _log(rng, 1, 16)
    hi = _log(rng, 1, 262144 // (B * Hkv))
    return {"op": op, "B": B, "Hkv": Hkv, "D": D, "lo": rng.choice([0, hi]), "hi": hi, "page": page,
            "out": rng.choice(["bf16", "f32"])}


# ------------------------------------------------------------------ inputs
def _quantise(x):
    """e2m1 codes (uint8, sign in bit 3) and e4m3 scales of x [..., D] fp32, sixteen channels a scale."""
    blocks = x.unflatten(-1, (-1, 16))
    amax = blocks.abs().amax(-1)
    # a true quotient (a scalar divisor would be a product with 1 / 6): scales next to a border round as defined
    sf = (amax / torch.full_like(amax, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = sf.float().unsqueeze(-1)
    r = torch.where(s > 0, blocks.abs() / s, torch.zeros_like(blocks))
    # halfway cases go to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    code = ((r > 0.25).to(torch.uint8) + (r >= 0.75) + (r > 1.25) + (r >= 1.75) + (r > 2.5) + (r >= 3.5) + (r > 5.0))
    return (code + 8 * torch.signbit(blocks).to(torch.uint8)).flatten(-2).to(torch.uint8), sf


def _swizzle(D, device):
    """Where chunk c of row t sits: [16, chunks]."""
    t = torch.arange(16, device=device).unsqueeze(1)
    c = torch.arange(D // 32, device=device).unsqueeze(0)
    return c ^ ((t // 2) % 4 if D == 128 else (t // 4) % 2)


def _pack(kc, ks, vc, vs):
    """Blocks [..., 18 * D] of codes [..., 16, D] and scales [..., 16, D / 16]."""
    D = kc.shape[-1]
    at = _swizzle(D, kc.device)
    chunks = (kc[..., 0::2] + 16 * kc[..., 1::2]).unflatten(-1, (D // 32, 16))  # [..., 16, C, 16 bytes]
    kb = torch.gather(chunks, -2, at.unsqueeze(-1).expand(chunks.shape))  # the swizzle is its own inverse
    vt = vc.transpose(-1, -2)
    vb = vt[..., 0::2] + 16 * vt[..., 1::2]
    parts = (kb, vb, ks.view(torch.uint8), vs.view(torch.uint8).transpose(-1, -2))
    lead = len(kc.shape) - 2
    return torch.cat([p.flatten(lead) for p in parts], -1).contiguous()


def _filled(blocks, Hkv, D, gen, dev):
    """A 4-bit cache of N(0, 1) keys and values: [blocks in all, 18 * D], made in pieces."""
    out = torch.empty((blocks * Hkv, 18 * D), dtype=torch.uint8, device=dev)
    step = 1 << 14
    for i in range(0, out.shape[0], step):
        m = min(step, out.shape[0] - i)
        x = torch.randn((2, m, 16, D), generator=gen, device=dev)
        # a few channels of the keys are larger than the others, as rotated keys have them
        x[0, ..., 3::17] *= 4.0
        kc, ks = _quantise(x[0])
        vc, vs = _quantise(x[1])
        out[i:i + m] = _pack(kc, ks, vc, vs)
    return out


def _lengths(case, gen):
    """Lengths log-uniform in [lo, hi], the longest one present."""
    lo, hi, B = case["lo"], case["hi"], case["B"]
    u = torch.rand(B, generator=gen, dtype=torch.float64)
    lens = torch.exp(math.log(lo + 1) + u * (math.log(hi + 1) - math.log(lo + 1))).floor().long() - 1
    lens = lens.clamp(lo, hi)
    lens[int(torch.randint(B, (1,), generator=gen))] = hi
    return lens


def _table(pages_per_seq, B, gen):
    perm = torch.randperm(B * pages_per_seq, generator=gen)
    return perm.view(B, pages_per_seq).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, D, Hkv, page = case["B"], case["D"], case["Hkv"], case["page"]
    s = dict(case)
    if case["op"] == "append":
        n, cap, Hq = case["n"], case["cap"], case["Hq"]
        nl = torch.randint(0, n + 1, (B,), generator=cpu) if case["ragged"] else torch.full((B,), n)
        lens = torch.randint(0, cap - n + 1, (B,), generator=cpu)
        dt = {"bf16": torch.bfloat16, "f32": torch.float32}[case["new"]]
        # one fused projection of all heads, as a layer makes it: q, k and v are slices of it
        qkv = torch.randn((B, n, Hq + 2 * Hkv, D), generator=gen, device=dev).to(dt)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        s["new_lens"] = nl.to(torch.int32).to(dev) if case["ragged"] else None
        s["seq_lens"] = lens.to(torch.int32).to(dev)
        s["ends"] = (lens + nl).to(torch.int32).to(dev)
        s["max_len"] = int(cap - n)
        max_pos = cap + 64
        s["positions"] = (torch.randint(0, max_pos, (B, n), generator=cpu).to(torch.int32).to(dev)
                          if case["positions"] else None)
        s["cos"] = s["sin"] = None
        if case["rot"]:
            inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev) / case["rot"])
            ang = torch.arange(max_pos, dtype=torch.float64, device=dev).unsqueeze(1) * inv
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        s["q_out"] = torch.zeros((B, Hq, n, D), device=dev)
        s["table"] = None
        if page:
            cap = -(-cap // page) * page
            s["table"] = _table(cap // page, B, cpu).to(dev)
        if case["cache"] == "4bit":
            shape = (B * cap // page, Hkv, page // 16, 18 * D) if page else (B, Hkv, cap // 16, 18 * D)
            s["kv4"] = _filled(B * cap // 16, Hkv, D, gen, dev).view(shape)
            s["k_rows"] = torch.zeros((B, Hkv, n, D), device=dev, dtype=torch.bfloat16)
            s["v_rows"] = torch.zeros((B, Hkv, n, D), device=dev, dtype=torch.bfloat16)
        else:
            ct = {"bf16": torch.bfloat16, "f32": torch.float32}[case["cache"]]
            shape = (B * cap // page, Hkv, page, D) if page else (B, Hkv, cap, D)
            s["k"] = torch.randn(shape, generator=gen, device=dev).to(ct)
            s["v"] = torch.randn(shape, generator=gen, device=dev).to(ct)
        return s
    lens = _lengths(case, cpu)
    unit = page or 16
    cap = max(unit, -(-case["hi"] // unit) * unit)
    s["cap"] = cap
    s["table"] = _table(cap // page, B, cpu).to(dev) if page else None
    shape = (B * cap // page, Hkv, page // 16, 18 * D) if page else (B, Hkv, cap // 16, 18 * D)
    s["kv4"] = _filled(B * cap // 16, Hkv, D, gen, dev).view(shape)
    s["seq_lens"] = lens.to(torch.int32).to(dev)
    s["max_len"] = int(case["hi"])
    if case["op"] == "attend":
        s["q"] = torch.randn((B, case["Hq"], case["nq"], D), generator=gen, device=dev)
    else:
        out = {"bf16": torch.bfloat16, "f32": torch.float32}[case["out"]]
        s["k_rows"] = torch.zeros((B, Hkv, case["hi"], D), device=dev, dtype=out)
        s["v_rows"] = torch.zeros((B, Hkv, case["hi"], D), device=dev, dtype=out)
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(x, cos, sin, interleaved):
    """x [B, n, H, D] with cos, sin [B, n, rot / 2]: the first rot channels rotated in fp32."""
    x = x.float()
    if cos is None:
        return x
    half = cos.shape[-1]
    c, s = cos.unsqueeze(2), sin.unsqueeze(2)
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    lo, hi = a * c - b * s, b * c + a * s
    turned = torch.stack([lo, hi], -1).flatten(-2) if interleaved else torch.cat([lo, hi], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _unpack(blocks):
    """fp32 K and V [..., 16, D] of blocks [..., 18 * D]."""
    D = blocks.shape[-1] // 18
    lut = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=blocks.device)
    kb, vb, ks, vs = torch.split(blocks, [8 * D, 8 * D, D, D], -1)
    kb = kb.unflatten(-1, (16, D // 32, 16))
    kb = torch.gather(kb, -2, _swizzle(D, blocks.device).unsqueeze(-1).expand(kb.shape)).flatten(-2)
    k = lut[torch.stack([kb & 15, kb >> 4], -1).flatten(-2).int()]
    vb = vb.unflatten(-1, (D, 8))
    v = lut[torch.stack([vb & 15, vb >> 4], -1).flatten(-2).int()].transpose(-1, -2)
    ks = ks.unflatten(-1, (16, D // 16)).contiguous().view(torch.float8_e4m3fn).float()
    vs = vs.unflatten(-1, (D // 16, 16)).contiguous().view(torch.float8_e4m3fn).float().transpose(-1, -2)
    return k * ks.repeat_interleave(16, -1), v * vs.repeat_interleave(16, -1)


def _sequences(s):
    """fp32 K and V [B, Hkv, tokens, D] of the state's 4-bit cache."""
    kv4 = s["kv4"]
    if s["table"] is not None:
        kv4 = kv4[s["table"].long()].transpose(1, 2)  # [B, Hkv, pages, blocks, bytes]
        kv4 = kv4.flatten(2, 3)
    k, v = _unpack(kv4)
    return k.flatten(2, 3), v.flatten(2, 3)


def _new_tokens(s):
    """Token number of each new row (negative: padding) and its place in the cache: [B, n] both."""
    n = s["n"]
    nl = s["new_lens"].long() if s["new_lens"] is not None else torch.full_like(s["seq_lens"], n).long()
    j = torch.arange(n, device=nl.device).unsqueeze(0) - (n - nl).unsqueeze(1)
    return j, s["seq_lens"].long().unsqueeze(1) + j


def _plain_append(s):
    j, t = _new_tokens(s)
    live = j >= 0
    cos = sin = None
    if s["cos"] is not None:
        at = s["positions"].long() if s["positions"] is not None else t.clamp(min=0)
        cos, sin = s["cos"][at], s["sin"][at]
    q = _rotate(s["q"], cos, sin, s["interleaved"]).transpose(1, 2)
    s["q_out"].copy_(torch.where(live[:, None, :, None], q, s["q_out"]))
    k, v = _rotate(s["k_new"], cos, sin, s["interleaved"]), s["v_new"].float()
    b, i = live.nonzero(as_tuple=True)
    if s["cache"] == "4bit":
        for_rows = j[b, i]
        kc, ks = _quantise(k)
        vc, vs = _quantise(v)
        lut = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=k.device)
        s["k_rows"][b, :, for_rows] = (lut[kc.int()] * ks.float().repeat_interleave(16, -1))[b, i].to(torch.bfloat16)
        s["v_rows"][b, :, for_rows] = (lut[vc.int()] * vs.float().repeat_interleave(16, -1))[b, i].to(torch.bfloat16)
        return {"q": s["q_out"], "k": s["k_rows"], "v": s["v_rows"]}
    place = t[b, i]
    if s["table"] is not None:
        page = s["k"].shape[2]
        at = (s["table"].long()[b, place // page], slice(None), place % page)
    else:
        at = (b, slice(None), place)
    s["k"][at] = k[b, i].to(s["k"].dtype)
    s["v"][at] = v[b, i].to(s["v"].dtype)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _plain_attend(s):
    B, Hq, nq, D = s["q"].shape
    k, v = _sequences(s)
    T = k.shape[2]
    q = s["q"].reshape(B, s["Hkv"], -1, D)  # the group's heads and rows together
    x = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    row = torch.arange(q.shape[2], device=q.device) % nq
    limit = s["seq_lens"].long().view(B, 1, 1, 1) - (nq - 1 - row).view(1, 1, -1, 1)
    x = x.masked_fill(torch.arange(T, device=q.device) >= limit, -math.inf)
    m = x.amax(-1, keepdim=True)
    some = m > -math.inf
    e = torch.exp(x - torch.where(some, m, torch.zeros_like(m)))
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e, v) / torch.where(some, total, torch.ones_like(total))
    lse = torch.where(some, m + torch.log(total), m)
    return {"out": out.view(B, Hq, nq, D), "lse": lse.view(B, Hq, nq)}


def _plain_read(s):
    k, v = _sequences(s)
    n = s["k_rows"].shape[2]
    live = (torch.arange(n, device=k.device) < s["seq_lens"].unsqueeze(1))[:, None, :, None]
    s["k_rows"].copy_(torch.where(live, k[:, :, :n], s["k_rows"].float()))
    s["v_rows"].copy_(torch.where(live, v[:, :, :n], s["v_rows"].float()))
    return {"k": s["k_rows"], "v": s["v_rows"]}


# ------------------------------------------------------------------ one pass
def run(s):
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "read": _plain_read}[s["op"]](s)
    import split_kv_decode_fd_gb300 as fd

    if s["op"] == "append":
        how = dict(q=s["q"], q_out=s["q_out"], interleaved=s["interleaved"], positions=s["positions"],
                   new_lens=s["new_lens"], seq_lens=s["seq_lens"], max_seq_len=s["max_len"], block_table=s["table"])
        if s["cache"] != "4bit":
            q = fd.append_rope(s["k_new"], s["v_new"], s["k"], s["v"], s["cos"], s["sin"], **how)
            return {"q": q, "k": s["k"], "v": s["v"]}
        q = fd.append_rope_kv4(s["k_new"], s["v_new"], s["kv4"], s["cos"], s["sin"], **how)
        k, v = fd.kv4_read(s["kv4"], s["n"], starts=s["seq_lens"], seq_lens=s["ends"], block_table=s["table"],
                           k_out=s["k_rows"], v_out=s["v_rows"])
        return {"q": q, "k": k, "v": v}
    if s["op"] == "attend":
        out, lse = fd.decode_kv4(s["q"], s["kv4"], seq_lens=s["seq_lens"], max_seq_len=s["max_len"],
                                 block_table=s["table"])
        return {"out": out, "lse": lse}
    k, v = fd.kv4_read(s["kv4"], s["hi"], seq_lens=s["seq_lens"], block_table=s["table"], k_out=s["k_rows"],
                       v_out=s["v_rows"])
    return {"k": k, "v": v}


def work(case):
    """Lengths count with their expected sum; a multiply and an add are two operations."""
    B, D, Hkv = case["B"], case["D"], case["Hkv"]
    if case["op"] == "append":
        es = {"bf16": 2, "f32": 4}[case["new"]]
        tokens = B * case["n"] * (0.5 if case["ragged"] else 1.0)
        cos = 4.0 * case["rot"] * min(tokens, case["cap"])
        q = tokens * case["Hq"] * D * (es + 4)
        kv = 2 * tokens * Hkv * D * es
        if case["cache"] == "4bit":  # the packed rows are written and read, their values written
            kv += 2 * tokens * Hkv * D * (2 * 0.5625 + 2)
        else:
            kv += 2 * tokens * Hkv * D * {"bf16": 2, "f32": 4}[case["cache"]]
        flops = tokens * (case["Hq"] + Hkv) * case["rot"] * 3
        return {"bytes": cos + q + kv, "flops": flops}
    lo, hi = case["lo"] + 1.0, case["hi"] + 1.0
    mean = (hi - lo) / math.log(hi / lo) - 1 if hi > lo else case["hi"]
    tokens = max(1.0, (B - 1) * mean + case["hi"])
    packed = tokens * Hkv * D * 2 * 0.5625
    if case["op"] == "attend":
        rows = B * case["Hq"] * case["nq"]
        return {"bytes": packed + rows * (2 * D + 1) * 4.0, "flops": 4.0 * tokens * case["Hq"] * case["nq"] * D}
    return {"bytes": packed + 2 * tokens * Hkv * D * {"bf16": 2, "f32": 4}[case["out"]], "flops": 2 * tokens * Hkv * D}


# ------------------------------------------------------------------ 64 bits
def _power_64(e):
    """2 ** e of whole numbers in [-64, 64], exactly."""
    return torch.tensor([2.0 ** k for k in range(-64, 65)], dtype=torch.float64, device=e.device)[e.long() + 64]


def _e4m3_64(x):
    """Nearest e4m3 value (halfway: even significand) of x >= 0 in 64 bits, at most 448."""
    step = _power_64((torch.frexp(x)[1] - 1).clamp(-6, 60) - 3)
    return (torch.round(x / step) * step).clamp(max=448.0)


def _fp4_64(x):
    """Values that x [..., D] in 64 bits is held as, sixteen channels a scale."""
    y = x.unflatten(-1, (-1, 16))
    amax = y.abs().amax(-1, keepdim=True)
    sf = _e4m3_64(amax / torch.full_like(amax, 6.0))
    r = (y.abs() / torch.where(sf > 0, sf, torch.ones_like(sf))).clamp(max=6.0) * (sf > 0)
    step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0)).to(r.dtype)
    return (torch.copysign(torch.round(r / step) * step, y) * sf).flatten(-2)


def _turn_64(x, angle_cos, angle_sin, interleaved):
    """Every pair of channels as a complex number times cos + i sin."""
    x = x.double()
    half = angle_cos.shape[-1]
    first = torch.arange(half, device=x.device) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    z = torch.complex(x[..., first], x[..., second]) * torch.complex(angle_cos.double(), angle_sin.double()).unsqueeze(2)
    out = x.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _tokens_64(s, b, count):
    """K and V [Hkv, count, D] of sequence b in 64 bits, byte by byte from the cache."""
    kv4, D, dev = s["kv4"], s["D"], s["kv4"].device
    t = torch.arange(count, device=dev)
    if s["table"] is not None:
        page = 16 * kv4.shape[2]
        rows = kv4[s["table"][b].long()[t // page], :, t % page // 16]  # [count, Hkv, bytes]
    else:
        rows = kv4[b][:, t // 16].transpose(0, 1)
    i, d = (t % 16).view(-1, 1), torch.arange(D, device=dev).view(1, -1)
    chunk = (d // 32) ^ ((i // 2) % 4 if D == 128 else (i // 4) % 2)
    def value(byte, high, scale):
        at = lambda x: torch.gather(rows, 2, x.expand(count, D).unsqueeze(1).expand(count, rows.shape[1], D)).int()  # noqa: E731
        c = at(byte) // torch.where(high, 16, 1).unsqueeze(1) % 16
        e, m = c % 8 // 2, c % 2
        size = torch.where(e > 0, (1.0 + 0.5 * m.double()) * _power_64(e - 1), 0.5 * m.double())
        f = at(scale)
        fe, fm = f // 8, f % 8
        sf = torch.where(fe > 0, (1.0 + fm.double() / 8) * _power_64(fe - 7), fm.double() / 8 * 2.0 ** -6)
        return (torch.where(c >= 8, -size, size) * sf).transpose(0, 1)
    zero = 0 * i + 0 * d
    k = value(i * (D // 2) + chunk * 16 + d % 32 // 2, (d % 2 == 1) | (zero == 1), 16 * D + i * (D // 16) + d // 16)
    v = value(8 * D + d * 8 + i // 2, (i % 2 == 1) | (zero == 1), 17 * D + (d // 16) * 16 + i)
    return k, v


def exact(case, seed):
    s = prepare(case, seed)
    B = case["B"]
    if case["op"] == "append":
        n = case["n"]
        q = s["q_out"].double()
        four = case["cache"] == "4bit"
        k, v = (s["k_rows"].double(), s["v_rows"].double()) if four else (s["k"].double(), s["v"].double())
        for b in range(B):
            L, end = int(s["seq_lens"][b]), int(s["ends"][b])
            if end == L:
                continue
            first = n - (end - L)
            rows = [x[b, first:].unsqueeze(0) for x in (s["q"], s["k_new"], s["v_new"])]
            if case["rot"]:
                at = s["positions"][b, first:].long() if s["positions"] is not None else torch.arange(L, end, device=q.device)
                c, sn = s["cos"][at].unsqueeze(0), s["sin"][at].unsqueeze(0)
                rows[:2] = [_turn_64(x, c, sn, case["interleaved"]) for x in rows[:2]]
            qb, kb, vb = [x[0].double().transpose(0, 1) for x in rows]  # [heads, tokens, D]
            q[b, :, first:] = qb
            if four:
                k[b, :, :end - L], v[b, :, :end - L] = _fp4_64(kb), _fp4_64(vb)
            elif s["table"] is None:
                k[b, :, L:end], v[b, :, L:end] = kb, vb
            else:
                page = s["k"].shape[2]
                t = torch.arange(L, end, device=q.device)
                pages = s["table"][b].long()[t // page]
                k[pages, :, t % page], v[pages, :, t % page] = kb.transpose(0, 1), vb.transpose(0, 1)
        return {"q": q, "k": k, "v": v}
    if case["op"] == "read":
        k, v = s["k_rows"].double(), s["v_rows"].double()
        for b in range(B):
            L = int(s["seq_lens"][b])
            if L:
                k[b, :, :L], v[b, :, :L] = _tokens_64(s, b, L)
        return {"k": k, "v": v}
    nq, Hkv, D = case["nq"], case["Hkv"], case["D"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=s["q"].device)
    for b in range(B):
        L = int(s["seq_lens"][b])
        if L == 0:
            continue
        k, v = _tokens_64(s, b, L)
        q = s["q"][b].double().view(Hkv, -1, nq, D)
        for i in range(nq):
            end = L - (nq - 1 - i)
            if end <= 0:
                continue
            x = torch.einsum("hgd,htd->hgt", q[:, :, i], k[:, :end]) / math.sqrt(D)
            out[b, :, i] = torch.einsum("hgt,htd->hgd", torch.softmax(x, -1), v[:, :end]).reshape(-1, D)
            lse[b, :, i] = torch.logsumexp(x, -1).reshape(-1)
    return {"out": out, "lse": lse}
