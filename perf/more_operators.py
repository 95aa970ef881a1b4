"""Cases of the operators of a step with a tree of drafted tokens: their plain forms and the library's calls.

Three operators, used one after another by a serving loop that drafts several tokens a step:

* ``tree``: attention of the drafted tokens over a KV cache that holds the sequence and, in its last places, the drafts
  themselves.  A token sees everything before the drafts, its ancestors in the tree and itself.
* ``verify``: which drafts stay, by the target's and the draft's probabilities and given random numbers, and the token
  that comes after them.
* ``keep``: the rows of the tokens that stay move together in the cache.

The trees are given as ``parents``: token j of a sequence's drafts has the number of its parent, which is below j, or -1
for the first.  Every sequence has n rows; where their number is ragged, the last ``new_lens[b]`` of them are tokens.
"""

import math

import torch

own = False


# ------------------------------------------------------------------ the cases
def listed():
    """What each stands for in real use is said beside it."""
    return [
        # the smallest step: a chain of four drafts after a short chat (latency counts)
        {"name": "tree_tiny", "op": "tree", "cache": "bf16", "B": 1, "n": 5, "Hq": 4, "Hkv": 4, "D": 64, "lo": 1024, "hi": 1024,
         "page": 0, "shape": "chain", "ragged": False},
        # sixteen drafts at the end of one sequence of 128k tokens, grouped heads: the split over the long axis counts
        {"name": "tree_128k", "op": "tree", "cache": "bf16", "B": 1, "n": 16, "Hq": 32, "Hkv": 8, "D": 128, "lo": 131072,
         "hi": 131072, "page": 0, "shape": "random", "ragged": False},
        # a tree of 64 drafts on the same sequence: 256 rows share each key
        {"name": "tree_128k_wide", "op": "tree", "cache": "bf16", "B": 1, "n": 64, "Hq": 32, "Hkv": 8, "D": 128, "lo": 131072,
         "hi": 131072, "page": 0, "shape": "random", "ragged": False},
        # a large served batch over scattered pages, eight heads a group, ragged trees
        {"name": "tree_paged", "op": "tree", "cache": "bf16", "B": 64, "n": 8, "Hq": 64, "Hkv": 8, "D": 128, "lo": 512,
         "hi": 16384, "page": 16, "shape": "random", "ragged": True},
        # an fp32 cache, odd sizes
        {"name": "tree_f32", "op": "tree", "cache": "f32", "B": 6, "n": 13, "Hq": 12, "Hkv": 4, "D": 64, "lo": 300, "hi": 3000,
         "page": 0, "shape": "random", "ragged": True},
        # one sequence's chain of drafts (latency counts)
        {"name": "verify_chain", "op": "verify", "B": 1, "n": 8, "V": 32000, "probs": "f32", "draft": True, "shape": "chain",
         "ragged": False},
        # a served batch of trees over a large vocabulary
        {"name": "verify_batch", "op": "verify", "B": 64, "n": 16, "V": 131072, "probs": "f32", "draft": True,
         "shape": "random", "ragged": True},
        # drafts that are the likeliest tokens (no draft probabilities), a vocabulary of odd size, probabilities in 16 bits
        {"name": "verify_likeliest", "op": "verify", "B": 32, "n": 32, "V": 65521, "probs": "bf16", "draft": False,
         "shape": "random", "ragged": False},
        # the accepted path of one sequence (latency counts)
        {"name": "keep_step", "op": "keep", "cache": "bf16", "B": 1, "n": 5, "Hkv": 8, "D": 128, "cap": 4096, "page": 0,
         "keep": "path"},
        # a served batch's accepted paths, over pages
        {"name": "keep_batch", "op": "keep", "cache": "bf16", "B": 64, "n": 16, "Hkv": 8, "D": 128, "cap": 1024, "page": 16,
         "keep": "path"},
        # the first tokens and the latest half of a long sequence stay
        {"name": "keep_window", "op": "keep", "cache": "bf16", "B": 1, "n": 65536, "Hkv": 8, "D": 128, "cap": 131200, "page": 0,
         "keep": "window"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "verify", "verify", "keep"])
    shape = rng.choice(["chain", "random", "random", "wide"])
    if op == "verify":
        n = _log(rng, 1, 64)
        B = _log(rng, 1, 64)
        V = _log(rng, 50, min(131072, 134217728 // (B * n)))
        return {"op": op, "B": B, "n": n, "V": V, "probs": rng.choice(["f32", "f32", "bf16"]), "draft": rng.random() < 0.6,
                "shape": shape, "ragged": rng.random() < 0.5}
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([0, 16, 32, 48, 64])
    cache = rng.choice(["bf16", "bf16", "bf16", "f32"])
    B = _log(rng, 1, 48)
    if op == "tree":
        g = rng.choice([1, 2, 3, 4, 5, 8, 16])
        hi = _log(rng, 1, 262144 // (B * Hkv))
        return {"op": op, "cache": cache, "B": B, "n": _log(rng, 1, 64), "Hq": g * Hkv, "Hkv": Hkv, "D": D,
                "lo": rng.choice([1, max(1, hi // 2), hi]), "hi": hi, "page": page, "shape": shape,
                "ragged": rng.random() < 0.5}
    keep = rng.choice(["path", "path", "window"])
    n = _log(rng, 1, 64) if keep == "path" else _log(rng, 1, max(1, 262144 // (B * Hkv)))
    return {"op": op, "cache": cache, "B": B, "n": n, "Hkv": Hkv, "D": D,
            "cap": -(-(2 * n + _log(rng, 1, 512)) // 16) * 16, "page": page, "keep": keep}


# ------------------------------------------------------------------ inputs
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _parents(case, tokens, gen):
    """[B, n] of the last tokens[b] rows' parents (0 in the padding rows, which nothing reads)."""
    B, n = case["B"], case["n"]
    out = torch.zeros((B, n), dtype=torch.int32)
    for b in range(B):
        m = int(tokens[b])
        if m == 0:
            continue
        j = torch.arange(m)
        if case["shape"] == "chain":
            p = j - 1
        elif case["shape"] == "wide":
            p = torch.zeros_like(j)
        else:  # two or three children to a token, as a draft model widens its likeliest prefixes
            p = ((j - 1) // 2 - torch.randint(0, 3, (m,), generator=gen)).clamp(min=0)
        p[0] = -1
        out[b, n - m:] = p.to(torch.int32)
    return out


def _lengths(case, gen):
    """Lengths log-uniform in [lo, hi], the longest one present."""
    lo, hi, B = case["lo"], case["hi"], case["B"]
    u = torch.rand(B, generator=gen, dtype=torch.float64)
    lens = torch.exp(math.log(lo) + u * (math.log(hi + 1) - math.log(lo))).floor().long().clamp(lo, hi)
    lens[int(torch.randint(B, (1,), generator=gen))] = hi
    return lens


def _cache(case, cap, cpu, gen, dev):
    """K, V and the block table of a cache of N(0, 1) rows; a few channels of the keys are larger, as rotated keys have them."""
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    table = None
    shape = (B, Hkv, cap, D)
    if page:
        per = -(-cap // page)
        table = torch.randperm(B * per, generator=cpu).view(B, per).to(torch.int32).to(dev)
        shape = (B * per, Hkv, page, D)
    k = torch.randn(shape, generator=gen, device=dev)
    k[..., 3::17] *= 2.0
    v = torch.randn(shape, generator=gen, device=dev)
    return k.to(TYPES[case["cache"]]), v.to(TYPES[case["cache"]]), table


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, n = case["B"], case["n"]
    s = dict(case)
    if case["op"] == "keep":
        cap = case["cap"]
        s["k"], s["v"], s["table"] = _cache(case, cap, cpu, gen, dev)
        index = torch.zeros((B, n), dtype=torch.int64)
        counts = torch.zeros(B, dtype=torch.int64)
        for b in range(B):
            # kept rows that do not move, then rows from behind all that is kept: a second pass finds its sources as they were
            m = int(torch.randint(1, n + 1, (1,), generator=cpu)) if case["keep"] == "path" else n
            same = min(m, int(torch.randint(1, 3, (1,), generator=cpu)) if case["keep"] == "path" else 4 + int(
                torch.randint(0, 60, (1,), generator=cpu)))
            far = m + torch.randperm(max(m, n) + 1, generator=cpu)[:m - same].sort().values
            if case["keep"] == "window":
                far = m + 1 + torch.arange(m - same)
            index[b, :m] = torch.cat([torch.arange(same), far])
            counts[b] = m
        reach = int(index.max()) + 1
        s["index"] = index.to(torch.int32).to(dev)
        s["counts"] = counts.to(torch.int32).to(dev)
        s["starts"] = torch.randint(0, cap - reach + 1, (B,), generator=cpu).to(torch.int32).to(dev)
        return s
    tokens = torch.randint(1, n + 1, (B,), generator=cpu) if case["ragged"] else torch.full((B,), n)
    parents = _parents(case, tokens, cpu)
    s["parents"] = parents.to(dev)
    s["new_lens"] = tokens.to(torch.int32).to(dev) if case["ragged"] else None
    if case["op"] == "tree":
        lens = torch.maximum(_lengths(case, cpu), tokens)
        s["max_len"] = int(lens.max())
        s["k"], s["v"], s["table"] = _cache(case, -(-max(case["hi"], n) // 16) * 16, cpu, gen, dev)
        s["seq_lens"] = lens.to(torch.int32).to(dev)
        s["q"] = torch.randn((B, case["Hq"], n, case["D"]), generator=gen, device=dev)
        # rows of padding stay as they are
        s["out"] = torch.zeros((B, case["Hq"], n, case["D"]), device=dev)
        s["lse"] = torch.zeros((B, case["Hq"], n), device=dev)
        return s
    V = case["V"]
    # a few likely words, and a draft model that agrees on most of them
    logits = 5.0 * torch.randn((B, n, V), generator=gen, device=dev)
    target = torch.softmax(logits, -1)
    logits = 0.95 * logits + torch.randn((B, n, V), generator=gen, device=dev)
    # rank of a token among its parent's children
    rank = torch.zeros((B, n), dtype=torch.int64)
    for b in range(B):
        seen = {}
        for i in range(n - int(tokens[b]), n):
            p = int(parents[b, i])
            rank[b, i] = seen.get(p, 0)
            seen[p] = int(rank[b, i]) + 1
    most = min(V, int(rank.max()) + 1)
    row = (parents.long() + (n - tokens).unsqueeze(1)).clamp(min=0).to(dev)
    s["draft"] = None
    if case["draft"]:
        draft = torch.softmax(logits, -1)
        picks = torch.multinomial(draft.view(-1, V), most, replacement=True, generator=gen).view(B, n, most)
        s["draft"] = draft.to(TYPES[case["probs"]])
        del draft
    else:
        picks = logits.topk(most, -1).indices
    del logits
    s["target"] = target.to(TYPES[case["probs"]])
    at = row.unsqueeze(2).expand(B, n, most)
    s["tokens"] = torch.gather(torch.gather(picks, 1, at), 2, (rank % most).to(dev).unsqueeze(2)).squeeze(2).to(torch.int32)
    s["uniforms"] = torch.rand((B, n), generator=gen, device=dev)
    return s


# ------------------------------------------------------------------ plain forms
def _tokens(s):
    """Token number of each row (negative: padding) [B, n], and the number of tokens [B]."""
    B, n = s["parents"].shape
    m = s["new_lens"].long() if s["new_lens"] is not None else torch.full((B,), n, device=s["parents"].device)
    return torch.arange(n, device=m.device).unsqueeze(0) - (n - m).unsqueeze(1), m


def _ancestors(s):
    """[B, n, n] truth values: row i's token has row j's among its ancestors, or is it."""
    j, m = _tokens(s)
    n = j.shape[1]
    parent = s["parents"].long() + (n - m).unsqueeze(1)  # the parent's row
    rows = torch.arange(n, device=j.device)
    step = (parent.unsqueeze(2) == rows) & (s["parents"] >= 0).unsqueeze(2) & (j >= 0).unsqueeze(2)
    up = (step | (rows.unsqueeze(1) == rows)).float()
    for _ in range(max(1, (n - 1).bit_length())):  # twice as far up each time
        up = (torch.matmul(up, up) > 0).float()
    return up > 0


def _places(s, k):
    """[B, Hkv, T, D] in fp32 of a cache tensor."""
    if s["table"] is None:
        return k.float()
    return k[s["table"].long()].transpose(1, 2).flatten(2, 3).float()


def _plain_tree(s):
    B, Hq, n, D = s["q"].shape
    k, v = _places(s, s["k"]), _places(s, s["v"])
    T = k.shape[2]
    j, m = _tokens(s)
    first = s["seq_lens"].long() - m  # tokens before the drafts
    t = torch.arange(T, device=k.device)
    # a place's row of the window
    row = (t.unsqueeze(0) - first.unsqueeze(1) + (n - m).unsqueeze(1)).clamp(0, n - 1)
    sees = torch.gather(_ancestors(s), 2, row.unsqueeze(1).expand(B, n, T))
    sees = sees & (t.view(1, 1, -1) >= first.view(-1, 1, 1)) & (t.view(1, 1, -1) < s["seq_lens"].view(-1, 1, 1))
    sees = sees | (t.view(1, 1, -1) < first.view(-1, 1, 1))
    q = s["q"].view(B, s["Hkv"], -1, n, D)
    x = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).view(B, s["Hkv"], -1, n, T) * (1.0 / math.sqrt(D))
    x = x.masked_fill(~sees.view(B, 1, 1, n, T), -math.inf)
    top = x.amax(-1, keepdim=True)
    some = top > -math.inf
    e = torch.exp(x - torch.where(some, top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e.flatten(2, 3), v).view(B, s["Hkv"], -1, n, D) / torch.where(some, total, torch.ones_like(total))
    lse = torch.where(some, top + torch.log(total), top)
    live = (j >= 0).view(B, 1, n)
    s["out"].copy_(torch.where(live.unsqueeze(3), out.reshape(B, Hq, n, D), s["out"]))
    s["lse"].copy_(torch.where(live, lse.reshape(B, Hq, n), s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_verify(s):
    # One walk for all sequences: a child has a higher number than its parent, so each token is looked at once.  What is
    # left of the target after k refused children is max(0, p - c q): sums and products next to a border, in 64 bits.
    B, n = s["tokens"].shape
    V = s["target"].shape[2]
    j, m = _tokens(s)
    b = torch.arange(B, device=j.device)
    at = n - m  # the row that the walk stands at
    start = at.clamp(max=n - 1)
    p = s["target"][b, start].double()
    q = s["draft"][b, start].double() if s["draft"] is not None else torch.zeros_like(p)
    c = torch.zeros(B, dtype=torch.float64, device=j.device)  # of the draft's, taken off
    left = p
    mass = torch.ones_like(c)
    path = torch.full((B, n), -1, dtype=torch.int64, device=j.device)
    path[:, 0] = torch.where(m > 0, 0, -1)
    count = (m > 0).long()
    for i in range(1, n):
        child = (j[:, i] > 0) & (s["parents"][:, i].long() + (n - m) == at)
        x, u = s["tokens"][:, i].long(), s["uniforms"][:, i].double()
        px = left[b, x]
        taken = child & (u * mass * (q[b, x] if s["draft"] is not None else 1.0) < px)
        refused = child & ~taken
        if s["draft"] is not None:
            c = torch.where(refused, c + mass, c)
        else:
            mass = torch.where(refused, mass - px, mass)
            left = torch.where(refused.unsqueeze(1) & (torch.arange(V, device=x.device) == x.unsqueeze(1)), 0.0, left)
        at = torch.where(taken, i, at)
        p = torch.where(taken.unsqueeze(1), s["target"][:, i].double(), p)
        if s["draft"] is not None:
            q = torch.where(taken.unsqueeze(1), s["draft"][:, i].double(), q)
            c = torch.where(taken, torch.zeros_like(c), c)
            left = (p - c.unsqueeze(1) * q).clamp(min=0.0)
            mass = torch.where(refused, left.sum(1), torch.where(taken, torch.ones_like(mass), mass))
        else:
            mass = torch.where(taken, torch.ones_like(mass), mass)
            left = torch.where(taken.unsqueeze(1), p, left)
        end = count.clamp(max=n - 1)
        path[b, end] = torch.where(taken, j[:, i], path[b, end])
        count = count + taken.long()
    total = left.sum(1)
    left = torch.where((total > 0).unsqueeze(1), left, p)  # nothing left: the target's own
    sums = left.cumsum(1)
    u = s["uniforms"][b, start].double()
    token = (sums <= (u * sums[:, -1]).unsqueeze(1)).sum(1)
    ids = torch.arange(V, device=j.device)
    token = torch.minimum(token, torch.where(left > 0, ids, -1).amax(1))
    token = torch.where(m > 0, token, -1)
    return {"path": path.to(torch.int32), "count": count.to(torch.int32), "token": token.to(torch.int32)}


def _plain_keep(s):
    j = torch.arange(s["n"], device=s["index"].device)
    b, i = (j.unsqueeze(0) < s["counts"].unsqueeze(1)).nonzero(as_tuple=True)
    start = s["starts"].long()[b]
    source, place = start + s["index"].long()[b, i], start + i
    if s["table"] is not None:
        page, table = s["k"].shape[2], s["table"].long()
        source, place = ((table[b, t // page], slice(None), t % page) for t in (source, place))
    else:
        source, place = (b, slice(None), source), (b, slice(None), place)
    s["k"][place] = s["k"][source]
    s["v"][place] = s["v"][source]
    return {"k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------ one pass
def run(s):
    if not own:
        return {"tree": _plain_tree, "verify": _plain_verify, "keep": _plain_keep}[s["op"]](s)
    import split_kv_decode_fd_gb300 as fd

    if s["op"] == "tree":
        out, lse = fd.decode_tree(s["q"], s["k"], s["v"], s["parents"], new_lens=s["new_lens"], seq_lens=s["seq_lens"],
                                  max_seq_len=s["max_len"], block_table=s["table"], out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    if s["op"] == "verify":
        path, count, token = fd.verify_tree(s["tokens"], s["parents"], s["target"], s["uniforms"], draft=s["draft"],
                                            new_lens=s["new_lens"])
        return {"path": path, "count": count, "token": token}
    fd.keep_rows(s["k"], s["v"], s["index"], counts=s["counts"], starts=s["starts"], block_table=s["table"])
    return {"k": s["k"], "v": s["v"]}


def work(case):
    """Lengths and counts go in with their expected sum; a multiply and an add are two operations."""
    B, n = case["B"], case["n"]
    if case["op"] == "verify":
        # the walk's rows of p and q at its last token, once each
        es = {"bf16": 2, "f32": 4}[case["probs"]]
        rows = 2 if case["draft"] else 1
        return {"bytes": B * (rows * case["V"] * es + n * 20.0), "flops": 4.0 * B * case["V"]}
    es = {"bf16": 2, "f32": 4}[case["cache"]]
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "keep":
        rows = B * (n + 1) / 2 if case["keep"] == "path" else B * n
        return {"bytes": rows * (4 + 4.0 * Hkv * D * es), "flops": 0.0}
    lo, hi = case["lo"], case["hi"] + 1.0
    mean = (hi - lo) / math.log(hi / lo)
    tokens = max(1.0, (B - 1) * mean + case["hi"])
    share = (n + 1) / 2 / n if case["ragged"] else 1.0  # of the rows that are tokens
    rows = B * case["Hq"] * n * share
    return {"bytes": 2 * tokens * Hkv * D * es + rows * (2 * D + 1) * 4.0, "flops": 4.0 * tokens * case["Hq"] * n * share * D}


# ------------------------------------------------------------------ 64 bits
def _exact_verify(s, b):
    """The walk of one sequence, child by child."""
    n, V = s["n"], s["V"]
    m = int(s["new_lens"][b]) if s["new_lens"] is not None else n
    if m == 0:
        return [], -1
    pad = n - m
    parents, words = s["parents"][b, pad:].tolist(), s["tokens"][b, pad:].tolist()
    uniforms = s["uniforms"][b, pad:].double().tolist()
    node, path, left = 0, [0], s["target"][b, pad].double()
    going = True
    while going:
        going = False
        share = left  # the target's probabilities, then what is left of them, not normalised
        mass = 1.0
        for child in (i for i in range(m) if i > node and parents[i] == node):
            x = words[child]
            if s["draft"] is not None:
                q = s["draft"][b, pad + node].double()
                ok = uniforms[child] * mass * float(q[x]) < float(share[x])
            else:
                ok = uniforms[child] * mass < float(share[x])
            if ok:
                path.append(child)
                node, left, going = child, s["target"][b, pad + child].double(), True
                break
            if s["draft"] is not None:
                share = torch.relu(share - mass * q)
                mass = float(share.sum())
            else:
                mass -= float(share[x])
                share = share.clone()
                share[x] = 0.0
        if not going:
            if not float(share.sum()) > 0:
                share = left
            sums = torch.cumsum(share, 0)
            found = int(torch.searchsorted(sums, sums[-1:] * uniforms[0], right=True))
            return path, min(found, int(torch.nonzero(share > 0).max()))


def exact(case, seed):
    s = prepare(case, seed)
    B, n = case["B"], case["n"]
    dev = s["k"].device if "k" in s else s["target"].device
    if case["op"] == "verify":
        path = torch.full((B, n), -1, dtype=torch.int32)
        count, token = torch.zeros(B, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
        for b in range(B):
            at, token[b] = _exact_verify(s, b)
            path[b, :len(at)] = torch.tensor(at, dtype=torch.int32)
            count[b] = len(at)
        return {"path": path.to(dev), "count": count.to(dev), "token": token.to(dev)}
    page = s["k"].shape[2]

    def rows_of(x, b, t):  # [heads, places, D]
        return x[b][:, t] if s["table"] is None else x[s["table"][b].long()[t // page], :, t % page].transpose(0, 1)

    if case["op"] == "keep":
        out = {}
        for name in ("k", "v"):
            x, y = s[name], s[name].double()
            for b in range(B):
                c, start = int(s["counts"][b]), int(s["starts"][b])
                got = rows_of(x, b, start + s["index"][b, :c].long()).double()
                to = torch.arange(start, start + c, device=dev)
                if s["table"] is None:
                    y[b][:, to] = got
                else:
                    y[s["table"][b].long()[to // page], :, to % page] = got.transpose(0, 1)
            out[name] = y
        return out
    Hkv, D = case["Hkv"], case["D"]
    out, lse = s["out"].double(), s["lse"].double()
    for b in range(B):
        L = int(s["seq_lens"][b])
        m = int(s["new_lens"][b]) if s["new_lens"] is not None else n
        if m == 0:
            continue
        t = torch.arange(L, device=dev)
        k, v = rows_of(s["k"], b, t).double(), rows_of(s["v"], b, t).double()
        parents = s["parents"][b, n - m:].tolist()
        sees = torch.zeros((m, L), dtype=torch.bool)
        sees[:, :L - m] = True
        for i in range(m):
            up = i
            while up >= 0:
                sees[i, L - m + up] = True
                up = parents[up]
        q = s["q"][b, :, n - m:].double().view(Hkv, -1, m, D)
        for h in range(Hkv):
            x = torch.einsum("gid,td->git", q[h], k[h]) / math.sqrt(D)
            x = torch.where(sees.to(dev), x, -math.inf)
            heads = slice(h * q.shape[1], (h + 1) * q.shape[1])
            out[b, heads, n - m:] = torch.einsum("git,td->gid", torch.softmax(x, -1), v[h])
            lse[b, heads, n - m:] = torch.logsumexp(x, -1)
    return {"out": out, "lse": lse}
