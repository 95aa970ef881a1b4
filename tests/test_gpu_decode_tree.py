"""GPU tests of attention for trees of drafted tokens against the float64 oracle.

Bound: products of q and k are exact or rounded once, sums are fp32.  With A = scale * max over keys of sum |q_d k_d|, a
score is off by at most (2^-21 + D 2^-24) A in natural units, a weight by that and 2^-20 (exp2, the running sums' ulps).  out is a
weighted mean of v, so that moves it by at most twice as much times max |v|, and the sums of p v by at most 2^-23 for each of
the 24 products of a tile of 128 keys and for each tile.  lse is off as a score is, plus 2^-22 of its size.
"""

import math

import numpy as np
import pytest
import torch

import oracle
import split_kv_decode_fd_gb300 as fd

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def np64(t):
    return t.detach().double().cpu().numpy()


def a_tree(r, m, shape):
    j = np.arange(m)
    if shape == "chain":
        p = j - 1
    elif shape == "wide":
        p = np.zeros(m, dtype=int)
    elif shape == "roots":  # no first token: every draft follows the sequence
        return -np.ones(m, dtype=np.int32)
    else:
        p = np.array([r.integers(0, max(1, x)) for x in j])
    if m:
        p[0] = -1
    return p.astype(np.int32)


class Case:
    def __init__(self, B, Hq, Hkv, D, n, lens, *, new_lens=None, cache="bf16", page=0, cap=None, seed=0, shape="random",
                 gain=1.0, scale=None):
        r = np.random.default_rng(seed)
        unit = page or 16
        cap = max(unit, -(-(cap or max(lens)) // unit) * unit)
        self.B, self.Hq, self.Hkv, self.D, self.n, self.lens, self.new_lens, self.cap, self.page = B, Hq, Hkv, D, n, lens, new_lens, cap, page
        k, v = (torch.from_numpy(r.standard_normal((B, Hkv, cap, D)).astype(np.float32)).to(TYPES[cache]) for _ in range(2))
        self.k_np, self.v_np = k.float().numpy(), v.float().numpy()
        self.table = self.table_np = None
        if page:
            per = cap // page
            self.table_np = r.permutation(B * per + 2)[:B * per].reshape(B, per).astype(np.int32)
            self.table = torch.from_numpy(self.table_np).cuda()
            pools = []
            for x in (k, v):
                pool = torch.full((B * per + 2, Hkv, page, D), math.nan, dtype=x.dtype)
                pool[torch.from_numpy(self.table_np).long()] = x.view(B, Hkv, per, page, D).transpose(1, 2)
                pools.append(pool.cuda())
            self.k, self.v = pools
        else:
            self.k, self.v = k.cuda(), v.cuda()
        self.parents_np = np.full((B, n), 1 << 20, dtype=np.int32)  # padding rows hold anything
        for b in range(B):
            m = n if new_lens is None else new_lens[b]
            self.parents_np[b, n - m:] = a_tree(r, m, shape)
        self.parents = torch.from_numpy(self.parents_np).cuda()
        self.q = torch.from_numpy((r.standard_normal((B, Hq, n, D)) * gain).astype(np.float32)).cuda()
        self.scale = 1.0 / math.sqrt(D) if scale is None else scale

    def place(self, b, t):
        """Index of place t of sequence b in the cache tensors."""
        return (b, slice(None), t) if not self.page else (int(self.table_np[b, t // self.page]), slice(None), t % self.page)

    def run(self, **kw):
        kw.setdefault("max_seq_len", self.cap)
        if "new_lens" not in kw and self.new_lens is not None:
            kw["new_lens"] = torch.tensor(self.new_lens, dtype=torch.int32, device="cuda")
        if "seq_lens" not in kw:
            kw["seq_lens"] = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        return fd.decode_tree(self.q, self.k, self.v, kw.pop("parents", self.parents), block_table=self.table, scale=self.scale, **kw)

    def check(self, out, lse):
        ro, rl = oracle.tree.attend(np64(self.q), self.k_np, self.v_np, self.parents_np, self.lens, self.new_lens, self.scale)
        g = self.Hq // self.Hkv
        live = ~np.isnan(rl)
        big = np.abs(self.k_np).max(2)
        A = abs(self.scale) * np.einsum("bhnd,bhd->bhn", np.abs(np64(self.q)), np.repeat(big, g, 1))
        es = (2.0 ** -21 + self.D * 2.0 ** -24) * A + 2.0 ** -20
        vm = np.repeat(np.abs(self.v_np).max((2, 3)), g, 1)[:, :, None]
        o, ls = np64(out), np64(lse)
        bound = 2 * es * vm + (24 + self.cap / 128) * 2.0 ** -23 * vm
        assert np.all(np.isfinite(o[live]))
        err = (np.abs(o - np.where(np.isnan(ro), 0, ro)) / bound[..., None])[live]
        assert err.size == 0 or err.max() <= 1.0, err.max()
        fin = live & np.isfinite(rl)
        assert np.array_equal(np.isneginf(ls[live]), np.isneginf(rl[live]))
        el = np.abs(ls - rl)[fin] / (es + 2.0 ** -22 * np.abs(rl))[fin]
        assert el.size == 0 or el.max() <= 1.0, el.max()


def exact_on_the_gpu(c):
    """The oracle's formulas in 64 bits in torch, for cases that are large: out and lse (NaN in padding rows)."""
    out, lse = (torch.full(x, math.nan, dtype=torch.float64, device="cuda") for x in (c.q.shape, c.q.shape[:3]))
    for b, L in enumerate(c.lens):
        m = c.n if c.new_lens is None else c.new_lens[b]
        if m == 0:
            continue
        k, v = (torch.from_numpy(x[b, :, :L]).double().cuda() for x in (c.k_np, c.v_np))
        sees = torch.ones((m, L), dtype=torch.bool)
        tree = torch.from_numpy(oracle.tree.ancestors(c.parents_np[b, c.n - m:]))
        first = max(0, L - m)
        sees[:, first:] = tree[:, m - (L - first):]
        q = c.q[b, :, c.n - m:].double().view(c.Hkv, -1, m, c.D)
        x = torch.einsum("hgid,htd->hgit", q, k) * c.scale
        x = x.masked_fill(~sees.cuda(), -math.inf)
        out[b, :, c.n - m:] = torch.nan_to_num(torch.einsum("hgit,htd->hgid", torch.softmax(x, -1), v), 0.0).reshape(-1, m, c.D)
        lse[b, :, c.n - m:] = torch.logsumexp(x, -1).reshape(-1, m)
    return out, lse


SHAPES = [  # B, Hq, Hkv, D, n, page
    (2, 4, 4, 128, 1, 0), (2, 4, 4, 64, 5, 16), (3, 8, 2, 128, 8, 16), (2, 8, 4, 64, 3, 0), (2, 24, 3, 128, 7, 48),
    (1, 32, 2, 128, 8, 0), (1, 32, 2, 64, 9, 32), (2, 10, 2, 128, 13, 0), (1, 3, 1, 64, 64, 16), (1, 34, 2, 128, 31, 64),
    (1, 8, 1, 128, 16, 0), (1, 8, 1, 128, 17, 16), (1, 16, 1, 64, 64, 0),
]


@pytest.mark.parametrize("B,Hq,Hkv,D,n,page", SHAPES)
@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("shape", ["chain", "random"])
@pytest.mark.parametrize("ragged", [False, True])
def test_against_the_oracle(B, Hq, Hkv, D, n, page, cache, shape, ragged):
    lens = [[701, 333, 129][i % 3] for i in range(B)]
    new_lens = [[max(1, n // 2), n, 1][i % 3] for i in range(B)] if ragged else None
    c = Case(B, Hq, Hkv, D, n, lens, new_lens=new_lens, cache=cache, page=page, shape=shape, seed=B + Hq + D + n)
    out, lse = c.run()
    assert fd.workspace_status() == 0
    c.check(out, lse)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,n", [(4, 1), (4, 9), (32, 16)])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_lengths_of_zero_one_and_around_tiles(D, Hq, n, page, cache):
    """Sequences shorter than their drafts among them: tokens whose place is below 0 see nothing."""
    lens = [0, 1, 2, 15, 16, 17, 127, 128, 129, 135, 255, 256, 257, 264]
    c = Case(len(lens), Hq, 2, D, n, lens, page=page, cache=cache, seed=D + Hq)
    c.check(*c.run())
    c.new_lens = [b % (n + 1) for b in range(len(lens))]
    r = np.random.default_rng(1)
    for b, m in enumerate(c.new_lens):
        c.parents_np[b, n - m:] = a_tree(r, m, "random")
    c.parents = torch.from_numpy(c.parents_np).cuda()
    c.check(*c.run())
    assert fd.workspace_status() == 0


@pytest.mark.parametrize("shape", ["wide", "roots"])
@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_wide_trees(shape, cache):
    c = Case(2, 8, 2, 128, 40, [500, 40], cache=cache, shape=shape, seed=4)
    c.check(*c.run())


@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_one_tree_for_all_and_lengths_that_are_all_alike(cache):
    c = Case(3, 8, 4, 64, 12, [384] * 3, cache=cache, seed=5)
    c.parents_np[:] = c.parents_np[0]
    c.parents = torch.from_numpy(c.parents_np).cuda()
    out, lse = c.run()
    c.check(out, lse)
    out2, lse2 = c.run(parents=c.parents[0].contiguous())
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    c.check(*c.run(seq_lens=None, max_seq_len=384))


@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hkv,n,lens", [
    (1, 1, 6, [9000]), (1, 2, 40, [5000]), (3, 1, 3, [1, 6000, 130]), (5, 2, 4, [1100, 20, 2900, 0, 640]),
])
def test_sequences_cut_over_many_shares(B, Hkv, n, lens, cache):
    c = Case(B, 4 * Hkv, Hkv, 128, n, lens, cache=cache, page=16, seed=n)
    c.check(*c.run())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [0, 16, 32])
@pytest.mark.parametrize("g,n", [(1, 5), (2, 32), (2, 33), (2, 64), (3, 64), (8, 64)])
@pytest.mark.parametrize("most", [130, 700, 6000])
def test_many_pieces_and_blocks_of_rows(D, page, g, n, most):
    """CTAs with many pieces, of one tile and of many, for one block of rows and for several."""
    r = np.random.default_rng(most + n)
    B, Hkv = (150, 2) if most < 1000 else (24, 2)
    lens = r.integers(0, most, B).tolist()
    c = Case(B, g * Hkv, Hkv, D, n, lens, page=page, seed=most + n, new_lens=[int(x) for x in r.integers(0, n + 1, B)])
    for _ in range(3):
        out, lse = c.run()
    assert fd.workspace_status() == 0
    ro, rl = exact_on_the_gpu(c)
    live = ~torch.isnan(rl)
    # scores of some units and values of a few, as in the bound above: 2 es vm + ... is below 1e-4 here
    assert (out.double() - ro)[live].abs().max() < 1e-4
    fin = live & torch.isfinite(rl)
    assert torch.equal(torch.isneginf(lse[live]), torch.isneginf(rl[live])) and (lse.double() - rl)[fin].abs().max() < 1e-4
    norm = (out.double() - ro)[live].norm() / ro[live].norm()
    assert norm < 2e-6, norm  # rounding errors of fp32 sums, unbiased: some 4e-7


@pytest.mark.parametrize("D,page", [(64, 0), (128, 16)])
@pytest.mark.parametrize("g,n", [(1, 5), (2, 33), (8, 64)])
@pytest.mark.parametrize("most", [100, 700, 6000])
@pytest.mark.parametrize("uniform", [False, True])
def test_blocks_of_token_rows_over_an_fp32_cache(D, page, g, n, most, uniform):
    """Blocks of rows that are pairs of their own, and that a sequence of few tokens does not have."""
    r = np.random.default_rng(most + n)
    B, Hkv = (150, 2) if most < 1000 else (10, 2)
    lens = [most] * B if uniform else r.integers(0, most, B).tolist()
    c = Case(B, g * Hkv, Hkv, D, n, lens, page=page, cache="f32", seed=most + n,
             new_lens=None if uniform else [int(x) for x in r.integers(0, n + 1, B)])
    out, lse = c.run(seq_lens=None, max_seq_len=most) if uniform else c.run()
    assert fd.workspace_status() == 0
    ro, rl = exact_on_the_gpu(c)
    live = ~torch.isnan(rl)
    # as above: the bound of the head of this file is below 1e-4 here
    assert (out.double() - ro)[live].abs().max() < 1e-4
    fin = live & torch.isfinite(rl)
    assert torch.equal(torch.isneginf(lse[live]), torch.isneginf(rl[live])) and (lse.double() - rl)[fin].abs().max() < 1e-4
    norm = (out.double() - ro)[live].norm() / ro[live].norm()
    assert norm < 2e-6, norm


@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,n", [(4, 5), (8, 30), (8, 64)])
def test_tokens_without_lengths_and_more_tokens_than_places(Hq, n, cache):
    """new_lens without seq_lens: every sequence has max_seq_len places, here fewer than some have tokens."""
    for T in (1, 40, 333):
        c = Case(4, Hq, 2, 128, n, [T] * 4, new_lens=[0, 1, n // 2, n], cap=336, cache=cache, seed=T)
        c.check(*c.run(seq_lens=None, max_seq_len=T))
        assert fd.workspace_status() == 0


@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_a_large_batch_of_short_sequences(cache):
    r = np.random.default_rng(0)
    B, n = 1500, 3
    lens = r.integers(0, 200, B).tolist()
    new_lens = r.integers(0, n + 1, B).tolist()
    c = Case(B, 2, 1, 64, n, lens, new_lens=new_lens, cache=cache, page=16, seed=3)
    c.check(*c.run())


@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_a_token_does_not_see_may_be_anything(cache, page, bad):
    """Places past the length, unseen drafts and rows of padding hold NaN or infinities."""
    n, lens, new_lens = 7, [300, 130, 5, 128], [7, 4, 5, 0]
    c = Case(4, 8, 2, 128, n, lens, new_lens=new_lens, cache=cache, page=page, cap=320, seed=6)
    ref = c.run()
    c.check(*ref)
    for b, L in enumerate(lens):
        for t in range(L, c.cap):
            c.k[c.place(b, t)], c.v[c.place(b, t)] = bad, bad
        c.q[b, :, :n - new_lens[b]] = bad
    out, lse = c.run()
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    # the last token of each sequence is a leaf: only its own row sees it
    for b, L in enumerate(lens):
        if new_lens[b]:
            c.k[c.place(b, L - 1)], c.v[c.place(b, L - 1)] = bad, bad
    out, lse = c.run()
    for b in range(4):
        assert torch.equal(out[b, :, :n - 1], ref[0][b, :, :n - 1]) and torch.equal(lse[b, :, :n - 1], ref[1][b, :, :n - 1])


@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_bad_values_that_a_token_sees_show(cache):
    c = Case(3, 4, 2, 128, 6, [300, 300, 300], cache=cache, seed=7)
    c.parents_np[:] = [-1, 0, 0, 1, 2, 3]
    c.parents = torch.from_numpy(c.parents_np).cuda()
    ref, _ = c.run()
    c.v[0, 0, 300 - 6 + 1, 5] = math.nan  # token 1 of sequence 0: seen by tokens 1, 3, 5
    c.v[1, 1, 300 - 6 + 2, 100] = math.inf  # token 2 of sequence 1: seen by tokens 2, 4
    c.v[2, 0, 17, 3] = math.nan  # before the drafts: seen by all
    out, lse = c.run()
    o, f = out.cpu(), ref.cpu()
    assert torch.isnan(o[0, :2, [1, 3, 5], 5]).all() and torch.isposinf(o[1, 2:, [2, 4], 100]).all()
    assert torch.isnan(o[2, :2, :, 3]).all()
    for b, heads, rows, d in ((0, [0, 1], [1, 3, 5], 5), (1, [2, 3], [2, 4], 100), (2, [0, 1], range(6), 3)):
        for h in heads:
            for i in rows:
                f[b, h, i, d] = o[b, h, i, d]
    assert torch.equal(torch.nan_to_num(o, 7.0, 8.0), torch.nan_to_num(f, 7.0, 8.0)) and torch.isfinite(lse).all()
    c.k[0, 1, 300 - 6 + 1, 0] = math.nan
    _, lse = c.run()
    seen = torch.zeros(6, dtype=torch.bool)
    seen[[1, 3, 5]] = True
    assert torch.equal(torch.isnan(lse[0, 2:].cpu()), seen.expand(2, 6)) and torch.isfinite(lse[0, :2]).all()


@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_padding_rows_are_left_as_they_were(cache):
    c = Case(3, 4, 2, 64, 5, [200, 3, 0], new_lens=[2, 0, 4], cache=cache, seed=8)
    out = torch.full((3, 4, 5, 64), 77.0, device="cuda")
    lse = torch.full((3, 4, 5), 78.0, device="cuda")
    c.run(out=out, lse=lse)
    c.check(out, lse)
    for b, m in enumerate(c.new_lens):
        assert (out[b, :, :5 - m] == 77.0).all() and (lse[b, :, :5 - m] == 78.0).all()
    assert (out[2, :, 1:] == 0).all() and torch.isneginf(lse[2, :, 1:]).all()
    made, made_lse = c.run()
    assert (made[0, :, :3] == 0).all() and (made_lse[0, :, :3] == 0).all()


@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("gain,scale", [(40.0, None), (1.0, -0.2), (1.0, 0.0), (1e-3, 30.0)])
def test_large_scores_and_any_scale(gain, scale, cache):
    c = Case(2, 8, 2, 128, 6, [700, 300], cache=cache, gain=gain, scale=scale, seed=9)
    c.check(*c.run())


@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_scores_that_rise_along_the_sequence(cache):
    c = Case(1, 4, 1, 128, 4, [2000], cache=cache, seed=10)
    c.k_np = (c.k_np * np.linspace(0.1, 8, c.cap)[None, None, :, None]).astype(np.float32)
    c.k = torch.from_numpy(c.k_np).to(TYPES[cache]).cuda()
    c.k_np = c.k.float().cpu().numpy()
    c.check(*c.run())


@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_bad_parents_and_pages_are_reported(cache):
    c = Case(2, 4, 2, 64, 4, [100, 60], cache=cache, page=16, seed=11)
    ref = c.run()
    for bad in (2, 3, -2, 1 << 30, -(1 << 31)):
        p = c.parents_np.copy()
        p[0, 2] = bad
        out, lse = c.run(parents=torch.from_numpy(p).cuda())
        assert fd.workspace_status() == fd.fdecode.FD_ERR_BAD_INDEX
        assert torch.equal(out[1], ref[0][1]) and torch.equal(lse[1], ref[1][1])
        p[0, 2] = -1  # counts as none
        want = c.run(parents=torch.from_numpy(p).cuda())
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and fd.workspace_status() == 0
    table = c.table.clone()
    for bad in (-1, c.k.shape[0], 1 << 30):
        table[0, 3] = bad
        out, lse = fd.decode_tree(c.q, c.k, c.v, c.parents, seq_lens=torch.tensor(c.lens, dtype=torch.int32, device="cuda"),
                                  max_seq_len=c.cap, block_table=table)
        assert fd.workspace_status() == fd.fdecode.FD_ERR_BAD_INDEX
        assert torch.equal(out[1], ref[0][1]) and torch.equal(lse[1], ref[1][1])
    assert fd.workspace_status() == 0


@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_deterministic_on_another_stream_and_captured(cache):
    c = Case(3, 8, 2, 128, 8, [3000, 900, 77], cache=cache, page=16, seed=12)
    out, lse = c.run()
    s = torch.cuda.Stream()
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    other = c.run(seq_lens=lens, stream=s)
    s.synchronize()
    assert torch.equal(out, other[0]) and torch.equal(lse, other[1])
    ws = fd.Workspace()
    o, l = torch.empty_like(out), torch.empty_like(lse)
    c.run(seq_lens=lens, out=o, lse=l, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(seq_lens=lens, out=o, lse=l, workspace=ws)
    for _ in range(3):
        o.zero_()
        l.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(lse, l)
    assert fd.workspace_status(ws) == 0


def test_a_workspace_shared_with_other_calls():
    """Counters of the decode and the states of this call lie apart."""
    ws = fd.Workspace()
    c = Case(2, 8, 2, 128, 8, [3000, 900], seed=13)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    ref, _ = c.run()
    want, _ = fd.decode(c.q[:, :, 0].contiguous(), c.k, c.v, seq_lens=lens)
    for _ in range(3):
        out, _ = c.run(workspace=ws)
        got, _ = fd.decode(c.q[:, :, 0].contiguous(), c.k, c.v, seq_lens=lens, workspace=ws)
        assert torch.equal(out, ref) and torch.equal(got, want)
    assert fd.workspace_status(ws) == 0


@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_offsets_past_32_bits(cache):
    """A pool of more than 2^31 elements, of which the first and the last pages are used."""
    D, page = 128, 64
    pages = (1 << 31) // (page * D) + 40
    c = Case(1, 4, 1, D, 5, [40 * page - 3], cache=cache, seed=14)
    per = 40
    table = torch.arange(per, dtype=torch.int32)
    table[1::2] = pages - 1 - torch.arange(per // 2, dtype=torch.int32)
    k, v = (torch.empty((pages, 1, page, D), dtype=TYPES[cache], device="cuda") for _ in range(2))
    k[table.long().cuda()] = c.k.view(per, 1, page, D)
    v[table.long().cuda()] = c.v.view(per, 1, page, D)
    want = c.run()
    c.k, c.v, c.table = k, v, table.view(1, per).cuda()
    out, lse = c.run()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    c.check(out, lse)


def test_refusals():
    c = Case(2, 8, 2, 64, 4, [100, 60], seed=15)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    call = lambda **kw: fd.decode_tree(**{**dict(q=c.q, k=c.k, v=c.v, parents=c.parents, seq_lens=lens), **kw})  # noqa: E731
    call()
    for kw in (dict(q=c.q.cpu()), dict(q=c.q.double()), dict(q=c.q[:, :, 0]), dict(q=c.q.transpose(0, 1)),
               dict(parents=c.parents.long()), dict(parents=c.parents[:, :3]), dict(parents=c.parents.cpu()),
               dict(parents=c.parents[0, :3]), dict(new_lens=lens[:1]), dict(seq_lens=lens.float()), dict(k=c.k.half(), v=c.v.half()),
               dict(v=c.v[:, :, :-16]), dict(out=torch.empty(2, 8, 4, 32, device="cuda")), dict(lse=torch.empty(2, 8, device="cuda")),
               dict(q=c.q[:1]), dict(max_seq_len=1 << 32), dict(parents=None)):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(max_seq_len=c.cap + 1), dict(max_seq_len=-1), dict(q=torch.empty(2, 7, 4, 64, device="cuda")),
               dict(q=torch.empty(2, 8, 65, 64, device="cuda"), parents=torch.zeros(2, 65, dtype=torch.int32, device="cuda"))):
        with pytest.raises(fd.FdError):
            call(**kw)
