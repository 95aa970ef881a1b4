"""GPU tests of decode attention over a 4-bit cache against the float64 oracle on the cache's values.

Bound: q and p are held as sums of two fp16 numbers (22 bits), products and sums in fp32.  With A = scale * max over
keys of sum |q_d k_d|, a score is off by at most (2^-21 + D 2^-24) A in natural units, counted once for the split and
once for each fp32 sum; p by that plus 2^-20 (its split, exp2 and the running sums' ulps).  out is a weighted mean of v, so its
error is at most twice that of a weight times max |v|; lse's is that of a score plus 2^-22 of its size.
"""

import math

import numpy as np
import pytest
import torch

import oracle
import split_kv_decode_fd_gb300 as fd

pytestmark = pytest.mark.gpu
kv4 = oracle.kv4


def np64(t):
    return t.detach().double().cpu().numpy()


class Case:
    def __init__(self, B, Hq, Hkv, D, lens, *, n_q=1, page=0, cap=None, seed=0, k_exp=0, v_exp=0, q_gain=1.0):
        r = np.random.default_rng(seed)
        unit = page or 16
        cap = max(unit, -(-(cap or max(lens)) // unit) * unit)
        self.B, self.Hq, self.Hkv, self.D, self.lens, self.n_q, self.cap = B, Hq, Hkv, D, lens, n_q, cap
        self.k_exp, self.v_exp = k_exp, v_exp
        x = r.standard_normal((2, B, Hkv, cap, D))
        x[0, ..., 3::17] *= 4.0
        kc, ks = kv4.quantise(x[0])
        vc, vs = kv4.quantise(x[1])
        self.k, self.v = kv4.values(kc, ks, k_exp), kv4.values(vc, vs, v_exp)
        cut = lambda a: a.reshape(B, Hkv, cap // 16, 16, a.shape[-1])  # noqa: E731
        blocks = kv4.pack_blocks(cut(kc), cut(ks), cut(vc), cut(vs))  # [B, Hkv, cap/16, bytes]
        self.table = None
        if page:
            per = cap // page
            self.table_np = r.permutation(B * per + 2)[:B * per].reshape(B, per).astype(np.int32)
            pool = r.integers(0, 256, (B * per + 2, Hkv, page // 16, 18 * D)).astype(np.uint8)
            pool[self.table_np] = np.swapaxes(blocks.reshape(B, Hkv, per, page // 16, 18 * D), 1, 2)
            blocks = pool
            self.table = torch.from_numpy(self.table_np).cuda()
        self.page = page
        self.kv4 = torch.from_numpy(np.ascontiguousarray(blocks)).cuda()
        shape = (B, Hq, n_q, D)
        self.q = torch.from_numpy(r.standard_normal(shape).astype(np.float32) * q_gain).cuda()
        self.scale = 1.0 / math.sqrt(D)

    def run(self, n_splits=0, causal=True, **kw):
        if "seq_lens" not in kw:
            kw["seq_lens"] = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        return fd.decode_kv4(self.q, self.kv4, k_exp=self.k_exp, v_exp=self.v_exp, causal=causal,
                             max_seq_len=self.cap, block_table=self.table, scale=self.scale, n_splits=n_splits, **kw)

    def check(self, out, lse, causal=True, lens=None):
        lens = lens or self.lens
        q = np64(self.q)
        ro, rl = oracle.decode_rows(q, self.k, self.v, self.scale, causal=causal, seq_lens=lens, max_seq_len=self.cap)
        g = self.Hq // self.Hkv
        big = np.abs(self.k).max(2) if self.cap else 0  # [B, Hkv, D]
        A = self.scale * np.einsum("bhnd,bhd->bhn", np.abs(q), np.repeat(big, g, 1))
        es = (2.0 ** -21 + self.D * 2.0 ** -24) * A + 2.0 ** -20
        vm = np.repeat(np.abs(self.v).max((2, 3)), g, 1)[:, :, None]
        o, ls = np64(out), np64(lse)
        assert np.array_equal(np.isneginf(ls), np.isneginf(rl))
        fin = np.isfinite(rl)
        err = np.abs(o - ro) / (2 * es * vm)[..., None]
        assert np.all(np.isfinite(o)) and err.max() <= 1.0, err.max()
        el = np.abs(ls - np.where(fin, rl, 0))[fin] / (es + 2.0 ** -22 * np.abs(np.where(fin, rl, 0)))[fin]
        assert el.size == 0 or el.max() <= 1.0, el.max()


SHAPES = [  # B, Hq, Hkv, D, n_q, page
    (2, 4, 4, 128, 1, 0), (2, 4, 4, 64, 1, 16), (3, 8, 2, 128, 1, 16), (2, 8, 4, 64, 1, 0), (2, 24, 3, 128, 1, 48),
    (2, 32, 2, 128, 1, 0), (2, 32, 2, 64, 1, 32), (2, 10, 2, 128, 1, 0), (1, 3, 1, 64, 1, 16), (1, 34, 2, 128, 1, 64),
    (2, 8, 2, 128, 2, 16), (2, 8, 2, 64, 3, 0), (2, 4, 4, 128, 5, 0), (1, 8, 1, 128, 7, 16), (2, 2, 2, 64, 64, 0),
]


@pytest.mark.parametrize("B,Hq,Hkv,D,n_q,page", SHAPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n_splits", [0, 3])
def test_against_the_oracle(B, Hq, Hkv, D, n_q, page, causal, n_splits):
    lens = [[700, 333, 129][i % 3] for i in range(B)]
    c = Case(B, Hq, Hkv, D, lens, n_q=n_q, page=page, seed=B + Hq + D + n_q)
    out, lse = c.run(n_splits, causal)
    assert fd.workspace_status() == 0
    c.check(out, lse, causal)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,n_q", [(4, 1), (4, 4), (16, 1), (32, 2)])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("n_splits", [0, 2])
def test_lengths_of_zero_one_and_around_tiles(D, Hq, n_q, page, n_splits):
    lens = [0, 1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257]
    c = Case(len(lens), Hq, 2, D, lens, n_q=n_q, page=page, seed=D + Hq)
    c.check(*c.run(n_splits))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq", [4, 32])
@pytest.mark.parametrize("page", [0, 16])
def test_bytes_past_the_length_never_reach_a_result(D, Hq, page):
    lens = [1, 13, 16, 100, 130, 250, 0]
    c = Case(len(lens), Hq, 2, D, lens, n_q=2, page=page, cap=272, seed=D)
    out, lse = c.run()
    c.check(out, lse)
    # codes and scales of every token at or past the length become 0xff: NaN scales
    parts = [list(x) for x in [kv4.unpack_blocks(c.kv4.cpu().numpy())]][0]
    for b, L in enumerate(lens):
        for t in range(L, c.cap):
            at, row = (int(c.table_np[b, t // page]), t % page) if page else (b, t)
            for x, fill in zip(parts, (15, 255, 15, 255)):
                x[at, :, row // 16, row % 16] = fill
    c.kv4 = torch.from_numpy(kv4.pack_blocks(*parts)).cuda()
    out2, lse2 = c.run()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_nan_in_the_cache_and_in_q_shows():
    c = Case(3, 4, 2, 64, [300, 300, 300], seed=2)
    parts = list(kv4.unpack_blocks(c.kv4.cpu().numpy()))
    parts[1][0, 0, 200 // 16, 200 % 16, 1] = 0x7F  # a NaN key block of sequence 0, KV head 0
    parts[3][1, 1, 10 // 16, 10 % 16, 2] = 0x7F    # NaN values, channels 32..47 of sequence 1, KV head 1
    c.kv4 = torch.from_numpy(kv4.pack_blocks(*parts)).cuda()
    c.q[2, 3, 0, 7] = float("nan")
    for n_splits in (0, 1, 4):
        out, lse = c.run(n_splits)
        nan = torch.isnan(out[:, :, 0])
        assert torch.all(nan[0, :2]) and torch.all(torch.isnan(lse[0, :2])) and not torch.any(nan[0, 2:])
        assert torch.all(nan[1, 2:, 32:48]) and not torch.any(nan[1, 2:, :32]) and not torch.any(nan[1, :2])
        assert torch.all(nan[2, 3]) and torch.isnan(lse[2, 3, 0]) and not torch.any(nan[2, :3])


@pytest.mark.parametrize("page", [0, 16])
def test_no_lengths_no_lse_and_3d_queries(page):
    c = Case(2, 8, 2, 128, [256, 256], page=page, seed=4)
    out, lse = c.run(seq_lens=None)
    c.check(out, lse)
    o3, none = fd.decode_kv4(c.q[:, :, 0].contiguous(), c.kv4, block_table=c.table, return_lse=False)
    assert none is None and torch.equal(o3, out[:, :, 0])


def test_bad_pages_are_reported():
    c = Case(2, 4, 2, 64, [300, 200], page=16, seed=5)
    c.table[0, 3] = 1 << 20
    c.table[1, 13:] = -7  # past the length: never read
    out, lse = c.run()
    assert fd.workspace_status() == 4 and fd.workspace_status() == 0
    out1, _ = c.run(seq_lens=torch.tensor([40, 200], dtype=torch.int32, device="cuda"))
    assert fd.workspace_status() == 0 and torch.equal(out1[1], out[1])
    c.v[0, :, 48:64] = 0.0
    c.k[0, :, 48:64] = 0.0
    c.check(out, lse)


@pytest.mark.parametrize("Hq,gain", [(4, 30.0), (16, 8.0)])
def test_peaked_and_rising_scores(Hq, gain):
    c = Case(2, Hq, 2, 128, [3000, 2111], seed=6, q_gain=gain)
    c.check(*c.run())
    # scores that rise along the sequence: the running maximum moves again and again
    order = np.argsort(np.einsum("bd,bhtd->bht", np64(c.q)[:, 0, 0], c.k)[:, :1], axis=-1)
    kc, ks = kv4.quantise(np.take_along_axis(c.k, np.repeat(order, 2, 1)[..., None], 2))
    c.k = kv4.values(kc, ks)
    vc, vs = kv4.quantise(c.v)
    c.v = kv4.values(vc, vs)
    cut = lambda a: a.reshape(2, 2, c.cap // 16, 16, a.shape[-1])  # noqa: E731
    c.kv4 = torch.from_numpy(kv4.pack_blocks(cut(kc), cut(ks), cut(vc), cut(vs))).cuda()
    c.check(*c.run())


@pytest.mark.parametrize("exps", [(0, 0), (5, -7), (-20, 30)])
def test_exponents(exps):
    c = Case(2, 4, 1, 64, [500, 77], k_exp=exps[0], v_exp=exps[1], q_gain=2.0 ** -exps[0], seed=7)
    c.check(*c.run())


def test_many_sequences():
    """More sequences than the balanced plan takes, and more than there are SMs."""
    r = np.random.default_rng(1)
    for B in (300, 1100):
        lens = r.integers(0, 40, B).tolist()
        c = Case(B, 2, 1, 64, lens, page=16, seed=B)
        c.check(*c.run())


@pytest.mark.parametrize("Hq", [4, 8, 16, 32])
def test_same_bits_every_time(Hq):
    c = Case(4, Hq, 2, 128, [5000, 1, 700, 2500], page=16, seed=8)
    first = [x.clone() for x in c.run()]
    junk = Case(2, 8, 2, 64, [900, 100], seed=9)
    for _ in range(5):
        junk.run()
        got = c.run()
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    ws = fd.Workspace()
    assert all(torch.equal(a, b) for a, b in zip(first, c.run(workspace=ws)))


def test_refusals_of_the_binding():
    c = Case(2, 4, 2, 64, [32, 32], seed=1)
    with pytest.raises(ValueError, match="kv4"):
        fd.decode_kv4(c.q, c.kv4.float())
    with pytest.raises(ValueError, match="head_dim"):
        fd.decode_kv4(torch.zeros((2, 4, 128), device="cuda"), c.kv4)
    with pytest.raises(ValueError, match="sequences"):
        fd.decode_kv4(c.q[:1], c.kv4)
    with pytest.raises(ValueError, match="seq_lens"):
        c.run(seq_lens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(fd.FdError):
        fd.decode_kv4(torch.zeros((2, 2, 65, 64), device="cuda"), c.kv4)
    with pytest.raises(fd.FdError):
        fd.decode_kv4(c.q, c.kv4, max_seq_len=33)


# ------------------------------------------------------------------ together
def serve(D, page, steps, Hq=8, Hkv=2, B=3, n0=21):
    """A prompt, then single tokens: append_rope_kv4 and decode_kv4, with what the cache has to hold."""
    g = torch.Generator(device="cuda").manual_seed(D + page)
    cap = 96
    table = None
    if page:
        table = torch.randperm(B * cap // page, device="cuda", generator=g).view(B, -1).int()
    kv = fd.kv4_cache(B * cap // page if page else B, Hkv, page or cap, D)
    inv = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    ang = torch.arange(cap, dtype=torch.float64, device="cuda")[:, None] * inv
    cos, sin = ang.cos().float(), ang.sin().float()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    done = []
    for step in range(steps + 1):
        n = n0 if step == 0 else 1
        nl = torch.tensor([n0, 1, 0][:B], dtype=torch.int32, device="cuda") if step == 0 else None
        x = torch.randn((B, n, Hq + 2 * Hkv, D), device="cuda", generator=g).bfloat16()
        q = fd.append_rope_kv4(x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], kv, cos, sin, q=x[:, :, :Hq], new_lens=nl,
                               seq_lens=lens, max_seq_len=cap - n, block_table=table)
        lens = lens + (n if nl is None else nl)
        out, lse = fd.decode_kv4(q, kv, seq_lens=lens, max_seq_len=cap, block_table=table)
        done.append((q, out, lse, lens.tolist()))
    return kv, table, done


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [0, 16])
def test_a_serving_loop(D, page):
    kv, table, done = serve(D, page, 12)
    k, v = fd.kv4_read(kv, 96, block_table=table, dtype=torch.float32)
    assert fd.workspace_status() == 0
    c = Case.__new__(Case)
    c.Hq, c.Hkv, c.D, c.cap, c.scale = 8, 2, D, 96, 1.0 / math.sqrt(D)
    c.k, c.v = np64(k), np64(v)
    for step, (q, out, lse, lens) in enumerate(done):
        c.q = q
        c.check(out, lse, lens=lens)


def test_on_another_stream_and_captured():
    c = Case(3, 16, 4, 128, [900, 33, 512], page=16, seed=3)
    want = [x.clone() for x in c.run()]
    s = torch.cuda.Stream()
    ws = fd.Workspace()
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    c.run(out=out, lse=lse, workspace=ws, stream=s, seq_lens=lens)
    s.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=out, lse=lse, workspace=ws, seq_lens=lens)
    for L in ([900, 33, 512], [1, 0, 700]):
        lens.copy_(torch.tensor(L, dtype=torch.int32))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, lse, lens=L)
    with pytest.raises(RuntimeError, match="capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            c.run(out=out, lse=lse, workspace=fd.Workspace(), seq_lens=lens)
