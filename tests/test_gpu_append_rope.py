"""GPU tests of the rotating append (bf16, fp32 and 4-bit caches) and of reading a 4-bit cache back.

Bounds, with u = 2^-24 (fp32 rounds by at most half a step): a turned channel is fma(a, c, -(b s)), so its error is at
most u |b s| + u |a c - b s| <= 2 u (|a c| + |b s|).  A bf16 cache adds half a step of bf16, 2^-8 of the value.  A code
of a 4-bit cache is that of a value within the fp32 error, on the scale of an amax within it; values that are not
turned are exact, and so are their codes and scales.
"""

import numpy as np
import pytest
import torch

import oracle
import split_kv_decode_fd_gb300 as fd

pytestmark = pytest.mark.gpu
kv4 = oracle.kv4
U = 2.0 ** -24


def np64(t):
    return t.detach().double().cpu().numpy()


def tables(max_pos, rot, dev="cuda"):
    if rot == 0:
        return None, None
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return a.cos().float().to(dev), a.sin().float().to(dev)


class Setup:
    """New rows of a batch and a cache of random bytes, as the library and the oracle take them."""

    def __init__(self, B, n, Hq, Hkv, D, cache, *, new="bf16", page=0, rot=None, interleaved=False, lens=None,
                 new_lens=None, positions=False, cap=96, k_exp=0, v_exp=0, seed=0, scale=1.0):
        self.B, self.n, self.Hq, self.Hkv, self.D, self.cache = B, n, Hq, Hkv, D, cache
        self.page, self.inter, self.k_exp, self.v_exp = page, interleaved, k_exp, v_exp
        self.rot = D if rot is None else rot
        g = torch.Generator().manual_seed(seed)
        if page:
            cap = -(-cap // page) * page
        self.cap = cap
        dt = torch.bfloat16 if new == "bf16" else torch.float32
        # slices of one fused projection: strided rows
        qkv = (torch.randn((B, n, Hq + 2 * Hkv, D), generator=g) * scale).to(dt).cuda()
        self.q, self.k_new, self.v_new = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        self.lens = lens if lens is not None else torch.randint(0, cap - n + 1, (B,), generator=g).tolist()
        self.new_lens = new_lens
        max_pos = cap + 7
        self.cos, self.sin = tables(max_pos, self.rot)
        self.positions = torch.randint(0, max_pos, (B, n), generator=g).int().cuda() if positions else None
        self.table = None
        if page:
            self.table = torch.randperm(B * cap // page + 3, generator=g)[:B * cap // page].view(B, -1).int().cuda()
        num = B * cap // page + 3 if page else B
        unit = page or cap
        if cache == "4bit":
            self.kv = torch.randint(0, 256, (num, Hkv, unit // 16, 18 * D), generator=g, dtype=torch.uint8).cuda()
        else:
            ct = torch.bfloat16 if cache == "bf16" else torch.float32
            self.kv = [torch.randn((num, Hkv, unit, D), generator=g).to(ct).cuda() for _ in range(2)]

    def call(self, **kw):
        i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        how = dict(q=self.q if self.Hq else None, interleaved=self.inter, positions=self.positions,
                   new_lens=i32(self.new_lens), seq_lens=i32(self.lens), max_seq_len=self.cap - self.n,
                   block_table=self.table)
        how.update(kw)
        if self.cache == "4bit":
            return fd.append_rope_kv4(self.k_new, self.v_new, self.kv, self.cos, self.sin, k_exp=self.k_exp,
                                      v_exp=self.v_exp, **how)
        return fd.append_rope(self.k_new, self.v_new, self.kv[0], self.kv[1], self.cos, self.sin, **how)

    def tokens(self):
        """(b, row, place, position) of every token."""
        for b in range(self.B):
            nl = self.n if self.new_lens is None else self.new_lens[b]
            for j in range(nl):
                i = self.n - nl + j
                t = self.lens[b] + j
                yield b, i, t, t if self.positions is None else int(self.positions[b, i])

    def turned(self, x, b, i, pos):
        """Row (b, i) of x turned, and its error bound: [heads, D] both."""
        r = np64(x[b, i])
        if self.rot == 0:
            return r, np.zeros_like(r)
        c, s = np64(self.cos[pos]), np64(self.sin[pos])
        big = kv4.rotate(np.abs(r), np.abs(c), -np.abs(s), self.inter)  # |a c| + |b s| in the first halves
        big2 = kv4.rotate(np.abs(r), np.abs(c), np.abs(s), self.inter)  # ... and in the second
        err = 2 * U * np.maximum(np.abs(big), np.abs(big2))
        err[:, self.rot:] = 0
        return kv4.rotate(r, c, s, self.inter), err

    def place(self, b, t):
        """Index of token t's row (block and row of it) in the cache."""
        if self.page:
            return int(self.table[b, t // self.page]), t % self.page
        return b, t


def check_rows(s, before, got):
    """bf16 / fp32 caches: written rows within the bound, every other row bit for bit as before."""
    seen = np.zeros(before[0].shape[:1] + before[0].shape[2:3], dtype=bool)
    k, v = [np64(x) for x in got]
    half = 2.0 ** -8 if s.cache == "bf16" else 2.0 ** -24
    for b, i, t, pos in s.tokens():
        at, row = s.place(b, t)
        seen[at, row] = True
        want, err = s.turned(s.k_new, b, i, pos)
        assert np.all(np.abs(k[at, :, row] - want) <= err + half * (np.abs(want) + err)), (b, i)
        want = np64(s.v_new[b, i])
        tol = 0 if s.v_new.dtype == got[1].dtype or s.cache == "f32" else half * np.abs(want)
        assert np.all(np.abs(v[at, :, row] - want) <= tol), (b, i)
    for x, y in zip(before, got):
        keep = torch.from_numpy(~seen).cuda()[:, None, :, None].expand(x.shape)
        assert torch.equal(x[keep], y[keep])


def code_range(y, err, scale):
    """Values that codes of y - err and y + err stand for on the scale."""
    r = np.where(scale > 0, 1.0 / np.where(scale > 0, scale, 1.0), 0.0)
    val = lambda z: kv4.values(kv4.e2m1_nearest(z), np.full(z.shape[:-1] + (z.shape[-1] // 16,), 0x38))  # noqa: E731
    return val((y - err) * r), val((y + err) * r)


def check_4bit(s, before, got):
    """Written rows on the scale and codes of their values within the bound, every other bit as before."""
    D = s.D
    parts = [list(kv4.unpack_blocks(x.cpu().numpy())) for x in (before, got)]
    kc, ks, vc, vs = parts[1]
    for b, i, t, pos in s.tokens():
        at, row = s.place(b, t)
        blk, r = row // 16, row % 16
        want, err = s.turned(s.k_new, b, i, pos)
        want, err = want * 2.0 ** -s.k_exp, err * 2.0 ** -s.k_exp
        sf = ks[at, :, blk, r]
        big = np.abs(want).reshape(s.Hkv, -1, 16)
        e = err.reshape(s.Hkv, -1, 16).max(-1)
        lo, hi = kv4.e4m3_nearest(np.maximum(big.max(-1) - e, 0) / 6 * (1 - U)), kv4.e4m3_nearest((big.max(-1) + e) / 6 * (1 + U))
        exact = e == 0
        lo[exact], hi[exact] = (kv4.e4m3_nearest(big.max(-1) / 6)[exact],) * 2
        assert np.all((sf >= lo) & (sf <= hi)), (b, i)
        scale = np.repeat(kv4.e4m3_value(sf), 16, -1)
        wide = np.where(err > 0, err + 2 * U * np.abs(want), 0.0)  # the quotient of turned channels rounds too
        low, high = code_range(want, wide, scale)
        val = kv4.values(kc[at, :, blk, r], np.full(sf.shape, 0x38))
        known = np.repeat(sf != 0x7F, 16, -1)  # under a NaN scale the codes say nothing
        assert np.all(((val >= low) & (val <= high))[known]), (b, i)
        c, f = kv4.quantise(np64(s.v_new[b, i]), s.v_exp)
        assert np.array_equal(vs[at, :, blk, r], f) and np.array_equal(vc[at, :, blk, r], c), (b, i)
        for o, w in zip(parts[0], parts[1]):  # what was checked is taken out of the comparison below
            o[at, :, blk, r] = w[at, :, blk, r]
    for o, w in zip(parts[0], parts[1]):
        assert np.array_equal(o, w)


def check(s, **kw):
    before = s.kv.clone() if s.cache == "4bit" else [x.clone() for x in s.kv]
    q = s.call(**kw)
    torch.cuda.synchronize()
    assert fd.workspace_status() == 0
    (check_4bit if s.cache == "4bit" else check_rows)(s, before, s.kv)
    live = set()
    for b, i, _, pos in s.tokens():
        live.add((b, i))
        if s.Hq:
            want, err = s.turned(s.q, b, i, pos)
            assert np.all(np.abs(np64(q[b, :, i]) - want) <= err)
    if s.Hq and "q_out" not in kw:
        for b in range(s.B):
            for i in range(s.n):
                if (b, i) not in live:
                    assert torch.all(q[b, :, i] == 0)
    return q


CACHES = ["bf16", "f32", "4bit"]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("page", [0, 48])
def test_types_and_layouts(cache, D, new, interleaved, page):
    check(Setup(3, 19, 6, 2, D, cache, new=new, interleaved=interleaved, page=page, seed=D + page))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("D,rot", [(64, 0), (64, 32), (128, 0), (128, 32), (128, 64), (128, 96)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_part_of_the_channels_turned(cache, D, rot, interleaved):
    check(Setup(2, 5, 3, 1, D, cache, rot=rot, interleaved=interleaved, seed=rot))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("n,lens", [(1, [0, 1, 15, 16, 17, 95]), (2, [0, 14, 15, 31, 94, 33]), (16, [0, 16, 1, 15, 80, 40]),
                                    (17, [0, 16, 79, 31, 15, 2]), (96, [0] * 6)])
@pytest.mark.parametrize("page", [0, 16])
def test_places_around_block_and_page_ends(cache, n, lens, page):
    check(Setup(6, n, 2, 2, 64, cache, lens=lens, page=page, seed=n))


@pytest.mark.parametrize("cache", CACHES)
def test_padded_rows_are_neither_read_nor_written(cache):
    s = Setup(5, 7, 4, 2, 128, cache, new_lens=[0, 1, 7, 3, 6], page=16, positions=True, seed=3)
    for b, nl in enumerate(s.new_lens):  # padding holds NaN and positions outside the tables
        for x in (s.q, s.k_new, s.v_new):
            x[b, :7 - nl] = float("nan")
        s.positions[b, :7 - nl] = 1 << 30
    check(s)
    mark = torch.full((5, 4, 7, 128), 7.0, device="cuda")
    q = check(s, q_out=mark)
    assert q is mark
    for b, nl in enumerate(s.new_lens):
        assert torch.all(mark[b, :, :7 - nl] == 7.0)


@pytest.mark.parametrize("cache", CACHES)
def test_without_queries_and_with_lengths_past_the_range(cache):
    s = Setup(3, 4, 0, 2, 64, cache, lens=[5, 92, 0], seed=9)
    lens = torch.tensor([5, 4000, -3], dtype=torch.int32, device="cuda")  # clamped to [0, 92]
    assert check(s, seq_lens=lens) is None


@pytest.mark.parametrize("cache", CACHES)
def test_broadcast_rows(cache):
    s = Setup(3, 4, 2, 2, 64, cache, seed=4)
    s.k_new = s.k_new[:1, :, :1].expand(3, 4, 2, 64)  # one head for all: strides of 0
    s.v_new = s.v_new[:1, :, :1].expand(3, 4, 2, 64)
    check(s)


@pytest.mark.parametrize("exps", [(0, 0), (3, -4), (-64, 64)])
@pytest.mark.parametrize("scale", [1.0, 1e-3, 600.0])
def test_exponents_and_small_or_large_values(exps, scale):
    check(Setup(2, 20, 1, 2, 64, "4bit", k_exp=exps[0], v_exp=exps[1], scale=scale, rot=32, seed=5))


def test_nan_and_infinity_into_a_4bit_cache():
    s = Setup(1, 3, 0, 1, 64, "4bit", rot=0, lens=[6], seed=6)
    s.k_new[0, 0, 0, 5] = float("nan")
    s.v_new[0, 1, 0, 17] = float("inf")
    s.v_new[0, 2, 0, 40] = -float("inf")
    check(s)
    k, v = fd.kv4_read(s.kv, 3, starts=torch.tensor([6], dtype=torch.int32, device="cuda"), dtype=torch.float32)
    assert torch.all(torch.isnan(k[0, 0, 0, :16])) and not torch.any(torch.isnan(k[0, 0, 0, 16:]))
    assert v[0, 0, 1, 17] == 2688.0 and v[0, 0, 2, 40] == -2688.0 and not torch.any(torch.isnan(v))


@pytest.mark.parametrize("cache", CACHES)
def test_bad_page_and_bad_position_are_left_out_and_reported(cache):
    s = Setup(3, 2, 2, 2, 64, cache, page=16, lens=[4, 4, 4], positions=True, seed=8)
    s.positions[1, 0], s.positions[1, 1] = s.cos.shape[0], -1
    s.table[2, 0] = 1 << 20
    before = s.kv.clone() if cache == "4bit" else [x.clone() for x in s.kv]
    q = s.call()
    torch.cuda.synchronize()
    assert fd.workspace_status() == 4
    assert fd.workspace_status() == 0
    s.new_lens = [2, 0, 0]  # what was written: the first sequence's rows
    (check_4bit if cache == "4bit" else check_rows)(s, before, s.kv)
    assert torch.all(q[1] == 0)
    want, err = s.turned(s.q, 2, 1, int(s.positions[2, 1]))
    assert np.all(np.abs(np64(q[2, :, 1]) - want) <= err)


def test_refusals_of_the_binding():
    s = Setup(2, 3, 2, 2, 64, "4bit", seed=1)
    with pytest.raises(ValueError, match="positions"):
        s.call(positions=torch.zeros((2, 2), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="new_lens"):
        s.call(new_lens=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="heads"):
        fd.append_rope_kv4(s.k_new[:, :, :1], s.v_new, s.kv, s.cos, s.sin)
    with pytest.raises(ValueError, match="contiguous"):
        fd.append_rope_kv4(s.k_new.transpose(2, 3).contiguous().transpose(2, 3), s.v_new, s.kv, s.cos, s.sin)
    with pytest.raises(ValueError, match="together"):
        fd.append_rope_kv4(s.k_new, s.v_new, s.kv, s.cos)
    with pytest.raises(ValueError, match="bfloat16"):
        fd.append_rope_kv4(s.k_new, s.v_new.float(), s.kv, s.cos, s.sin)
    with pytest.raises(fd.FdError):
        s.call(max_seq_len=s.cap)
    with pytest.raises(fd.FdError):  # rows that start off a 16-byte boundary
        wide = torch.zeros((2, 3, 2, 72), dtype=torch.bfloat16, device="cuda")
        fd.append_rope_kv4(wide[..., 1:65], s.v_new, s.kv, s.cos, s.sin)
    with pytest.raises(ValueError, match="16"):
        fd.kv4_cache(2, 2, 40, 64)


# ------------------------------------------------------------------ reading back
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_read_is_exact(D, page, dtype):
    s = Setup(4, 1, 0, 3, D, "4bit", page=page, cap=192, seed=D)
    sf = s.kv[..., 16 * D:]
    sf[(sf & 0x7F) == 0x7F] = 0x30  # finite scales
    sf &= 0x7F
    starts, lens, n = [0, 5, 63, 190], [192, 70, 63, 500], 130
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k_out = torch.full((4, 3, n, D), 9.0, dtype=dtype, device="cuda")
    v_out = k_out.clone()
    k, v = fd.kv4_read(s.kv, n, starts=i32(starts), seq_lens=i32(lens), block_table=s.table, k_exp=2, v_exp=-3,
                       k_out=k_out, v_out=v_out)
    assert k is k_out and v is v_out and fd.workspace_status() == 0
    for b in range(4):
        table = None if s.table is None else s.table.cpu().numpy()
        kc, ks, vc, vs = kv4.unpack_blocks(kv4.token_blocks(s.kv.cpu().numpy(), b, table))
        for out, c, f, e in ((k, kc, ks, 2), (v, vc, vs, -3)):
            want = kv4.values(c, f, e).reshape(3, -1, D)[:, starts[b]:min(lens[b], starts[b] + n, 192)]
            m = want.shape[1]
            assert np.array_equal(np64(out[b, :, :m]), want)
            assert torch.all(out[b, :, m:] == 9.0)


def test_read_of_a_bad_page_is_reported():
    s = Setup(1, 1, 0, 1, 64, "4bit", page=16, cap=48, seed=2)
    s.table[0, 1] = -1
    k, _ = fd.kv4_read(s.kv, 48, block_table=s.table)
    assert fd.workspace_status() == 4 and torch.all(k[0, 0, 16:32] == 0)


def test_offsets_past_32_bits():
    """Pages, codes and rows that lie more than 4 GB into their buffers."""
    D, Hkv, pages = 128, 8, 120000  # pages of 32 tokens, 36 KB each
    kv = fd.kv4_cache(pages, Hkv, 32, D)
    assert kv.numel() > 1 << 32
    table = torch.tensor([[pages - 1, 3], [1, pages - 2]], dtype=torch.int32, device="cuda")
    x = torch.randn((2, 33, Hkv, D), device="cuda").bfloat16()
    fd.append_rope_kv4(x, x, kv, seq_lens=torch.zeros(2, dtype=torch.int32, device="cuda"), max_seq_len=0, block_table=table)
    k, v = fd.kv4_read(kv, 33, block_table=table, dtype=torch.float32)
    c, f = kv4.quantise(np64(x))
    want = np.swapaxes(kv4.values(c, f), 1, 2)
    assert np.array_equal(np64(k), want) and np.array_equal(np64(v), want)
    assert int(torch.count_nonzero(kv[4:pages - 2].view(-1)[::4099])) == 0
