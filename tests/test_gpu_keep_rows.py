"""GPU tests of rows that move together in a cache: every byte equal to the oracle's."""

import numpy as np
import pytest
import torch

import oracle
import split_kv_decode_fd_gb300 as fd

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


class Case:
    def __init__(self, B, Hkv, D, cap, *, cache="bf16", page=0, seed=0):
        r = np.random.default_rng(seed)
        unit = page or 1
        self.cap = cap = -(-cap // unit) * unit
        self.page = page
        self.views = []  # K and V as [B, Hkv, T, D] and as given
        self.table = None
        if page:
            per = cap // page
            self.table_np = r.permutation(B * per + 1)[:B * per].reshape(B, per).astype(np.int32)
            self.table = torch.from_numpy(self.table_np).cuda()
            shape = (B * per + 1, Hkv, page, D)
        else:
            shape = (B, Hkv, cap, D)
        self.k, self.v = (torch.from_numpy(r.standard_normal(shape).astype(np.float32)).to(TYPES[cache]).cuda() for _ in range(2))

    def flat(self, x):
        x = x.float().cpu().numpy()
        if not self.page:
            return x
        x = x[self.table_np]  # [B, per, Hkv, page, D]
        return np.swapaxes(x, 1, 2).reshape(x.shape[0], x.shape[2], -1, x.shape[4])

    def check(self, index, counts=None, starts=None, want_counts=None, status=0, **kw):
        index = np.asarray(index, dtype=np.int32)
        B = len(index)
        as_t = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        c = want_counts if want_counts is not None else [index.shape[1]] * B if counts is None else counts
        s = [0] * B if starts is None else starts
        want = [oracle.tree.keep(self.flat(x), index, s, c) for x in (self.k, self.v)]
        spare = None if not self.page else [x[[i for i in range(len(x)) if i not in self.table_np]].clone() for x in (self.k, self.v)]
        fd.keep_rows(self.k, self.v, torch.from_numpy(index).cuda(), counts=as_t(counts), starts=as_t(starts), block_table=self.table, **kw)
        assert fd.workspace_status(kw.get("workspace")) == status
        for x, w in zip((self.k, self.v), want):
            assert np.array_equal(self.flat(x), w)
        if spare:
            for x, w in zip((self.k, self.v), spare):
                assert torch.equal(x[[i for i in range(len(x)) if i not in self.table_np]], w)


def rising(r, n, reach):
    return np.sort(r.permutation(reach)[:n])


@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [0, 16, 48])
@pytest.mark.parametrize("n,reach", [(1, 1), (1, 9), (5, 16), (16, 17), (64, 64), (64, 200), (65, 65), (65, 150), (300, 301), (1000, 2500), (3000, 3001)])
def test_against_the_oracle(cache, D, page, n, reach):
    r = np.random.default_rng(n + reach + D)
    B = 3
    c = Case(B, 2, D, reach + 40, cache=cache, page=page, seed=n)
    index = np.stack([rising(r, n, reach) for _ in range(B)])
    starts = r.integers(0, 40, B).tolist()
    c.check(index, [n, n // 2, 0], starts)
    c.check(index)


def test_lists_that_move_by_one_and_lists_that_stay():
    for n in (5, 64, 2000):
        c = Case(2, 3, 128, n + 8, seed=n)
        c.check([np.arange(1, n + 1), np.arange(n)])
        c.check([np.r_[np.arange(n - 1), n + 3], np.r_[0, np.arange(2, n + 1)]], starts=[2, 4])


def test_counts_are_clamped():
    c = Case(3, 2, 64, 40, seed=1)
    c.check([[0, 2, 5]] * 3, counts=[-4, 99, 1 << 30], want_counts=[0, 3, 3])


@pytest.mark.parametrize("n", [6, 80, 2100])
def test_a_list_that_does_not_rise_ends_there(n):
    for at, bad in ((0, -1), (0, -(1 << 31)), (3, 3), (3, 0), (n - 1, n - 2), (n // 2, 1 << 30), (n // 2, (1 << 31) - 1), (1, -7)):
        c = Case(2, 2, 64, 2 * n + 4, seed=n)
        index = np.stack([2 * np.arange(n) + 1] * 2).astype(np.int32)
        index[0, at] = bad
        if at == 3 and bad == 3:
            index[0, 2] = 5  # 5, then 3: the entry itself is in range
        stop = at
        c.check(index, want_counts=[stop, n], status=fd.fdecode.FD_ERR_BAD_INDEX)


@pytest.mark.parametrize("cache,D", [("bf16", 128), ("bf16", 64), ("f32", 128)])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("n", [65, 700, 5000])
def test_rows_from_behind_all_that_is_written(cache, D, page, n):
    """The first rows stay where they are, the others come from behind: the list is shared."""
    r = np.random.default_rng(n)
    c = Case(3, 2, D, 3 * n + 90, cache=cache, page=page, seed=n)
    index = np.stack([np.r_[np.arange(s), n + np.sort(r.permutation(2 * n)[:n - s])] for s in (0, 4, n)]).astype(np.int32)
    c.check(index, starts=[5, 0, 80])
    c.check(index, counts=[n, n - 1, n // 2], starts=[5, 0, 80])
    index[0, n // 3] = 0  # the list ends there
    index[1, n - 1] = 1 << 30
    c.check(index, want_counts=[n // 3, n - 1, n], status=fd.fdecode.FD_ERR_BAD_INDEX)


def test_places_past_the_end_and_before_the_start():
    bad = fd.fdecode.FD_ERR_BAD_INDEX
    c = Case(3, 2, 128, 64, seed=2)
    c.check([[1, 3, 40]] * 3, starts=[24, 23, -1], want_counts=[2, 3, 0], status=bad)
    c.check([[1, 3, 40]] * 3, starts=[0, 9, 10], max_seq_len=50, want_counts=[3, 3, 2], status=bad)
    c.check([[1, 3, 40]] * 3, starts=[(1 << 31) - 1, -(1 << 31), 0], want_counts=[0, 0, 3], status=bad)


@pytest.mark.parametrize("n", [8, 100])
def test_pages_outside_the_pool(n):
    c = Case(2, 2, 64, 4 * n, page=16, seed=3)
    index = np.stack([3 * np.arange(n)] * 2).astype(np.int32)
    table = c.table.clone()
    good = [c.flat(x) for x in (c.k, c.v)]
    page = 16 * int(n // 16 + 1)  # of which rows come
    table[0, page // 16] = 1 << 30
    fd.keep_rows(c.k, c.v, torch.from_numpy(index).cuda(), block_table=table)
    assert fd.workspace_status() == fd.fdecode.FD_ERR_BAD_INDEX
    for x, w in zip((c.k, c.v), good):
        got = c.flat(x)
        assert np.array_equal(got[1], oracle.tree.keep(w, index, [0, 0], [n, n])[1])
        for j in range(n):  # rows from the missing page are left as they were
            src = 3 * j
            lost = src // 16 == page // 16 or j // 16 == page // 16
            assert np.array_equal(got[0, :, j], w[0, :, j if lost else src]), j


@pytest.mark.parametrize("n", [9, 500])
def test_on_another_stream_and_captured(n):
    r = np.random.default_rng(n)
    c = Case(2, 2, 128, 3 * n, seed=n)
    index = torch.from_numpy(np.stack([n + rising(r, n, 2 * n) for _ in range(2)]).astype(np.int32)).cuda()  # a second pass changes nothing
    k0, v0 = c.k.clone(), c.v.clone()
    fd.keep_rows(c.k, c.v, index)
    k1, v1 = c.k.clone(), c.v.clone()
    s = torch.cuda.Stream()
    c.k.copy_(k0), c.v.copy_(v0)
    torch.cuda.synchronize()
    fd.keep_rows(c.k, c.v, index, stream=s)
    s.synchronize()
    assert torch.equal(c.k, k1) and torch.equal(c.v, v1)
    ws = fd.Workspace()
    fd.keep_rows(c.k, c.v, index, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fd.keep_rows(c.k, c.v, index, workspace=ws)
    c.k.copy_(k0), c.v.copy_(v0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.k, k1) and torch.equal(c.v, v1)


def test_offsets_past_32_bits():
    D = 128
    T = (1 << 31) // D + 4096
    k, v = (torch.empty((1, 1, T, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for n in (40, 1500):
        rows = torch.randn((2, 2 * n, D), device="cuda").bfloat16()
        start = T - 2 * n - 5
        k[0, 0, start:start + 2 * n], v[0, 0, start:start + 2 * n] = rows[0], rows[1]
        index = torch.arange(1, 2 * n, 2, dtype=torch.int32, device="cuda")[None, :n].contiguous()
        fd.keep_rows(k, v, index, starts=torch.tensor([start], dtype=torch.int32, device="cuda"))
        for x, w in zip((k, v), rows):
            assert torch.equal(x[0, 0, start:start + n], w[1::2]) and torch.equal(x[0, 0, start + n:start + 2 * n], w[n:])


def test_refusals():
    c = Case(2, 2, 64, 32, seed=4)
    index = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    fd.keep_rows(c.k, c.v, index)
    for a in ((c.k, c.v, index.long()), (c.k, c.v, index[0]), (c.k, c.v, index[:1]), (c.k.cpu(), c.v, index), (c.k, c.v.float(), index),
              (c.k, c.v[:, :1], index), (c.k.half(), c.v.half(), index), (c.k, c.v, index.cpu()), (c.k[0], c.v[0], index), (c.k, c.v, None)):
        with pytest.raises(ValueError):
            fd.keep_rows(*a)
    for kw in (dict(counts=lens.long()), dict(starts=lens[:1]), dict(block_table=lens)):
        with pytest.raises(ValueError):
            fd.keep_rows(c.k, c.v, index, **kw)
    for kw in (dict(max_seq_len=33), dict(max_seq_len=-1)):
        with pytest.raises(fd.FdError):
            fd.keep_rows(c.k, c.v, index, **kw)
    with pytest.raises(fd.FdError):
        fd.keep_rows(c.k, c.v, torch.empty((2, 0), dtype=torch.int32, device="cuda"))
