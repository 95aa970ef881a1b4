"""Refusals of the calls for trees of drafted tokens, through the C ABI: none of these reaches a GPU."""

import ctypes
import os

import pytest
import torch

import split_kv_decode_fd_gb300 as fd
from split_kv_decode_fd_gb300 import fdecode as fdb

FAKE = 0x7F0000000000  # a 256-byte aligned address that is never read
BAD, NO = fdb.FD_ERR_INVALID_ARG, fdb.FD_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fd.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return fd.load_library()


def kv(layout=0, dtype=1, k=FAKE, v=FAKE + 4096, capacity=1024, table=None, max_pages=0, page=0, pages=0):
    d = fdb.KvDesc()
    d.layout, d.dtype, d.k, d.v, d.capacity = layout, dtype, k, v, capacity
    d.block_table, d.max_pages_per_seq, d.page_size, d.num_pages = table, max_pages, page, pages
    return d


def tree(parents=FAKE, stride=8, new_lens=None, n=8):
    d = fdb.TreeDesc()
    d.parents, d.parents_stride, d.new_lens, d.n = parents, stride, new_lens, n
    return d


BAD_TREES = [
    (dict(parents=None), BAD),
    (dict(n=0), BAD),
    (dict(n=-1), BAD),
    (dict(n=64 + 1, stride=0), NO),
    (dict(n=1 << 30, stride=0), NO),
    (dict(stride=7), BAD),
    (dict(stride=-8), BAD),
]


def decode(lib, t=None, c=None, q=FAKE, out=FAKE, B=1, Hq=4, Hkv=4, max_len=1024, D=128, ws=FAKE, size=1 << 40):
    return lib.fd_decode_tree(q, t if t is not None else tree(), c if c is not None else kv(), out, None, B, Hq, Hkv, None,
                              max_len, D, 0.1, ws, size, None)


@pytest.mark.parametrize("t,expected", BAD_TREES)
def test_decode_tree_refuses_trees(lib, t, expected):
    assert decode(lib, tree(**t)) == expected


@pytest.mark.parametrize("case,expected", [
    (dict(q=None), BAD), (dict(out=None), BAD), (dict(ws=None), BAD),
    (dict(q=FAKE + 4), BAD), (dict(out=FAKE + 8), BAD), (dict(ws=FAKE + 4), BAD),
    (dict(B=0), BAD), (dict(B=-1), BAD), (dict(Hq=6), BAD), (dict(Hkv=0), BAD),
    (dict(D=96), NO), (dict(D=256), NO), (dict(D=0), NO),
    (dict(max_len=1025), BAD), (dict(max_len=-1), BAD),
    (dict(c=kv(k=None)), BAD), (dict(c=kv(v=FAKE + 8)), BAD), (dict(c=kv(dtype=7)), NO), (dict(c=kv(layout=3)), BAD),
    (dict(c=kv(layout=1, table=FAKE, max_pages=64, page=24, pages=100)), BAD),
    (dict(c=kv(layout=1, table=FAKE, max_pages=32, page=16, pages=100)), BAD),
    (dict(c=kv(layout=1, table=None, max_pages=64, page=16, pages=100)), BAD),
    (dict(c=kv(capacity=2 ** 31 - 1), max_len=2 ** 31 - 1), NO),  # a tile's end would pass 32 bits
    (dict(Hq=1 << 22, Hkv=1 << 22), NO),                          # rows of a KV head's group are counted in 32 bits
])
def test_decode_tree_refuses_arguments(lib, case, expected):
    assert decode(lib, **case) == expected


def test_no_workspace_for_shapes_that_are_refused(lib):
    for B, Hq, Hkv, D, n in ((1, 4, 4, 128, 0), (1, 4, 4, 128, 64 + 1), (1, 6, 4, 128, 8), (1, 4, 4, 80, 8),
                             (0, 4, 4, 128, 8), (1, 1 << 22, 1 << 22, 128, 8)):
        assert lib.fd_tree_workspace_bytes(B, Hq, Hkv, D, n, 152) == 0
    assert lib.fd_tree_workspace_bytes(1, 32, 8, 128, 64, 152) > 0


def strides(*x):
    return (ctypes.c_int64 * 2)(*x)


def verify(lib, t=None, tokens=FAKE, uniforms=FAKE, target=FAKE, ts=(800, 100), draft=FAKE, ds=(800, 100), dtype=1, path=FAKE,
           count=FAKE, word=FAKE, B=1, V=100, ws=FAKE, size=256):
    return lib.fd_verify_tree(t if t is not None else tree(), tokens, uniforms, target, strides(*ts) if ts else None, draft,
                              strides(*ds) if ds else None, dtype, path, count, word, B, V, ws, size, None)


@pytest.mark.parametrize("t,expected", BAD_TREES)
def test_verify_tree_refuses_trees(lib, t, expected):
    assert verify(lib, tree(**t)) == expected


@pytest.mark.parametrize("case,expected", [
    (dict(tokens=None), BAD), (dict(uniforms=None), BAD), (dict(target=None), BAD), (dict(ts=None), BAD), (dict(ds=None), BAD),
    (dict(path=None), BAD), (dict(count=None), BAD), (dict(word=None), BAD), (dict(ws=None), BAD), (dict(ws=FAKE + 8), BAD),
    (dict(V=0), BAD), (dict(V=-4), BAD), (dict(V=2 ** 31 - 1), NO), (dict(B=0), BAD), (dict(B=2 ** 31 - 1), NO),
    (dict(dtype=3), NO), (dict(dtype=0, target=FAKE + 2), BAD), (dict(target=FAKE + 1), BAD), (dict(draft=FAKE + 1), BAD),
    (dict(ts=(-1, 100)), BAD), (dict(ds=(800, -100)), BAD),
    (dict(size=255), fdb.FD_ERR_WORKSPACE_TOO_SMALL),
])
def test_verify_tree_refuses_arguments(lib, case, expected):
    assert verify(lib, **case) == expected


def keep(lib, c=None, index=FAKE, n=8, B=1, Hkv=4, max_len=1024, D=128, ws=FAKE, size=256):
    return lib.fd_keep_rows(c if c is not None else kv(), index, n, None, None, B, Hkv, max_len, D, ws, size, None)


@pytest.mark.parametrize("case,expected", [
    (dict(index=None), BAD), (dict(n=0), BAD), (dict(n=-3), BAD), (dict(n=2 ** 31 - 1), NO),
    (dict(B=0), BAD), (dict(Hkv=0), BAD), (dict(D=96), NO), (dict(max_len=1025), BAD), (dict(max_len=-1), BAD),
    (dict(ws=None), BAD), (dict(ws=FAKE + 4), BAD), (dict(size=128), fdb.FD_ERR_WORKSPACE_TOO_SMALL),
    (dict(c=kv(v=None)), BAD), (dict(c=kv(dtype=5)), NO), (dict(B=1 << 20, Hkv=1 << 10), NO),
    (dict(c=kv(layout=1, table=FAKE, max_pages=64, page=8, pages=100)), BAD),
])
def test_keep_rows_refuses_arguments(lib, case, expected):
    assert keep(lib, **case) == expected


def test_the_binding_refuses_cpu_tensors(lib):
    q, cache = torch.zeros(1, 4, 3, 64), torch.zeros(1, 4, 16, 64)
    ints = torch.zeros(1, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        fd.decode_tree(q, cache, cache, ints)
    with pytest.raises(ValueError):
        fd.verify_tree(ints, ints, torch.zeros(1, 3, 10), torch.zeros(1, 3))
    with pytest.raises(ValueError):
        fd.keep_rows(cache, cache, ints)
