"""The float64 oracle of the 4-bit cache: closed forms, and the library's refusals on the host (no GPU is reached)."""

import ctypes
import os

import numpy as np
import pytest

import oracle
import split_kv_decode_fd_gb300 as fd
from split_kv_decode_fd_gb300 import fdecode as fdb

kv4 = oracle.kv4
FAKE = 0x7F0000000000  # a 256-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fd.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return fd.load_library()


# ------------------------------------------------------------------ the oracle
def test_e4m3_values():
    # 0x38 = 1, 0x7e = 448, 0x01 = 2^-9, 0x08 = 2^-6 (the smallest normal), 0x7f NaN
    v = kv4.e4m3_value([0x00, 0x01, 0x08, 0x38, 0x39, 0x7E])
    assert v.tolist() == [0.0, 2.0 ** -9, 2.0 ** -6, 1.0, 1.125, 448.0]
    assert np.isnan(kv4.e4m3_value(0x7F))


def test_rounding_goes_to_the_nearest_and_halfway_to_even():
    halves = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert kv4.e2m1_nearest(halves).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert kv4.e2m1_nearest([-0.3, -100.0, np.inf, -0.0]).tolist() == [9, 15, 7, 8]
    assert kv4.e4m3_nearest([1.0625, 1.1875, 2.0 ** -10, 1e9, np.inf]).tolist() == [0x38, 0x3A, 0, 0x7E, 0x7E]
    x = np.linspace(0, 6.5, 5001)
    assert np.all(np.abs(kv4.E2M1[kv4.e2m1_nearest(x)] - x) <= np.min(np.abs(kv4.E2M1[None] - x[:, None]), 1) + 1e-15)


@pytest.mark.parametrize("D", [64, 128])
def test_blocks_hold_what_was_packed(D):
    r = np.random.default_rng(D)
    kc, vc = (r.integers(0, 16, (3, 2, 16, D)).astype(np.uint8) for _ in range(2))
    ks, vs = (r.integers(0, 0x7F, (3, 2, 16, D // 16)).astype(np.uint8) for _ in range(2))
    blocks = kv4.pack_blocks(kc, ks, vc, vs)
    assert blocks.shape == (3, 2, 18 * D)
    for got, want in zip(kv4.unpack_blocks(blocks), (kc, ks, vc, vs)):
        assert np.array_equal(got, want)
    # a byte by its place: channel 35 of token 5's K, channel 9 of token 11's V, and their scales
    t, d = 5, 35
    sw = (t // 2) % 4 if D == 128 else (t // 4) % 2
    assert blocks[1, 1, t * D // 2 + ((d // 32) ^ sw) * 16 + d % 32 // 2] >> 4 == kc[1, 1, t, d]
    assert blocks[1, 1, 8 * D + 9 * 8 + 11 // 2] >> 4 == vc[1, 1, 11, 9]
    assert blocks[1, 1, 16 * D + t * (D // 16) + 2] == ks[1, 1, t, 2]
    assert blocks[1, 1, 17 * D + 3 * 16 + 11] == vs[1, 1, 11, 3]


def test_quantised_values_are_near_and_exact_values_stay():
    r = np.random.default_rng(0)
    x = r.standard_normal((40, 64))
    c, s = kv4.quantise(x)
    v = kv4.values(c, s)
    # half of the widest gap (2) of the scale, or clipping of what lies past 6 scales (a scale is at most 1/16 too small)
    assert np.all(np.abs(v - x) <= np.repeat(kv4.e4m3_value(s), 16, -1) * 1.0 + 1e-12)
    c2, s2 = kv4.quantise(v * 2.0 ** 5, exp=5)
    # a block whose largest code is 6 keeps its scale, and with it every code
    full = np.max(np.abs(c & 7).reshape(40, 4, 16), -1) == 7
    assert full.any() and np.array_equal(s2[full], s[full])
    assert np.array_equal((c2.reshape(40, 4, 16))[full], c.reshape(40, 4, 16)[full])


def test_nan_and_infinity():
    x = np.zeros((1, 64))
    x[0, 3], x[0, 20], x[0, 21] = np.nan, np.inf, 1.0
    v = kv4.values(*kv4.quantise(x))
    assert np.all(np.isnan(v[0, :16])) and v[0, 20] == 2688.0 and v[0, 21] == 0.0 and np.all(v[0, 32:] == 0)


def test_rotation_by_a_right_angle():
    x = np.arange(8.0)[None]
    assert kv4.rotate(x, np.zeros((1, 2)), np.ones((1, 2))).tolist() == [[-2, -3, 0, 1, 4, 5, 6, 7]]
    assert kv4.rotate(x, np.zeros((1, 2)), np.ones((1, 2)), True).tolist() == [[-1, 0, -3, 2, 4, 5, 6, 7]]


# ------------------------------------------------------------------ refusals
def rows(**kw):
    r = fdb.NewRows()
    r.dtype, r.q, r.k, r.v = fdb.FD_BF16, FAKE, FAKE, FAKE
    r.q_stride[:] = r.k_stride[:] = r.v_stride[:] = (6144, 6144, 128)
    r.cos = r.sin = FAKE
    r.max_pos, r.rot_dim, r.interleaved = 2048, 128, 0
    for k, v in kw.items():
        if k.endswith("_stride"):
            getattr(r, k)[:] = v
        else:
            setattr(r, k, v)
    return r


def cache4(**kw):
    d = fdb.Kv4Desc()
    d.layout, d.kv, d.capacity = 0, FAKE, 1024
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def cache16(**kw):
    d = fdb.KvDesc()
    d.layout, d.dtype, d.k, d.v, d.capacity = 0, fdb.FD_BF16, FAKE, FAKE, 1024
    for k, v in kw.items():
        setattr(d, k, v)
    return d


INVALID, UNSUPPORTED, SMALL = fdb.FD_ERR_INVALID_ARG, fdb.FD_ERR_UNSUPPORTED, fdb.FD_ERR_WORKSPACE_TOO_SMALL

ROWS_CASES = [
    (dict(k=0), {}, INVALID), (dict(v=0), {}, INVALID), (dict(q=0), {}, INVALID), (dict(k=FAKE + 8), {}, INVALID),
    (dict(k_stride=(6144, 6140, 128)), {}, INVALID), (dict(v_stride=(-128, 128, 128)), {}, INVALID),
    (dict(q_stride=(1, 128, 128)), {}, INVALID), (dict(dtype=5), {}, UNSUPPORTED),
    (dict(cos=0), {}, INVALID), (dict(sin=FAKE + 4), {}, INVALID), (dict(rot_dim=160), {}, INVALID),
    (dict(rot_dim=48), {}, UNSUPPORTED), (dict(rot_dim=-32), {}, INVALID), (dict(interleaved=2), {}, INVALID),
    (dict(max_pos=1023), {}, INVALID),  # places up to 1023 need 1024 rows
    ({}, dict(q_out=0), INVALID), ({}, dict(q_out=FAKE + 4), INVALID), ({}, dict(B=0), INVALID), ({}, dict(n=0), INVALID),
    ({}, dict(Hkv=0), INVALID), ({}, dict(Hq=-1), INVALID), ({}, dict(D=96), UNSUPPORTED), ({}, dict(max_len=-1), INVALID),
    ({}, dict(max_len=1024), INVALID),  # 1024 + 1 tokens in a cache of 1024
    ({}, dict(ws=0), INVALID), ({}, dict(ws_bytes=128), SMALL), ({}, dict(max_len=2 ** 31 - 1), UNSUPPORTED),
]


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("row,call,expected", ROWS_CASES)
def test_append_refuses(lib, four, row, call, expected):
    a = dict(q_out=FAKE, B=2, n=1, Hq=4, Hkv=2, max_len=1023, D=128, ws=FAKE, ws_bytes=256)
    a.update(call)
    fn, kv = (lib.fd_append_rope_kv4, cache4()) if four else (lib.fd_append_rope, cache16())
    r = rows(**row)
    assert fn(ctypes.byref(r), ctypes.byref(kv), a["q_out"], a["B"], a["n"], a["Hq"], a["Hkv"], None, a["max_len"],
              a["D"], a["ws"], a["ws_bytes"], None) == expected


KV4_CASES = [
    (dict(kv=0), INVALID), (dict(kv=FAKE + 8), INVALID), (dict(capacity=0), INVALID), (dict(capacity=1000), INVALID),
    (dict(k_exp=65), INVALID), (dict(v_exp=-65), INVALID), (dict(layout=2), INVALID),
    (dict(layout=1, block_table=0, page_size=16, max_pages_per_seq=64, num_pages=9), INVALID),
    (dict(layout=1, block_table=FAKE, page_size=24, max_pages_per_seq=64, num_pages=9), INVALID),
    (dict(layout=1, block_table=FAKE, page_size=16, max_pages_per_seq=63, num_pages=9), INVALID),
    (dict(layout=1, block_table=FAKE, page_size=16, max_pages_per_seq=64, num_pages=0), INVALID),
]


@pytest.mark.parametrize("kv,expected", KV4_CASES)
def test_bad_caches_are_refused_by_every_call(lib, kv, expected):
    d = cache4(**kv)
    r = rows()
    assert lib.fd_append_rope_kv4(ctypes.byref(r), ctypes.byref(d), FAKE, 2, 1, 4, 2, None, 1023, 128, FAKE, 256,
                                  None) == expected
    assert lib.fd_kv4_read(ctypes.byref(d), FAKE, FAKE, fdb.FD_BF16, 2, 8, 2, None, None, 1024, 128, FAKE, 256,
                           None) == expected
    assert lib.fd_decode_kv4(FAKE, 1, 1, ctypes.byref(d), FAKE, None, 2, 4, 2, None, 1024, 128, 0.1, 4, FAKE, 1 << 30,
                             None) == expected


@pytest.mark.parametrize("call,expected", [
    (dict(k=0), INVALID), (dict(v=FAKE + 4), INVALID), (dict(dtype=3), UNSUPPORTED), (dict(B=0), INVALID),
    (dict(n=0), INVALID), (dict(D=80), UNSUPPORTED), (dict(ws=0), INVALID), (dict(ws_bytes=64), SMALL),
    (dict(max_len=1040), INVALID),
])
def test_read_refuses(lib, call, expected):
    a = dict(k=FAKE, v=FAKE, dtype=fdb.FD_F32, B=2, n=8, D=128, ws=FAKE, ws_bytes=256, max_len=1024)
    a.update(call)
    assert lib.fd_kv4_read(ctypes.byref(cache4()), a["k"], a["v"], a["dtype"], a["B"], a["n"], 2, None, None,
                           a["max_len"], a["D"], a["ws"], a["ws_bytes"], None) == expected


@pytest.mark.parametrize("call,expected", [
    (dict(q=0), INVALID), (dict(q=FAKE + 4), INVALID), (dict(out=0), INVALID), (dict(n_q=0), INVALID),
    (dict(n_q=65), INVALID), (dict(causal=2), INVALID), (dict(Hq=3), INVALID), (dict(Hq=3, n_q=2), INVALID),
    (dict(D=32), UNSUPPORTED), (dict(n_splits=-1), INVALID), (dict(n_splits=70000), INVALID), (dict(max_len=1040), INVALID),
    (dict(ws=0), INVALID), (dict(ws_bytes=256), SMALL),
])
def test_decode_refuses(lib, call, expected):
    a = dict(q=FAKE, out=FAKE, n_q=1, causal=1, Hq=4, D=128, n_splits=3, max_len=1024, ws=FAKE, ws_bytes=1 << 30)
    a.update(call)
    assert lib.fd_decode_kv4(a["q"], a["n_q"], a["causal"], ctypes.byref(cache4()), a["out"], None, 2, a["Hq"], 2, None,
                             a["max_len"], a["D"], 0.1, a["n_splits"], a["ws"], a["ws_bytes"], None) == expected


def test_block_bytes(lib):
    assert fd.kv4_block_bytes(64) == 1152 and fd.kv4_block_bytes(128) == 2304
    with pytest.raises(fd.FdError):
        fd.kv4_block_bytes(96)


def test_binding_refuses_cpu_tensors(lib):
    import torch
    x = torch.zeros(1, 1, 4, 64)
    c = torch.zeros(1, 4, 2, 18 * 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        fd.decode_kv4(x[0, 0][None], c)
    with pytest.raises(ValueError, match="CUDA"):
        fd.append_rope_kv4(x, x, c)
    with pytest.raises(ValueError, match="CUDA"):
        fd.append_rope(x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        fd.kv4_read(c, 4)
