"""Plain float64 oracle of the 4-bit KV cache and of the rotating append.

TEST INFRASTRUCTURE ONLY, as ``fd_oracle``: NumPy alone, no code shared with the CUDA library.

A cache value is ``code * scale * 2**exp``: an e2m1 code and one e4m3 scale for sixteen consecutive channels of a
token.  The sources name appending to paged caches and low-precision caches without a format; the format is the
library's, restated here from its description: blocks of sixteen tokens of one KV head, ``18 * D`` bytes,
K codes ``[16][D/2]`` with swizzled 16-byte chunks, V codes ``[D][8]``, K scales ``[16][D/16]``, V scales ``[D/16][16]``.
"""

from __future__ import annotations

import numpy as np

__all__ = ["E2M1", "e4m3_value", "e4m3_nearest", "e2m1_nearest", "quantise", "values", "pack_blocks", "unpack_blocks",
           "rotate", "token_blocks"]

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_value(byte) -> np.ndarray:
    """Value of non-negative e4m3 bytes; 0x7f is NaN."""
    b = np.asarray(byte).astype(np.int64)
    e, m = b >> 3 & 15, b & 7
    v = np.where(e > 0, (1.0 + m / 8.0) * 2.0 ** (e - 7.0), m / 8.0 * 2.0 ** -6)
    v = np.where((b & 0x7F) == 0x7F, np.nan, v)
    return np.where(b & 0x80, -v, v)


_SCALES = e4m3_value(np.arange(0x7F))


def _nearest(x, grid) -> np.ndarray:
    """Index of the nearest grid value, halfway cases to the even index, past the end to the last."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dlo, dhi = x - grid[lo], grid[hi] - x
    return np.where(dlo < dhi, lo, np.where(dhi < dlo, hi, np.where(lo % 2 == 0, lo, hi)))


def e4m3_nearest(x) -> np.ndarray:
    """Byte of the e4m3 value nearest to x >= 0, at most 448; NaN gives 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    return np.where(np.isnan(x), 0x7F, _nearest(np.nan_to_num(x, nan=0.0, posinf=448.0), _SCALES)).astype(np.uint8)


def e2m1_nearest(r) -> np.ndarray:
    """Code of the e2m1 value nearest to r, at most 6 in size; bit 3 is the sign."""
    r = np.asarray(r, dtype=np.float64)
    return (_nearest(np.nan_to_num(np.abs(r), nan=0.0, posinf=6.0), E2M1) + 8 * np.signbit(r)).astype(np.uint8)


def quantise(x, exp=0):
    """Codes ``[..., D]`` and scale bytes ``[..., D/16]`` of x."""
    y = np.asarray(x, dtype=np.float64) * 2.0 ** -exp
    blocks = y.reshape(y.shape[:-1] + (-1, 16))
    with np.errstate(invalid="ignore", divide="ignore"):
        sf = e4m3_nearest(np.max(np.abs(blocks), -1) / 6.0)
        s = e4m3_value(sf)[..., None]
        r = np.where(s > 0, blocks / np.where(s > 0, s, 1.0), np.copysign(0.0, blocks))
    return e2m1_nearest(r).reshape(y.shape), sf


def values(codes, sf, exp=0) -> np.ndarray:
    """float64 values of codes ``[..., D]`` with scale bytes ``[..., D/16]``."""
    c = np.asarray(codes)
    v = np.where(c & 8, -E2M1[c & 7], E2M1[c & 7])
    return v * np.repeat(e4m3_value(sf), 16, axis=-1) * 2.0 ** exp


def _chunk_of(D) -> np.ndarray:
    t, c = np.arange(16)[:, None], np.arange(D // 32)[None, :]
    return c ^ ((t // 2) % 4 if D == 128 else (t // 4) % 2)


def pack_blocks(kc, ks, vc, vs) -> np.ndarray:
    """Blocks ``[..., 18 * D]`` of codes ``[..., 16, D]`` and scale bytes ``[..., 16, D/16]``."""
    lead, D = kc.shape[:-2], kc.shape[-1]
    rows = (kc[..., 0::2] | kc[..., 1::2] << 4).reshape(lead + (16, D // 32, 16))
    kb = np.empty_like(rows)
    at = _chunk_of(D)
    for t in range(16):
        kb[..., t, at[t], :] = rows[..., t, :, :]
    vt = np.swapaxes(vc, -1, -2)
    vb = vt[..., 0::2] | vt[..., 1::2] << 4
    flat = lambda a: np.ascontiguousarray(a).reshape(lead + (-1,)).astype(np.uint8)  # noqa: E731
    return np.concatenate([flat(kb), flat(vb), flat(ks), flat(np.swapaxes(vs, -1, -2))], -1)


def unpack_blocks(blocks):
    """(kc, ks, vc, vs) of ``pack_blocks``."""
    b = np.asarray(blocks)
    lead, D = b.shape[:-1], b.shape[-1] // 18
    kb = b[..., :8 * D].reshape(lead + (16, D // 32, 16))
    at = _chunk_of(D)
    rows = np.stack([kb[..., t, at[t], :] for t in range(16)], -3).reshape(lead + (16, D // 2))
    kc = np.stack([rows & 15, rows >> 4], -1).reshape(lead + (16, D))
    vb = b[..., 8 * D:16 * D].reshape(lead + (D, 8))
    vc = np.swapaxes(np.stack([vb & 15, vb >> 4], -1).reshape(lead + (D, 16)), -1, -2)
    ks = b[..., 16 * D:17 * D].reshape(lead + (16, D // 16))
    vs = np.swapaxes(b[..., 17 * D:].reshape(lead + (D // 16, 16)), -1, -2)
    return kc, ks, vc, vs


def token_blocks(kv4, b, block_table=None) -> np.ndarray:
    """Blocks ``[Hkv, blocks, 18 * D]`` of sequence b, every place its table names."""
    kv4 = np.asarray(kv4)
    if block_table is None:
        return kv4[b]
    pages = kv4[np.asarray(block_table)[b]]  # [pages, Hkv, blocks of a page, bytes]
    return np.swapaxes(pages, 0, 1).reshape(kv4.shape[1], -1, kv4.shape[-1])


def rotate(x, cos, sin, interleaved=False) -> np.ndarray:
    """Rows ``[..., D]`` with cos, sin ``[..., rot/2]`` (the rows of their positions): pairs of the first rot channels turned."""
    x = np.asarray(x, dtype=np.float64).copy()
    c, s = np.asarray(cos, dtype=np.float64), np.asarray(sin, dtype=np.float64)
    half = c.shape[-1]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    u, w = x[..., a].copy(), x[..., b].copy()
    x[..., a] = u * c - w * s
    x[..., b] = w * c + u * s
    return x
