"""GPU tests of the 4-bit decode's softmax weights far below the largest one.

One key of score s among N - 1 of score 0, whose weights lie between 2^-33 and 2^-36 of its own: each alone is far below
an fp32 result's last bit, and all of them together are not.  With one split a CTA holds the whole sequence.

Bound.  A score is off by 2^-24 of itself for each of scale * log2(e) and its product with q, by 2^-22 for q's split and
2^-24 for the reference: at most 36 * 2^-21.4 in log2, which moves a weight by less than 2^-16.5 of itself.  A weight's
two fp16 numbers, the lower one held 2^11 times up, leave 2^-36 of 2^9 (the largest weight): 2^-45.  With T the sum of
the small weights over that of all, |v| <= 1, and F sums of O over the tiles, each rounded by 2^-25 of the sum,
out is off by T 2^-16 + N 2^-45 + (F + 8) 2^-24 |out's largest part|; that part is the large key's value, or T where it is 0.
"""

import math

import numpy as np
import pytest
import torch

import oracle
import split_kv_decode_fd_gb300 as fd

pytestmark = pytest.mark.gpu
kv4 = oracle.kv4


def block(k0, v, D):
    """A block of sixteen equal tokens: key (k0, 0, 0, ...), value v, as codes with scales of one."""
    one = np.full((16, D // 16), 0x38, dtype=np.uint8)
    k = np.zeros(D)
    k[0] = k0
    rows = [np.tile(kv4.e2m1_nearest(x), (16, 1)) for x in (k, v)]
    return kv4.pack_blocks(rows[0], one, rows[1], one)


@pytest.mark.parametrize("N", [1 << 17, (1 << 18) + 5])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq", [1, 4, 8, 16])
@pytest.mark.parametrize("n_splits", [1, 0])
def test_many_small_weights_count(N, D, Hq, n_splits):
    even = np.arange(D) % 2 == 0
    small = np.where(even, 1.0, -0.5)
    large = np.where(even, 0.0, 1.0)
    at = N // 3 // 16 * 16
    cap = -(-N // 16) * 16
    cache = torch.from_numpy(block(0.0, small, D)).cuda().expand(1, 1, cap // 16, 18 * D).contiguous()
    parts = [x.copy() for x in kv4.unpack_blocks(block(0.0, small, D))]
    key, _, value, _ = kv4.unpack_blocks(block(6.0, large, D))
    parts[0][3], parts[2][3] = key[3], value[3]
    cache[0, 0, at // 16] = torch.from_numpy(kv4.pack_blocks(*parts)).cuda()

    scale = 0.125
    gaps = np.linspace(33.1, 35.9, Hq)  # log2 of the largest weight over a small one
    q = torch.zeros((1, Hq, D), device="cuda")
    q[0, :, 0] = torch.from_numpy(gaps * math.log(2.0) / (6.0 * scale)).cuda()
    out, lse = fd.decode_kv4(q, cache, scale=scale, n_splits=n_splits, max_seq_len=N)
    assert fd.workspace_status() == 0

    s = q[0, :, 0].double().cpu().numpy() * 6.0 * scale
    w = (N - 1) * np.exp(-s)
    T = (w / (1.0 + w))[:, None]
    want = (1.0 - T) * large + T * small
    F = N / 512
    bound = T * 2.0 ** -16 + N * 2.0 ** -45 + (F + 8) * 2.0 ** -24 * np.where(even, T, 1.0)
    err = np.abs(out[0].double().cpu().numpy() - want)
    assert np.all(err <= bound), (err / bound).max()
    assert np.all(np.abs(lse[0].double().cpu().numpy() - (s + np.log1p(w))) <= s * 2.0 ** -21 + 2.0 ** -20)
