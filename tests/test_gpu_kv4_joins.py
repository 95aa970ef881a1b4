"""GPU tests of the joins of the 4-bit decode's partial states: more states than a warp takes at once, and more (sequence,
virtual KV head) pairs than there are counters, where a second kernel joins them.  Bounds as in test_gpu_decode_kv4."""

import math

import numpy as np
import pytest
import torch

import split_kv_decode_fd_gb300 as fd

from test_gpu_decode_kv4 import Case, kv4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,n_q", [(4, 1), (16, 1), (3, 2)])
@pytest.mark.parametrize("n_splits", [0, 33, 40, 70])
def test_more_than_32_states_of_a_sequence(D, Hq, n_q, n_splits):
    c = Case(2, Hq, 1, D, [60000, 700], n_q=n_q, page=16, seed=D + Hq)
    out, lse = c.run(n_splits)
    assert fd.workspace_status() == 0
    c.check(out, lse)


def formula(c, lens):
    """Attention of a Case with one KV head in 64 bits, all rows at once, and the bounds of out and lse."""
    k, v = (torch.from_numpy(x[:, 0]).cuda() for x in (c.k, c.v))  # [B, T, D]
    B, Hq, n_q, D = c.q.shape
    T = k.shape[1]
    q = c.q.double().view(B, Hq * n_q, D)
    s = q @ k.transpose(1, 2) * c.scale
    row = torch.arange(Hq * n_q, device="cuda") % n_q
    limit = torch.tensor(lens, device="cuda").view(B, 1, 1) - (n_q - 1 - row).view(1, -1, 1)
    s = s.masked_fill(torch.arange(T, device="cuda") >= limit, -math.inf)
    lse = torch.logsumexp(s, -1)
    out = torch.exp(s - torch.where(lse > -math.inf, lse, 0.0).unsqueeze(-1)) @ v
    A = c.scale * (q.abs() @ k.abs().amax(1).unsqueeze(-1)).squeeze(-1)
    es = (2.0 ** -21 + D * 2.0 ** -24) * A + 2.0 ** -20
    shape = (B, Hq, n_q)
    eo = 2 * es * v.abs().amax((1, 2)).unsqueeze(-1)
    el = es + 2.0 ** -22 * torch.where(lse > -math.inf, lse, 0.0).abs()
    return out.view(shape + (D,)), lse.view(shape), eo.view(shape + (1,)), el.view(shape)


@pytest.mark.parametrize("n_splits", [0, 2, 3])
def test_more_pairs_than_counters(n_splits):
    B, Hq, n_q = 1030, 16, 64  # 64 virtual heads of 16 rows each
    r = np.random.default_rng(3)
    lens = r.integers(0, 48, B)
    lens[:5] = 0, 1, 47, 16, 0
    lens = lens.tolist()
    c = Case(B, Hq, 1, 64, lens, n_q=n_q, page=16, seed=4)
    lens[7], lens[8] = 40, 41
    parts = list(kv4.unpack_blocks(c.kv4.cpu().numpy()))
    parts[1][c.table_np[7, 2], 0, 0, 3, 1] = 0x7F  # token 35 of sequence 7: NaN keys
    parts[3][c.table_np[8, 0], 0, 0, 5, 2] = 0x7F  # token 5 of sequence 8: NaN values, channels 32 to 47
    c.kv4 = torch.from_numpy(kv4.pack_blocks(*parts)).cuda()
    want, wl, eo, el = formula(c, lens)
    out, lse = c.run(n_splits, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    assert fd.workspace_status() == 0
    rest = torch.ones(B, dtype=torch.bool, device="cuda")
    rest[7:9] = False
    assert torch.equal(torch.isneginf(lse), torch.isneginf(wl))
    some = wl > -math.inf
    assert bool((torch.where(some, lse - wl, 0.0).abs() <= el)[rest].all())
    assert bool(((out - want).abs() <= eo)[rest].all()) and bool((out[~some] == 0).all())
    # row i of sequence 7 sees keys below 40 - (63 - i): the NaN key from row 59 on
    assert torch.isnan(out[7, :, 59:]).all() and torch.isnan(lse[7, :, 59:]).all()
    assert bool(((out - want).abs() <= eo)[7, :, :59].all())
    # sequence 8: token 5 is one of the window's own, so it shows in its channels in every row that sees a key
    assert torch.isnan(out[8, :, 28:, 32:48]).all() and not torch.isnan(lse[8]).any()
    assert bool(((out - want).abs() <= eo)[8, :, :, :32].all())
