"""GPU tests of the joins of tree attention where there are more (sequence, KV head) pairs than shares of the keys.

A share then has one entry, which says which pair it begins and leaves unfinished.  The batches have shares whose first piece is
such a pair: there the entry is written right after the walk has begun.  Outputs hold NaN before each call, so that a pair that is not joined shows.
"""

import math

import numpy as np
import pytest
import torch

import split_kv_decode_fd_gb300 as fd
from test_gpu_decode_tree import Case, exact_on_the_gpu

pytestmark = pytest.mark.gpu

TILE = {"bf16": 128, "f32": 64}
PIECE = {"bf16": 12, "f32": 4}  # cost units of a piece, four a tile


def first_pieces_that_go_on(lens, heads, shares, cache):
    """How many shares begin with a pair that later shares go on with: the shares are equal parts of the line of cost units."""
    units = [4 * -(-L // TILE[cache]) + PIECE[cache] if L else 0 for L in lens for _ in range(heads)]
    starts = np.concatenate([[0], np.cumsum(units)])
    total = int(starts[-1])
    used = min(shares, total // 4)
    found = 0
    for r in range(used):
        pos, end = total * r // used, total * (r + 1) // used
        pair = int(np.searchsorted(starts, pos, side="right")) - 1
        if pos - starts[pair] <= PIECE[cache] < end - starts[pair] and starts[pair + 1] > end:
            found += 1
    return found


@pytest.mark.parametrize("cache,g,n", [("bf16", 2, 5), ("bf16", 4, 16), ("bf16", 4, 30), ("bf16", 8, 64), ("f32", 2, 5)])
@pytest.mark.parametrize("page", [0, 16])
def test_shares_that_begin_with_a_pair_that_goes_on(cache, g, n, page):
    r = np.random.default_rng(g * n)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    Hkv, D = 2, 128
    blocks = -(-g * n // 128) if cache == "bf16" and g * n > 64 else 1
    shares = (2 if cache == "f32" else 1) * sms // blocks
    B = shares // Hkv + 9  # more pairs than shares
    lens = [int(x) for x in np.where(r.random(B) < 0.15, r.integers(1500, 2500, B), r.integers(1, 300, B))]
    assert first_pieces_that_go_on(lens, Hkv, shares, cache) > 0
    c = Case(B, g * Hkv, Hkv, D, n, lens, cache=cache, page=page, seed=n)
    ro, rl = exact_on_the_gpu(c)
    seq_lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    ws = fd.Workspace()
    first = None
    for _ in range(20):
        out, lse = torch.full_like(c.q, math.nan), torch.full(c.q.shape[:3], math.nan, device="cuda")
        c.run(out=out, lse=lse, workspace=ws, seq_lens=seq_lens)
        if first is None:
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert fd.workspace_status(ws) == 0
    # scores of some units, values of a few: the bound of the head of test_gpu_decode_tree.py is below 1e-4 here
    assert (first[0].double() - ro).abs().max() < 1e-4
    some = torch.isfinite(rl)
    assert torch.equal(torch.isneginf(first[1]), torch.isneginf(rl)) and (first[1].double() - rl)[some].abs().max() < 1e-4
