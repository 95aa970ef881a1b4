"""GPU tests of the draft's probabilities in the verification of drafted trees, against the float64 oracle."""

import math

import numpy as np
import pytest
import torch

import split_kv_decode_fd_gb300 as fd
from test_gpu_verify_tree import Case

pytestmark = pytest.mark.gpu


def childless(c):
    """Truth values [B, n]: rows of padding, and rows of tokens without children."""
    rows = np.ones((c.B, c.n), dtype=bool)
    for b in range(c.B):
        pad = c.n - (c.n if c.new_lens is None else c.new_lens[b])
        for j in range(pad + 1, c.n):
            if c.parents[b, j] >= 0 and 0 <= c.tokens[b, j] < c.V:
                rows[b, pad + c.parents[b, j]] = False
    return torch.from_numpy(rows).cuda()


def equal(got, want):
    return all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(got, want))


@pytest.mark.parametrize("V", [1, 7, 1000, 4097, 50000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", ["chain", "random", "wide"])
@pytest.mark.parametrize("agree", [0.9, 1.0])
def test_rows_of_tokens_without_children_are_not_read(V, dtype, shape, agree):
    """A draft model has no reason to write them: NaN, infinities and numbers that are no probabilities."""
    c = Case(6, 7, V, dtype=dtype, shape=shape, agree=agree, new_lens=[7, 1, 4, 7, 0, 2], seed=V)
    want = c.want()
    rows = childless(c)
    for bad in (math.nan, math.inf, -math.inf, -1.0, 1e30):
        draft = c.draft.clone()
        draft[rows] = bad
        assert equal(c.run(draft=draft), want), bad
    # rows at odd addresses of their own, where the draft's would not be loaded 16 bytes at a time
    for off in (1, 3):
        flat = torch.full((c.draft.numel() + off,), math.nan, dtype=c.draft.dtype, device="cuda")
        draft = flat[off:].view(c.draft.shape)
        draft[~rows] = c.draft[~rows]
        assert equal(c.run(draft=draft), want), off
    assert fd.workspace_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_are_not_read_in_a_large_batch(dtype):
    c = Case(320, 5, 3001, dtype=dtype, agree=0.97, seed=2)
    want = c.want()
    draft = c.draft.clone()
    draft[childless(c)] = math.nan
    assert equal(c.run(draft=draft), want)


def test_the_row_of_a_token_whose_only_child_is_left_out():
    c = Case(3, 4, 900, shape="chain", agree=1.0, seed=3)
    c.uniforms[:, 1:] = 0.0  # every child stays
    c.tokens[:, 3] = [900, -1, 1 << 30]
    want = c.run()
    assert fd.workspace_status() == fd.fdecode.FD_ERR_BAD_INDEX and want[1].tolist() == [3, 3, 3]
    draft = c.draft.clone()
    draft[childless(c)] = math.nan
    got = c.run(draft=draft)
    assert fd.workspace_status() == fd.fdecode.FD_ERR_BAD_INDEX
    assert all(torch.equal(g, w) for g, w in zip(got, want)) and (got[2] >= 0).all()


@pytest.mark.parametrize("V", [3, 601, 5000, 40001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", ["chain", "random", "wide"])
@pytest.mark.parametrize("none", [math.nan, -math.inf, -1.0, -1e-30, -0.0])
def test_what_is_no_draft_probability_counts_as_zero(V, dtype, shape, none):
    """In a third of the words, those of some children among them."""
    c = Case(6, 9, V, dtype=dtype, shape=shape, agree=0.7, new_lens=[9, 3, 9, 6, 2, 9], seed=V)
    out = torch.from_numpy(np.random.default_rng(V).random(c.draft.shape) < 1 / 3).cuda()
    c.draft[out] = 0.0
    want = c.want()
    clean = c.run()
    c.draft[out] = none
    got = c.run()
    assert equal(clean, want) and equal(got, want)
    c.check(got)  # and the oracle's own reading of such numbers
    assert fd.workspace_status() == 0
