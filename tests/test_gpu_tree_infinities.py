"""GPU tests of tree attention with infinities in places that every token sees.

Over an fp32 cache the output is what the formula gives.  Over a bf16 cache it may be NaN instead, as q and the weights are sums of three
bf16 numbers there, of which some are 0; what does not see the infinity is the same bit for bit.
"""

import math

import numpy as np
import pytest
import torch

import split_kv_decode_fd_gb300 as fd
from test_gpu_decode_tree import Case

pytestmark = pytest.mark.gpu


def case(cache, Hq, n, page):
    return Case(3, Hq, 2, 128, n, [300, 1500, 64 + n], cache=cache, page=page, seed=Hq + n)


@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,n", [(4, 6), (8, 16), (8, 30)])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("bad", [math.inf, -math.inf])
def test_a_value_before_the_drafts(cache, Hq, n, page, bad):
    c = case(cache, Hq, n, page)
    out, lse = c.run()
    want = out.clone()
    want[1, Hq // 2:, :, 7] = bad  # weights are above 0
    b, heads, t = c.place(1, 700)
    c.v[b, 1, t, 7] = bad
    got, got_lse = c.run()
    assert torch.equal(got_lse, lse)
    row = got[1, Hq // 2:, :, 7]
    if cache == "bf16":
        assert (torch.isnan(row) | (row == bad)).all()
        got[1, Hq // 2:, :, 7] = bad
    assert torch.equal(got, want)
    assert fd.workspace_status() == 0


@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,n", [(4, 6), (8, 16), (8, 30)])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("place", [700, 1500 - 30])
def test_a_key(cache, Hq, n, page, place):
    """A key of -inf in one channel, before the drafts or that of token 0, which all see: the score is -inf where q is positive,
    which gives it no weight, and +inf, so that the row is NaN, where q is negative."""
    c = case(cache, Hq, n, page)
    out, lse = c.run()
    b, heads, t = c.place(1, place)
    old_k = c.k[b, 1, t].clone()
    h = slice(Hq // 2, Hq)
    q = c.q[1, h].double()
    k = torch.from_numpy(c.k_np[1, 1, :1500]).double().cuda()
    c.k[b, 1, t, 7] = -math.inf
    got, got_lse = c.run()
    assert torch.equal(got[[0, 2]], out[[0, 2]]) and torch.equal(got_lse[[0, 2]], lse[[0, 2]])
    assert torch.equal(got[1, :Hq // 2], out[1, :Hq // 2]) and torch.equal(got_lse[1, :Hq // 2], lse[1, :Hq // 2])
    up = q[:, :, 7] < 0
    assert torch.isnan(got[1, h][up]).all() and torch.isnan(got_lse[1, h][up]).all()
    # sum of weights without that one: lse + log(1 - exp(score - lse)), in 64 bits from the finite call's lse
    score = (q @ k[place]) * c.scale
    want = lse[1, h].double() + torch.log1p(-torch.exp(score - lse[1, h].double()))
    rest = got_lse[1, h][~up].double()
    # a score is off by at most (2^-21 + 128 * 2^-24) A, A = scale * sum |q k| < 25 here, twice, plus the 2^-20 of exp2: below 1e-3
    near = (rest - want[~up]).abs() < 1e-3
    if cache == "bf16":
        near |= torch.isnan(rest)
    assert near.all()
    c.k[b, 1, t] = old_k
    again, again_lse = c.run()
    assert torch.equal(again, out) and torch.equal(again_lse, lse)
    assert fd.workspace_status() == 0
