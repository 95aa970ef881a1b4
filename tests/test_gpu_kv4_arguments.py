"""GPU tests of the arguments of the appends, the read-back and the 4-bit decode: what is taken, and what is refused how."""

import pytest
import torch

import split_kv_decode_fd_gb300 as fd

pytestmark = pytest.mark.gpu


def cache(B=2, Hkv=2, tokens=64, D=64, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 120, (B, Hkv, tokens // 16, 18 * D), dtype=torch.uint8, device="cuda", generator=g)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("given", ["k_out", "v_out"])
def test_one_given_output_says_the_type_of_both(dtype, given):
    kv = cache()
    want = fd.kv4_read(kv, 64, dtype=dtype)
    out = torch.zeros_like(want[0])
    got = fd.kv4_read(kv, 64, **{given: out})
    assert got[given == "v_out"] is out and all(x.dtype is dtype for x in got)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
