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


def test_what_is_no_tensor_is_refused_as_a_value():
    kv = cache()
    x = torch.zeros((2, 1, 2, 64), device="cuda")
    q = torch.zeros((2, 4, 64), device="cuda")
    k = torch.zeros((2, 2, 64, 64), device="cuda")
    cos = torch.zeros((64, 16), device="cuda")
    flat = torch.zeros((18 * 64,), dtype=torch.uint8, device="cuda")
    for name, call in {
        "block_table": lambda: fd.kv4_read(kv, 4, block_table=[[0, 1], [2, 3]]),
        "k_out": lambda: fd.kv4_read(kv, 4, k_out=[1.0]),
        "v_out": lambda: fd.kv4_read(kv, 4, v_out=3.0),
        "kv4": lambda: fd.kv4_read(flat[0], 4),
        "cos": lambda: fd.append_rope_kv4(x, x, kv, cos.tolist(), cos, seq_lens=None),
        "sin": lambda: fd.append_rope(x, x, k, k.clone(), cos, "sin"),
    }.items():
        with pytest.raises(ValueError, match=name):
            call()
    for call in (lambda: fd.kv4_read(flat, 4), lambda: fd.decode_kv4(q, flat), lambda: fd.append_rope_kv4(x, x, flat)):
        with pytest.raises(ValueError, match="kv4"):
            call()
    for call in (lambda: fd.decode_kv4(q, kv, block_table=(0, 1)), lambda: fd.append_rope_kv4(x, x, kv, block_table=7),
                 lambda: fd.append_rope(x, x, k, k.clone(), block_table=[0])):
        with pytest.raises(ValueError, match="block_table"):
            call()


def test_numbers_past_32_bits_are_refused():
    """They are not cut down to their lowest 32 bits."""
    kv = cache(1, 1, 1 << 20)
    table = torch.zeros((1, 4097), dtype=torch.int32, device="cuda")  # 2^32 + 2^20 places
    q = torch.ones((1, 2, 64), device="cuda")
    x = torch.zeros((1, 1, 1, 64), device="cuda")
    big = 2 ** 32 + 16
    small = cache(1, 1, 64)
    for name, call in [
        ("max_seq_len", lambda: fd.decode_kv4(q, kv, block_table=table)),
        ("max_seq_len", lambda: fd.kv4_read(kv, 4, block_table=table)),
        ("max_seq_len", lambda: fd.append_rope_kv4(x, x, kv, block_table=table)),
        ("max_seq_len", lambda: fd.decode_kv4(q, small, max_seq_len=big)),
        ("max_seq_len", lambda: fd.decode_kv4(q, small, max_seq_len=-big)),
        ("max_seq_len", lambda: fd.kv4_read(small, 4, max_seq_len=big)),
        ("max_seq_len", lambda: fd.append_rope_kv4(x, x, small, max_seq_len=big)),
        ("n_splits", lambda: fd.decode_kv4(q, small, n_splits=big)),
        ("n ", lambda: fd.kv4_read(small, big, k_out=x[:, :, :, :], v_out=x)),
        ("n ", lambda: fd.append_rope_kv4(x.expand(1, big, 1, 64), x.expand(1, big, 1, 64), small)),
    ]:
        with pytest.raises(ValueError, match=name):
            call()
    out, _ = fd.decode_kv4(q, kv, block_table=table, max_seq_len=1 << 20)
    assert torch.isfinite(out).all() and fd.workspace_status() == 0


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_of_single_entries_do_not_matter(four, dtype):
    """A dimension of one entry is never stepped along, whatever its stride."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((1, 1, 1, 64), dtype=torch.float32, device="cuda", generator=g).to(dtype)
    odd = x.as_strided((1, 1, 1, 64), (5, 3, 7, 1))
    got = []
    for rows in (x, odd):
        if four:
            kv = torch.zeros((1, 1, 2, 18 * 64), dtype=torch.uint8, device="cuda")
            q = fd.append_rope_kv4(rows, rows, kv, q=rows)
        else:
            kv = torch.zeros((2, 1, 1, 32, 64), device="cuda")
            q = fd.append_rope(rows, rows, kv[0], kv[1], q=rows)
        got.append((q, kv))
    assert fd.workspace_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(*got)) and bool((got[0][1] != 0).any())
    with pytest.raises(fd.FdError):
        two = torch.zeros(200, dtype=dtype, device="cuda").as_strided((1, 2, 1, 64), (5, 65, 7, 1))
        fd.append_rope_kv4(two, two, torch.zeros((1, 1, 2, 18 * 64), dtype=torch.uint8, device="cuda"))
