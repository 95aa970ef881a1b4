"""GPU tests of the appended rows and of the read-back where places come near the end of 32 bits."""

import pytest
import torch

import split_kv_decode_fd_gb300 as fd

pytestmark = pytest.mark.gpu
PAGE = 1 << 20
END = 2 ** 31 - 257  # the longest sequence of a 4-bit cache


def one_page(D, Hkv=2):
    """A pool of one page that stands for every part of a sequence."""
    g = torch.Generator(device="cuda").manual_seed(D)
    pool = torch.randint(0, 120, (1, Hkv, PAGE // 16, 18 * D), dtype=torch.uint8, device="cuda", generator=g)
    return pool, torch.zeros((1, -(-END // PAGE)), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("back,n", [(5, 512), (0, 33), (300, 300), (1, 100000)])
def test_reads_that_start_near_the_end(D, back, n):
    """Rows past the length are asked for, and left as they were."""
    pool, table = one_page(D)
    at = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    ko, vo = (torch.full((1, 2, n, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fd.kv4_read(pool, n, starts=at(END - back), seq_lens=at(END), max_seq_len=END, block_table=table, k_out=ko, v_out=vo)
    want = fd.kv4_read(pool, back or 1, starts=at((END - back) % PAGE))
    assert fd.workspace_status() == 0
    for got, w in zip((ko, vo), want):
        assert torch.equal(got[:, :, :back].view(torch.int16), w[:, :, :back].view(torch.int16))
        assert bool((got[:, :, back:] == 3.0).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 20, 40])
def test_appends_up_to_the_end(D, n):
    pool, table = one_page(D)
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn((1, n, 4, D), device="cuda", generator=g)
    lens = torch.tensor([END - n], dtype=torch.int32, device="cuda")
    small = pool.clone()
    fd.append_rope_kv4(x[:, :, :2], x[:, :, 2:], pool, seq_lens=lens, max_seq_len=END - n, block_table=table)
    fd.append_rope_kv4(x[:, :, :2], x[:, :, 2:], small, seq_lens=lens % PAGE)
    assert fd.workspace_status() == 0
    assert torch.equal(pool, small)
