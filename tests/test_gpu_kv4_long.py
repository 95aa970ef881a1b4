"""GPU tests of the appended rows and of the read-back where places come near the end of 32 bits."""

import pytest
import torch

import split_kv_decode_fd_gb300 as fd
from split_kv_decode_fd_gb300 import fdecode as fdb

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


@pytest.mark.parametrize("n", [4000, 2 ** 31 - 15, 2 ** 31 - 1])
def test_a_read_of_more_rows_than_a_sequence_can_have(n):
    """One head, so that only the rows of tokens that exist are within the output's memory."""
    g = torch.Generator(device="cuda").manual_seed(1)
    kv = torch.randint(0, 120, (1, 1, 8, 18 * 64), dtype=torch.uint8, device="cuda", generator=g)
    lens, starts = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (100, 30))
    ko, vo = (torch.full((80, 64), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    desc = fdb.Kv4Desc(layout=fdb.FD_KV_CONTIGUOUS, kv=kv.data_ptr(), capacity=128)
    assert fd.load_library().fd_kv4_read(desc, ko.data_ptr(), vo.data_ptr(), fdb.FD_BF16, 1, n, 1, starts.data_ptr(),
                                         lens.data_ptr(), 128, 64, ws.data_ptr(), 256,
                                         torch.cuda.current_stream().cuda_stream) == fdb.FD_OK
    want = fd.kv4_read(kv, 70, starts=starts)
    torch.cuda.synchronize()
    for got, w in zip((ko, vo), want):
        assert torch.equal(got[:70].view(torch.int16), w[0, 0].view(torch.int16))
        assert bool((got[70:] == 3.0).all())


@pytest.mark.parametrize("D,Hq,n_q", [(64, 4, 1), (128, 8, 2)])
def test_decode_of_the_longest_sequence(D, Hq, n_q):
    """2^31 - 257 tokens, one page 2047 times and a part of it, against 64 bits.

    With F = 2^31 / 128 / 8 / (CTAs) sums of O over the tiles of a group and as many of the weights, each rounded by 2^-25
    of a sum that |v| bounds, and scores within (2^-21 + D 2^-24) A: out is off by (2 (that) + 4 F 2^-24 + 2^-19) max |v|.
    """
    pool, table = one_page(D, 1)
    pool[..., 16 * D:] = pool[..., 16 * D:] % 17 + 0x28  # scales of 1 / 8 to 1 / 2
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((1, Hq, n_q, D), device="cuda", generator=g) * 0.3
    lens = torch.tensor([END], dtype=torch.int32, device="cuda")
    out, lse = fd.decode_kv4(q, pool, seq_lens=lens, max_seq_len=END, block_table=table)
    assert fd.workspace_status() == 0
    k, v = (x[0, 0].double() for x in fd.kv4_read(pool, PAGE, dtype=torch.float32))
    times = torch.full((n_q, PAGE), float(END // PAGE), dtype=torch.float64, device="cuda")
    for i in range(n_q):
        times[i, :END % PAGE - (n_q - 1 - i)] += 1
    w = torch.exp(q[0].double() @ k.t() * D ** -0.5) * times
    L = w.sum(-1, keepdim=True)
    want, wl = w @ v / L, L[..., 0].log()
    A = (q[0].double().abs() @ k.abs().amax(0)) * D ** -0.5
    es = (2.0 ** -21 + D * 2.0 ** -24) * A
    F = 2 ** 31 / 128 / 8 / torch.cuda.get_device_properties(0).multi_processor_count
    far = 4 * F * 2.0 ** -24 + 2.0 ** -19
    assert bool(((out[0] - want).abs() <= (2 * es[..., None] + far) * v.abs().max()).all())
    assert bool(((lse[0] - wl).abs() <= es + far + 2.0 ** -22 * wl.abs()).all())
