"""GPU tests of a prompt chunk over a 4-bit cache: rows appended, read back, and attended by fd_prefill.

The read-back's bf16 values are the cache's exactly, so the prefill is held to its own bound against the oracle on them,
|out - ref| <= 1e-4 (1 + |ref|); the same window through decode_kv4, where it is short enough, to its own.
"""

import pytest
import torch

import oracle
import split_kv_decode_fd_gb300 as fd

from test_gpu_decode_kv4 import Case, np64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [0, 16, 48])
@pytest.mark.parametrize("Hq,n_q,lens", [(8, 200, [700, 333, 200]), (6, 65, [64, 1000, 0]), (8, 40, [300, 39, 77])])
@pytest.mark.parametrize("causal", [True, False])
def test_read_then_prefill(D, page, Hq, n_q, lens, causal):
    c = Case(3, Hq, 2, D, lens, n_q=n_q, page=page, seed=D + page + n_q)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k, v = fd.kv4_read(c.kv4, max(lens), seq_lens=ln, max_seq_len=c.cap, block_table=c.table)
    out, lse = fd.prefill(c.q, k, v, causal=causal, seq_lens=ln, max_seq_len=max(lens), scale=c.scale)
    assert fd.workspace_status() == 0
    ro, rl = oracle.decode_rows(np64(c.q), c.k, c.v, c.scale, causal=causal, seq_lens=lens, max_seq_len=c.cap)
    got, ls = np64(out), np64(lse)
    assert (abs(got - ro) <= 1e-4 * (1 + abs(ro))).all()
    some = rl > -1e300
    assert ((ls > -1e300) == some).all() and (abs(ls[some] - rl[some]) <= 1e-4 * (1 + abs(rl[some]))).all()
    if n_q <= 64:
        c.check(*c.run(causal=causal), causal=causal)


@pytest.mark.parametrize("page", [0, 16])
def test_a_prompt_in_chunks(page):
    """Chunks appended to a 4-bit cache; each attends all rows so far."""
    g = torch.Generator(device="cuda").manual_seed(page)
    B, Hq, Hkv, D, cap = 2, 8, 2, 128, 512
    table = torch.randperm(B * cap // page, generator=g, device="cuda").view(B, -1).int() if page else None
    kv = fd.kv4_cache(B * cap // page if page else B, Hkv, page or cap, D)
    ang = torch.rand((cap, D // 2), generator=g, device="cuda") * 6.0
    cos, sin = ang.cos(), ang.sin()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    for n, new in ((150, [150, 90]), (200, [200, 200]), (100, [33, 0])):
        x = torch.randn((B, n, Hq + 2 * Hkv, D), generator=g, device="cuda").bfloat16()
        nl = torch.tensor(new, dtype=torch.int32, device="cuda")
        q = fd.append_rope_kv4(x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], kv, cos, sin, q=x[:, :, :Hq], new_lens=nl,
                               seq_lens=lens, max_seq_len=cap - n, block_table=table)
        lens = lens + nl
        k, v = fd.kv4_read(kv, cap, seq_lens=lens, block_table=table)
        out, lse = fd.prefill(q, k, v, causal=True, seq_lens=lens, max_seq_len=cap)
        assert fd.workspace_status() == 0
        ro, rl = oracle.decode_rows(np64(q), np64(k), np64(v), D ** -0.5, causal=True, seq_lens=lens.tolist(), max_seq_len=cap)
        assert (abs(np64(out) - ro) <= 1e-4 * (1 + abs(ro))).all()
        some = rl > -1e300
        assert (abs(np64(lse)[some] - rl[some]) <= 1e-4 * (1 + abs(rl[some]))).all()
