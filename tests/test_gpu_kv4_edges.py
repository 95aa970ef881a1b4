"""GPU tests of the appended rows, the read-back and the 4-bit decode attention at their edges: waits that run out,
scores near the ends of fp32, rows at 16-byte addresses, graphs that share a workspace, pools past 32 bits."""

import math

import numpy as np
import pytest
import torch

import split_kv_decode_fd_gb300 as fd
from split_kv_decode_fd_gb300 import fdecode as fdb

from test_gpu_decode_kv4 import Case, np64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,page", [(4, 0), (8, 16), (32, 16)])
def test_scores_near_the_ends_of_fp32(Hq, page):
    """One key: the output is its value, whatever the score.  Several: the largest score's value alone, as scores of
    this size lie far more than 2^20 apart."""
    for size in (1e7, 2e8, 3e9, 1e20, 1e31, 1e-30):
        c = Case(3, Hq, 2, 64, [1, 1, 600], page=page, seed=11, q_gain=size)
        out, lse = c.run()
        assert fd.workspace_status() == 0
        g = Hq // 2
        v = np.repeat(c.v, g, 1)
        assert np.abs(np64(out)[:2, :, 0] - v[:2, :, 0]).max() <= 2.0 ** -20 * np.abs(v).max()
        s = np.einsum("bhd,bhtd->bht", np64(c.q)[:, :, 0], np.repeat(c.k, g, 1)) * c.scale
        A = np.einsum("bhd,bhd->bh", np.abs(np64(c.q)[:, :, 0]), np.repeat(np.abs(c.k).max(2), g, 1)) * c.scale
        err = (2.0 ** -20 + 64 * 2.0 ** -23) * A + 2.0 ** -19
        assert np.all(np.abs(np64(lse)[:2, :, 0] - s[:2, :, 0]) <= err[:2])
        top = s[2, :, :600].max(-1)
        assert np.all(np.abs(np64(lse)[2, :, 0] - top) <= err[2] + math.log(600))
        if size >= 1e20:
            order = np.argsort(s[2, :, :600], -1)
            for h in range(Hq):
                a, b = order[h, -1], order[h, -2]
                if s[2, h, a] - s[2, h, b] > 2 * err[2, h]:
                    assert np.abs(np64(out)[2, h, 0] - v[2, h, a]).max() <= 2.0 ** -20 * np.abs(v).max()
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("gain", [-1.0, 1.0])
def test_scores_past_the_range_of_floats_do_not_hang(gain):
    c = Case(2, 4, 2, 64, [300, 300], seed=12, k_exp=64, q_gain=1.0)
    c.q.fill_(gain * 3e38)
    out, lse = c.run()
    assert fd.workspace_status() == 0
    assert not torch.isfinite(lse).any()


@pytest.mark.parametrize("Hq,n_splits", [(4, 0), (16, 0), (8, 5)])
@pytest.mark.parametrize("page", [0, 16])
def test_infinite_queries_show_as_nan(Hq, n_splits, page):
    c = Case(2, Hq, 2, 128, [700, 700], page=page, seed=13)
    good, _ = c.run(n_splits)
    c.q[1, 1, 0, 5] = float("inf")
    out, lse = c.run(n_splits)
    assert torch.isnan(out[1, 1]).all() and torch.isnan(lse[1, 1]).all()
    out[1, 1] = good[1, 1] = 0.0
    # references move at other tiles: twice the bound of a result (A < 40, |v| < 8), not the same bits
    assert (out - good).abs().max() <= 2 * 2 * ((2.0 ** -21 + 128 * 2.0 ** -24) * 40 + 2.0 ** -20) * 8


def shifted(t, floats):
    """A copy of t that starts `floats` * 4 bytes past an allocation's address."""
    n = floats * 4 // t.element_size()
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
    out = buf[n:].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rot", [0, 32])
def test_rows_at_16_byte_addresses(D, dtype, rot):
    """The same results where no buffer starts on a 32-byte boundary."""
    g = torch.Generator(device="cuda").manual_seed(D)
    B, n, Hq, Hkv, cap = 2, 19, 4, 2, 64
    x = torch.randn((B, n, Hq + 2 * Hkv, D), generator=g, device="cuda").to(dtype)
    ang = torch.rand((cap, rot // 2), generator=g, device="cuda")
    lens = torch.tensor([3, 40], dtype=torch.int32, device="cuda")
    got = []
    for move in (0, 4):
        y = shifted(x, move)
        cos, sin = (shifted(ang.cos(), move), shifted(ang.sin(), move)) if rot else (None, None)
        k = shifted(torch.zeros((B, Hkv, cap, D), dtype=dtype, device="cuda"), move)
        v = shifted(torch.zeros_like(k), move)
        kv = shifted(fd.kv4_cache(B, Hkv, cap, D).zero_(), move)
        qo = [shifted(torch.zeros((B, Hq, n, D), device="cuda"), move) for _ in range(2)]
        how = dict(q=y[:, :, :Hq], seq_lens=lens, max_seq_len=cap - n)
        fd.append_rope(y[:, :, Hq:Hq + Hkv], y[:, :, Hq + Hkv:], k, v, cos, sin, q_out=qo[0], **how)
        fd.append_rope_kv4(y[:, :, Hq:Hq + Hkv], y[:, :, Hq + Hkv:], kv, cos, sin, q_out=qo[1], **how)
        ko, vo = (shifted(torch.zeros((B, Hkv, cap, D), dtype=dtype, device="cuda"), move) for _ in range(2))
        fd.kv4_read(kv, cap, seq_lens=lens + n, k_out=ko, v_out=vo)
        out, lse = fd.decode_kv4(qo[1], kv, seq_lens=lens + n, max_seq_len=cap,
                                 out=shifted(torch.zeros((B, Hq, n, D), device="cuda"), move))
        got.append([t.clone() for t in (k, v, kv, qo[0], qo[1], ko, vo, out, lse)])
    assert fd.workspace_status() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert torch.equal(got[0][3], got[0][4]) and got[0][0].abs().sum() > 0 and got[0][5].abs().sum() > 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rot,interleaved", [(0, False), (64, False), (64, True), (32, False), (32, True)])
@pytest.mark.parametrize("page", [0, 16])
def test_tokens_one_by_one_give_the_bytes_of_all_at_once(D, dtype, rot, interleaved, page):
    g = torch.Generator(device="cuda").manual_seed(D + rot + page)
    B, n, Hq, Hkv, cap = 3, 38, 4, 2, 64
    x = torch.randn((B, n, Hq + 2 * Hkv, D), generator=g, device="cuda").to(dtype)
    x[1, 5, :, 16:32] = 0.0
    x[2, 7, Hq, 3] = float("nan")
    x[0, 30, Hq + Hkv, 40] = float("inf")
    table = torch.randperm(B * cap // page, generator=g, device="cuda").view(B, -1).int() if page else None
    ang = torch.rand((cap, rot // 2), generator=g, device="cuda")
    cos, sin = (ang.cos(), ang.sin()) if rot else (None, None)
    got = []
    for step in (n, 1, 2, 3, 4, 5):
        kv = fd.kv4_cache(B * cap // page if page else B, Hkv, page or cap, D)
        lens = torch.tensor([0, 11, 25], dtype=torch.int32, device="cuda")
        q = []
        for at in range(0, n, step):
            y = x[:, at:at + step]
            q.append(fd.append_rope_kv4(y[:, :, Hq:Hq + Hkv], y[:, :, Hq + Hkv:], kv, cos, sin, q=y[:, :, :Hq], k_exp=1,
                                        v_exp=-2, interleaved=interleaved, seq_lens=lens,
                                        max_seq_len=cap - y.shape[1], block_table=table))
            lens += y.shape[1]
        got.append((kv, torch.cat(q, 2)))
    assert fd.workspace_status() == 0
    for kv, q in got[1:]:
        assert torch.equal(kv, got[0][0]) and torch.equal(q.view(torch.int32), got[0][1].view(torch.int32))


def test_two_captured_graphs_share_a_workspace():
    a = Case(3, 8, 2, 128, [900, 33, 512], page=16, seed=3)
    b = Case(5, 32, 2, 64, [2000, 1, 700, 0, 64], seed=4)
    ws = fd.Workspace()
    want = [[t.clone() for t in c.run(workspace=ws)] for c in (a, b)]
    lens = [torch.tensor(c.lens, dtype=torch.int32, device="cuda") for c in (a, b)]
    a.run(workspace=ws, seq_lens=lens[0])
    graphs, outs = [], []
    for c, ln in zip((a, b), lens):
        o = [torch.zeros_like(t) for t in want[len(graphs)]]
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.run(workspace=ws, seq_lens=ln, out=o[0], lse=o[1])
        graphs.append(gr)
        outs.append(o)
    for i in (0, 1, 1, 0, 1, 0):
        for t in outs[i]:
            t.fill_(7.0)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs[i], want[i]))
    assert fd.workspace_status(ws) == 0


@pytest.mark.parametrize("page", [0, 16])
def test_steps_replayed_on_another_stream(page):
    """A captured step (append, decode, read) replayed while lengths move on, against the same steps run one by one."""
    g = torch.Generator(device="cuda").manual_seed(5 + page)
    B, Hq, Hkv, D, cap, steps = 3, 8, 2, 128, 96, 20
    table = torch.randperm(B * cap // page, generator=g, device="cuda").view(B, -1).int() if page else None
    ang = torch.rand((cap, D // 2), generator=g, device="cuda")
    cos, sin = ang.cos(), ang.sin()
    xs = torch.randn((steps, B, 1, Hq + 2 * Hkv, D), generator=g, device="cuda").bfloat16()

    def state():
        kv = fd.kv4_cache(B * cap // page if page else B, Hkv, page or cap, D).zero_()
        return dict(kv=kv, lens=torch.tensor([0, 15, 70], dtype=torch.int32, device="cuda"), x=torch.empty_like(xs[0]),
                    q=torch.zeros((B, Hq, 1, D), device="cuda"), out=torch.zeros((B, Hq, 1, D), device="cuda"),
                    lse=torch.zeros((B, Hq, 1), device="cuda"), ws=fd.Workspace(),
                    k=torch.zeros((B, Hkv, cap, D), device="cuda"), v=torch.zeros((B, Hkv, cap, D), device="cuda"))

    def step(s):
        x = s["x"]
        fd.append_rope_kv4(x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], s["kv"], cos, sin, q=x[:, :, :Hq], q_out=s["q"],
                           seq_lens=s["lens"], max_seq_len=cap - 1, block_table=table, workspace=s["ws"])
        s["lens"].add_(1)
        fd.decode_kv4(s["q"], s["kv"], seq_lens=s["lens"], max_seq_len=cap, block_table=table, out=s["out"],
                      lse=s["lse"], workspace=s["ws"])
        fd.kv4_read(s["kv"], cap, seq_lens=s["lens"], block_table=table, k_out=s["k"], v_out=s["v"], workspace=s["ws"])

    one, two = state(), state()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        two["x"].copy_(xs[0])
        step(two)  # sizes the workspace
        two["kv"].zero_()
        two["lens"].copy_(torch.tensor([0, 15, 70], dtype=torch.int32))
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(two)
    for x in xs:
        one["x"].copy_(x)
        step(one)
        two["x"].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("kv", "lens", "q", "out", "lse", "k", "v"):
            assert torch.equal(one[name], two[name]), name
    assert fd.workspace_status(one["ws"]) == 0 and fd.workspace_status(two["ws"]) == 0


def test_outputs_and_workspaces_are_made_on_the_streams_of_the_calls():
    """Calls on a stream of their own while the current one is busy: nothing that they make waits for it."""
    g = torch.Generator(device="cuda").manual_seed(9)
    B, n, Hq, Hkv, D, cap = 2, 5, 4, 2, 64, 64
    x = torch.randn((B, n, Hq + 2 * Hkv, D), generator=g, device="cuda")
    new = torch.tensor([5, 2], dtype=torch.int32, device="cuda")
    lens = torch.tensor([10, 20], dtype=torch.int32, device="cuda")
    ends = lens + new
    kv = fd.kv4_cache(B, Hkv, cap, D)
    k, v = (torch.zeros((B, Hkv, cap, D), device="cuda") for _ in range(2))

    def calls(stream):
        ws = [fd.Workspace() for _ in range(4)] if stream is not None else [None] * 4
        how = dict(q=x[:, :, :Hq], new_lens=new, seq_lens=lens, max_seq_len=cap - n, stream=stream)
        rows = x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
        q = fd.append_rope_kv4(*rows, kv, workspace=ws[0], **how)
        q2 = fd.append_rope(*rows, k, v, workspace=ws[1], **how)
        ko, vo = fd.kv4_read(kv, cap, seq_lens=ends, workspace=ws[2], stream=stream)
        out, lse = fd.decode_kv4(q, kv, seq_lens=ends, max_seq_len=cap, workspace=ws[3], stream=stream)
        return (q, q2, ko, vo, out, lse), ws

    want, _ = calls(None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    got, ws = calls(s)
    s.synchronize()
    early = [t.cpu() for t in want]  # waits for the current stream
    torch.cuda.synchronize()
    assert all(torch.equal(a, b.cpu()) for a, b in zip(early, got))
    assert all(fd.workspace_status(w) == 0 for w in ws)
    assert got[0][1, :, :3].abs().max() == 0 and got[0][1, :, 3:].abs().min() > 0


def test_decode_of_pages_past_32_bits():
    c = Case(2, 8, 2, 128, [500, 70], page=16, seed=14)
    want = [t.clone() for t in c.run()]
    pages, per = 560000, 2 * 18 * 128  # 2.58 GB
    pool = torch.zeros((pages, 2, 1, 18 * 128), dtype=torch.uint8, device="cuda")
    at = torch.arange(c.table.numel(), device="cuda") * 17 + (2 ** 31 // per + 5)
    pool[at] = c.kv4[c.table.flatten().long()].view(-1, 2, 1, 18 * 128)
    assert int(at.min()) * per > 2 ** 31 and int(at.max()) < pages
    c.kv4, c.table = pool, at.int().view_as(c.table)
    got = c.run()
    assert fd.workspace_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))


LONG = [16000, 300, 0, 129]
MANY = [300 - 37 * (i % 8) for i in range(200)]


@pytest.mark.parametrize("lens,Hq,page,n_splits,stage", [
    (LONG, 4, 0, 0, 0), (LONG, 8, 16, 0, 2), (LONG, 64, 16, 0, 1), (LONG, 16, 0, 2, 0), (LONG, 4, 16, 2, 30),
    (MANY, 4, 16, 0, 0), (MANY, 16, 0, 0, 5), (MANY, 64, 16, 0, 7),
])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_clean(lens, Hq, page, n_splits, stage):
    """One tile's copy is skipped in every CTA that has so many, and waits give up after 1 ms: the call reports it,
    leaves the workspace's counters as they were, and the next one is right."""
    c = Case(len(lens), Hq, 4, 64, lens, page=page, seed=15)
    want = [t.clone() for t in c.run(n_splits)]
    ws = fd.Workspace()
    lib = fd.load_library()
    try:
        lib.fd_debug_stall(stage, 1_000_000)
        c.run(n_splits, workspace=ws)
        assert fd.workspace_status(ws) == fdb.FD_ERR_TIMEOUT
    finally:
        lib.fd_debug_stall(-1, 0)
    assert fd.workspace_status(ws) == 0
    got = c.run(n_splits, workspace=ws)
    assert fd.workspace_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))
