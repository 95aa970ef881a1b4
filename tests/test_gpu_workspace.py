"""GPU tests of workspaces that grow, and of calls that share one."""

import pytest
import torch

import split_kv_decode_fd_gb300 as fd
from split_kv_decode_fd_gb300 import fdecode as fdb

from test_gpu_decode_kv4 import Case

pytestmark = pytest.mark.gpu


def bf16_run(c):
    """fd_decode of a Case's queries over a bf16 cache."""
    k, v = (torch.from_numpy(x).cuda().bfloat16() for x in (c.k, c.v))
    q = c.q[:, :, 0].contiguous()
    return lambda **kw: fd.decode(q, k, v, max_seq_len=c.cap, scale=c.scale, **kw)


@pytest.mark.parametrize("four", [True, False])
def test_a_captured_graph_outlives_its_workspaces_growth(four):
    small, large = Case(2, 8, 2, 128, [900, 33], seed=1), Case(8, 32, 4, 128, [2000] * 8, seed=2)
    run, run_large = (small.run, large.run) if four else (bf16_run(small), bf16_run(large))
    lens = torch.tensor(small.lens, dtype=torch.int32, device="cuda")
    more = torch.tensor(large.lens, dtype=torch.int32, device="cuda")
    ws = fd.Workspace()
    want = [t.clone() for t in run(workspace=ws, seq_lens=lens)]
    out, lse = (torch.zeros_like(t) for t in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(workspace=ws, seq_lens=lens, out=out, lse=lse)
    size, at = ws.buf.numel(), ws.buf.data_ptr()
    first = [t.clone() for t in run_large(workspace=ws, seq_lens=more)]
    assert ws.buf.numel() > size
    taken = [torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert all(t.data_ptr() != at for t in taken)
    for _ in range(3):
        out.fill_(7.0)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip((out, lse), want))
        assert all(torch.equal(a, b) for a, b in zip(first, run_large(workspace=ws, seq_lens=more)))
    assert all(bool((t == 0x5A).all()) for t in taken)
    assert fd.workspace_status(ws) == 0


@pytest.mark.parametrize("default", [False, True])
def test_errors_raised_before_a_workspace_grew_are_reported(default):
    c = Case(2, 8, 2, 64, [300, 200], page=16, seed=3)
    large = Case(64, 64, 4, 128, [40] * 64, seed=4)
    ws = fd.Workspace()
    how = {} if default else dict(workspace=ws)
    of = [] if default else [ws]
    assert fd.workspace_status(*of) == 0
    table = c.table.clone()
    table[1, 3] = 1 << 20
    lens = torch.tensor([40, 48], dtype=torch.int32, device="cuda")
    x = torch.zeros((2, 1, 2, 64), device="cuda", dtype=torch.bfloat16)
    append = lambda: fd.append_rope_kv4(x, x, c.kv4, seq_lens=lens, max_seq_len=48, block_table=table, **how)  # noqa: E731
    append()
    assert fd.workspace_status(*of) == 4 and fd.workspace_status(*of) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        append()
    append()
    for n_splits, cause in ((7, lambda: None), (40, graph.replay)):
        cause()
        large.run(n_splits=n_splits, **how)
        assert fd.workspace_status(*of) == 4 and fd.workspace_status(*of) == 0
    graph.replay()
    assert fd.workspace_status(*of) == 4 and fd.workspace_status(*of) == 0


def test_a_dropped_workspace_waits_for_the_streams_that_used_it():
    """Its memory is not given out again while a call on another stream still writes there."""
    c = Case(2, 8, 2, 128, [900, 333], page=16, seed=5)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    ws = fd.Workspace()
    want = [t.clone() for t in c.run(workspace=ws, seq_lens=lens)]
    out, lse = (torch.zeros_like(t) for t in want)
    size, at = ws.buf.numel(), ws.buf.data_ptr()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    c.run(workspace=ws, stream=s, seq_lens=lens, out=out, lse=lse)
    del ws
    taken = [torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert not s.query() and all(t.data_ptr() != at for t in taken)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert all(bool((t == 0x5A).all()) for t in taken)


@pytest.mark.parametrize("given", [True, False])
def test_calls_on_two_streams_without_a_workspace(given):
    """Each stream has its own counters and partial states; errors of both are reported."""
    cases = Case(3, 8, 2, 128, [9000, 33, 512], page=16, seed=6), Case(5, 32, 2, 64, [7000, 1, 700, 0, 64], seed=7)
    lens = [torch.tensor(c.lens, dtype=torch.int32, device="cuda") for c in cases]
    want = [[t.clone() for t in c.run(seq_lens=ln)] for c, ln in zip(cases, lens)]
    outs = [[[torch.zeros_like(t) for t in w] for w in want] for _ in range(10)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for o in outs:
        for c, ln, s, (out, lse) in zip(cases, lens, streams, o):
            if given:
                c.run(seq_lens=ln, out=out, lse=lse, stream=s)
            else:
                with torch.cuda.stream(s):
                    c.run(seq_lens=ln, out=out, lse=lse)
    torch.cuda.synchronize()
    for o in outs:
        for got, w in zip(o, want):
            assert all(torch.equal(a, b) for a, b in zip(got, w))
    assert fd.workspace_status() == 0
    cases[0].table[0, 3] = -1
    for s in streams:
        torch.cuda.synchronize()
        cases[0].run(seq_lens=lens[0], stream=s)
        assert fd.workspace_status() == 4 and fd.workspace_status() == 0
        cases[0].run(seq_lens=lens[0], stream=s)
        assert fd.workspace_status(stream=s) == 4 and fd.workspace_status() == 0


def test_a_capture_without_a_workspace_takes_one_that_calls_have_sized(monkeypatch):
    monkeypatch.setattr(fdb, "_STREAM_WS", {})
    c = Case(3, 8, 2, 128, [900, 33, 512], page=16, seed=8)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        want = [t.clone() for t in c.run(seq_lens=lens)]
    s.synchronize()
    out, lse = (torch.zeros_like(t) for t in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(seq_lens=lens, out=out, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    with pytest.raises(RuntimeError, match="capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            c.run(n_splits=60000, seq_lens=lens, out=out, lse=lse)
    assert fd.workspace_status() == 0


def test_a_capture_without_a_workspace_may_take_the_devices(monkeypatch):
    """Only calls that share one per device have run before."""
    monkeypatch.setattr(fdb, "_STREAM_WS", {})
    c = Case(2, 8, 2, 128, [60, 33], seed=9)
    bf16_run(c)()
    x = torch.randn((2, 1, 2, 128), device="cuda")
    kv, want = (fd.kv4_cache(2, 2, 64, 128) for _ in range(2))
    lens = torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    fd.append_rope_kv4(x, x, want, seq_lens=lens, workspace=fd.Workspace())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fd.append_rope_kv4(x, x, kv, seq_lens=lens)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kv, want) and bool((kv != 0).any()) and fd.workspace_status() == 0
