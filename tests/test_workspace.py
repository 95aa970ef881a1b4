"""Workspaces on the host: what happens to their buffers (here of CPU memory) as they grow."""

import weakref

import torch

import split_kv_decode_fd_gb300 as fd

CPU = torch.device("cpu")


def test_outgrown_buffers_stay_as_long_as_the_workspace():
    """A captured graph holds the address of the buffer that it was captured with."""
    ws = fd.Workspace()
    seen = []
    for nbytes in (256, 1000, 1 << 16, (1 << 16) + 1, 1 << 20):
        buf = ws.get(nbytes, CPU)
        assert buf.numel() >= nbytes and int(buf.sum()) == 0
        seen.append((weakref.ref(buf), buf.data_ptr()))
        del buf
    assert all(ref() is not None and ref().data_ptr() == at for ref, at in seen)
    del ws
    assert all(ref() is None for ref, _ in seen)


def test_growing_in_small_steps_takes_no_more_than_twice_the_last_buffer():
    ws = fd.Workspace()
    held = {}
    for nbytes in range(1000, 100_000, 1000):
        buf = ws.get(nbytes, CPU)
        held[buf.data_ptr()] = buf.numel()
    assert sum(held.values()) <= 2 * ws.buf.numel() and ws.buf.numel() < 4 * 100_000


def test_a_buffer_that_is_large_enough_is_used_again():
    ws = fd.Workspace()
    a = ws.get(1000, CPU)
    assert ws.get(900, CPU) is a
    meta = ws.get(500, torch.device("meta"))
    assert ws.get(800, CPU) is a and ws.get(400, torch.device("meta")) is meta


def test_a_device_without_an_index_is_the_same_device():
    ws = fd.Workspace()
    a = ws.get(1000, torch.device("cpu"))
    for _ in range(3):
        assert ws.get(1000, torch.device("cpu", 0)).numel() >= 1000
    assert len({ws.get(1000, d).data_ptr() for d in (CPU, CPU)}) == 1 and a.numel() == 1000
    assert len(ws._outgrown) <= 1
