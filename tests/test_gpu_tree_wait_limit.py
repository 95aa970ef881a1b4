"""The bounded waits of the tree attention over bf16 caches: a wait that runs out is reported, not hung on.

``fd_debug_stall`` makes every CTA skip one copy of K (nothing is issued for it, so nothing is left in flight) and shortens
the limit to 1 ms.  A piece's first use of K's slots brings q, so its first copy of K is use 1.  The call has to report
FD_ERR_TIMEOUT, and the next one on the same workspace to be right.
"""

import pytest
import torch

import split_kv_decode_fd_gb300 as fd
from split_kv_decode_fd_gb300 import fdecode as fdb

from test_gpu_decode_tree import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("Hq,Hkv,n", [(4, 4, 7), (8, 2, 14), (8, 2, 40)], ids=["32_rows", "64_rows", "blocks_of_128_rows"])
@pytest.mark.parametrize("use", [1, 2])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_clean(D, page, Hq, Hkv, n, use):
    # 40 pairs of 16 tiles: four or more of them a CTA
    c = Case(20, Hq, Hkv, D, n, [2000 + 3 * b for b in range(20)], page=page, cap=2064, seed=use)
    ws = fd.Workspace()
    call = lambda: fd.decode_tree(c.q, c.k, c.v, c.parents, seq_lens=torch.tensor(c.lens, dtype=torch.int32, device="cuda"),
                                  max_seq_len=2064, block_table=c.table, workspace=ws)
    out, lse = call()
    assert fd.workspace_status(ws) == fdb.FD_OK
    lib = fd.load_library()
    try:
        lib.fd_debug_stall(use, 1_000_000)
        call()
        assert fd.workspace_status(ws) == fdb.FD_ERR_TIMEOUT
    finally:
        lib.fd_debug_stall(-1, 0)
    assert fd.workspace_status(ws) == fdb.FD_OK  # reading the word cleared it
    again, lse_again = call()
    assert fd.workspace_status(ws) == fdb.FD_OK
    assert torch.equal(out, again) and torch.equal(lse, lse_again)
