"""GPU tests of a step with a tree of drafted tokens as it is used: append_rope writes the drafts, decode_tree attends them,
verify_tree says which stay, keep_rows moves the rows of those together, and the next step goes on from there.

Attention is held to the bound of the tests of decode_tree; what is decided and moved has to be equal, and the cache that is left
equal, bit by bit, to one that has got the kept tokens alone.
"""

import math

import numpy as np
import pytest
import torch

import oracle
import split_kv_decode_fd_gb300 as fd

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
V, MAX_POS = 700, 512


class Model:
    """Tensors of a few steps: B sequences, n rows of drafts, a cache, and a head that turns outputs into probabilities."""

    def __init__(self, B, Hq, Hkv, D, n, cache, page, cap=384, seed=0):
        self.B, self.Hq, self.Hkv, self.D, self.n, self.page, self.cap = B, Hq, Hkv, D, n, page, cap
        self.r = np.random.default_rng(seed)
        shape = (B * (cap // page), Hkv, page, D) if page else (B, Hkv, cap, D)
        self.k, self.v = (torch.zeros(shape, dtype=TYPES[cache], device="cuda") for _ in range(2))
        self.table = None
        if page:
            self.table = torch.from_numpy(self.r.permutation(shape[0]).reshape(B, -1).astype(np.int32)).cuda()
        angles = np.outer(np.arange(MAX_POS), 10000.0 ** (-np.arange(D // 2) / (D // 2)))
        self.cos, self.sin = (torch.from_numpy(f(angles).astype(np.float32)).cuda() for f in (np.cos, np.sin))
        self.head = torch.from_numpy((self.r.standard_normal((Hq * D, V)) / 6).astype(np.float32)).cuda()
        self.ws = fd.Workspace()

    def normal(self, *shape):
        return torch.from_numpy(self.r.standard_normal(shape).astype(np.float32)).cuda()

    def drafts(self, tokens):
        """A random tree for every sequence: what a step takes, and the places of its depths."""
        B, n, D = self.B, self.n, self.D
        d = {"k": self.normal(B, n, self.Hkv, D), "v": self.normal(B, n, self.Hkv, D), "q": self.normal(B, n, self.Hq, D)}
        parents, depth = np.full((B, n), -1, np.int32), np.zeros((B, n), np.int32)
        for b, m in enumerate(tokens):
            for j in range(1, m):
                parents[b, n - m + j] = self.r.integers(max(0, j - 3), j)
                depth[b, n - m + j] = depth[b, n - m + parents[b, n - m + j]] + 1
        d["parents"], d["depth"] = torch.from_numpy(parents).cuda(), torch.from_numpy(depth).cuda()
        d["new"] = torch.tensor(tokens, dtype=torch.int32, device="cuda")
        d["words"] = torch.from_numpy(self.r.integers(0, V, (B, n)).astype(np.int32)).cuda()
        d["uniforms"] = torch.from_numpy(self.r.random((B, n), dtype=np.float32) * np.float32(0.02)).cuda()
        d["uniforms"][:, 0::3] *= 49.0
        d["draft"] = torch.softmax(2 * self.normal(B, n, V), -1)
        return d

    def step(self, d, lens):
        """One step on the cache; ``lens`` [B] int32 on the device are the lengths before it."""
        common = dict(block_table=self.table, workspace=self.ws)
        q = torch.zeros((self.B, self.Hq, self.n, self.D), device="cuda")
        fd.append_rope(d["k"], d["v"], self.k, self.v, self.cos, self.sin, q=d["q"], q_out=q, positions=lens[:, None] + d["depth"],
                       new_lens=d["new"], seq_lens=lens, max_seq_len=self.cap - self.n, **common)
        out, lse = fd.decode_tree(q, self.k, self.v, d["parents"], new_lens=d["new"], seq_lens=lens + d["new"],
                                  max_seq_len=self.cap, **common)
        target = torch.softmax(out.transpose(1, 2).reshape(self.B, self.n, -1) @ self.head, -1)
        path, count, word = fd.verify_tree(d["words"], d["parents"], target, d["uniforms"], draft=d["draft"], new_lens=d["new"],
                                           workspace=self.ws)
        before = self.rows() if not torch.cuda.is_current_stream_capturing() else None
        fd.keep_rows(self.k, self.v, path, counts=count, starts=lens, **common)
        return {"q": q, "out": out, "lse": lse, "target": target, "path": path, "count": count, "word": word, "before": before}

    def rows(self):
        """The cache as [B, Hkv, cap, D], K and V."""
        if not self.page:
            return self.k.clone(), self.v.clone()
        return tuple(x[self.table.long()].transpose(1, 2).reshape(self.B, self.Hkv, self.cap, self.D) for x in (self.k, self.v))


def tokens_of(r, B, n, t):
    m = r.integers(1, n + 1, B)
    m[t % B] = n
    if B > 2:
        m[(t + 1) % B] = 0  # a sequence that sits out
    return [int(x) for x in m]


@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("B,Hq,Hkv,D,n", [(1, 4, 4, 64, 5), (4, 8, 2, 128, 9), (3, 12, 2, 64, 20)])
def test_steps(cache, page, B, Hq, Hkv, D, n):
    m = Model(B, Hq, Hkv, D, n, cache, page, seed=B)
    clean = Model(B, Hq, Hkv, D, n, cache, page, seed=B)  # gets the kept tokens alone
    lens = np.zeros(B, dtype=np.int64)
    for t in range(4):
        tokens = tokens_of(m.r, B, n, t)
        d = m.drafts(tokens)
        before = torch.from_numpy(lens.astype(np.int32)).cuda()
        got = m.step(d, before)
        assert fd.workspace_status(m.ws) == 0
        k, v = (x.double().cpu().numpy() for x in got["before"])
        q = got["q"].cpu().numpy()
        parents = d["parents"].cpu().numpy()
        ref, ref_lse = oracle.tree.attend(q, k, v, parents, lens + tokens, tokens, 1 / math.sqrt(D))
        live = ~np.isnan(ref_lse)
        # scores are off by (2^-21 + D 2^-24) of their largest sum of sizes, weights by that and 2^-20: out by twice
        # that of max |v|, and by 2^-23 for each of 24 products a tile and each tile
        A = np.abs(q).sum(-1).max() * np.abs(k).max() / math.sqrt(D)
        slack = ((2.0 ** -21 + D * 2.0 ** -24) * A + 2.0 ** -20) * 2 + (24 + m.cap / 128) * 2.0 ** -23
        assert np.abs(got["out"].cpu().numpy() - ref)[live].max() <= slack * np.abs(v).max()
        path, count, word = (got[x].cpu().numpy() for x in ("path", "count", "word"))
        target, draft = got["target"].double().cpu().numpy(), d["draft"].double().cpu().numpy()
        for b, mb in enumerate(tokens):
            p, w = oracle.tree.verify(d["words"][b, n - mb:].tolist(), parents[b, n - mb:], target[b, n - mb:],
                                      d["uniforms"][b, n - mb:].tolist(), draft[b, n - mb:])
            assert path[b].tolist() == p + [-1] * (n - len(p)) and count[b] == len(p) and word[b] == w
        # the rows that stay, with those of the tokens' own appends on the other cache
        kept = torch.zeros((B, n), dtype=torch.int64)
        for b, mb in enumerate(tokens):
            for j in range(count[b]):
                kept[b, n - int(count[b]) + j] = n - mb + int(path[b, j])
        at = kept.cuda()[:, :, None, None]
        depth = torch.gather(d["depth"], 1, kept.cuda())
        fd.append_rope(torch.gather(d["k"], 1, at.expand(-1, -1, Hkv, D)), torch.gather(d["v"], 1, at.expand(-1, -1, Hkv, D)),
                       clean.k, clean.v, m.cos, m.sin, positions=before[:, None] + depth, new_lens=got["count"], seq_lens=before,
                       max_seq_len=m.cap - n, block_table=clean.table)
        lens += count
        for x, y in zip(m.rows(), clean.rows()):
            for b in range(B):
                assert torch.equal(x[b, :, :lens[b]], y[b, :, :lens[b]])
    assert lens.max() > 4 and fd.workspace_status(m.ws) == 0


@pytest.mark.parametrize("cache,page", [("bf16", 16), ("f32", 0)])
def test_a_captured_step(cache, page):
    """The step as a graph whose lengths live on the device: replays are the eager calls, bit by bit."""
    B, Hq, Hkv, D, n = 3, 8, 2, 128, 6
    eager, graph = (Model(B, Hq, Hkv, D, n, cache, page, seed=7) for _ in range(2))
    r = np.random.default_rng(3)
    steps = [eager.drafts(tokens_of(r, B, n, t)) for t in range(4)]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    want = []
    for d in steps:
        got = eager.step(d, lens)
        want.append({x: got[x].clone() for x in ("out", "lse", "path", "count", "word")})
        lens = lens + got["count"]
    held = {x: y.clone() for x, y in steps[0].items()}
    at = torch.zeros(B, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph.step(held, at)  # warms up; what it writes lies past the lengths and is written again
    torch.cuda.synchronize()
    graph.k.zero_()
    graph.v.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        got = graph.step(held, at)
        at.add_(got["count"])
    for d, w in zip(steps, want):
        for x in held:
            held[x].copy_(d[x])
        g.replay()
        torch.cuda.synchronize()
        for x in w:
            assert torch.equal(got[x], w[x]), x
    assert torch.equal(at, lens)
    for x, y in zip(graph.rows(), eager.rows()):
        for b in range(B):
            assert torch.equal(x[b, :, :lens[b]], y[b, :, :lens[b]])
    assert fd.workspace_status(graph.ws) == 0 and fd.workspace_status(eager.ws) == 0


def test_steps_on_two_streams_at_once():
    """Two models on streams of their own, their launches mixed: each gets what it gets alone."""
    models = [Model(4, 8, 2, 128, 12, "bf16", 16, seed=s) for s in (1, 2)]
    alone = [Model(4, 8, 2, 128, 12, "bf16", 16, seed=s) for s in (1, 2)]
    drafts = [[m.drafts(tokens_of(m.r, 4, 12, t)) for t in range(3)] for m in models]
    want = []
    for m, ds in zip(alone, drafts):
        lens = torch.zeros(4, dtype=torch.int32, device="cuda")
        for d in ds:
            lens = lens + m.step(d, lens)["count"]
        want.append((lens, m.rows()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in models]
    lens = [torch.zeros(4, dtype=torch.int32, device="cuda") for _ in models]
    torch.cuda.synchronize()
    for t in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                lens[i] = lens[i] + models[i].step(drafts[i][t], lens[i])["count"]
    torch.cuda.synchronize()
    for m, got, (n, rows) in zip(models, lens, want):
        assert torch.equal(got, n) and fd.workspace_status(m.ws) == 0
        for x, y in zip(m.rows(), rows):
            for b in range(4):
                assert torch.equal(x[b, :, :n[b]], y[b, :, :n[b]])
