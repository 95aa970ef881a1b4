"""GPU tests of the verification of drafted trees against the float64 oracle: every output is a whole number and equal."""

import numpy as np
import pytest
import torch

import oracle
import split_kv_decode_fd_gb300 as fd

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


class Case:
    def __init__(self, B, n, V, *, dtype="f32", draft=True, new_lens=None, seed=0, shape="random", peak=4.0, agree=0.9):
        r = np.random.default_rng(seed)
        self.B, self.n, self.V, self.new_lens = B, n, V, new_lens
        logits = peak * r.standard_normal((B, n, V))
        other = agree * logits + peak * (1 - agree) * r.standard_normal((B, n, V))
        soft = lambda x: np.exp(x - x.max(-1, keepdims=True)) / np.exp(x - x.max(-1, keepdims=True)).sum(-1, keepdims=True)  # noqa: E731
        self.target = torch.from_numpy(soft(logits).astype(np.float32)).to(TYPES[dtype]).cuda()
        q = soft(other)
        self.draft = torch.from_numpy(q.astype(np.float32)).to(TYPES[dtype]).cuda() if draft else None
        self.parents = np.full((B, n), 77, dtype=np.int32)
        self.tokens = np.full((B, n), -5, dtype=np.int32)
        for b in range(B):
            m = n if new_lens is None else new_lens[b]
            pad = n - m
            for j in range(m):
                p = -1 if j == 0 else {"chain": j - 1, "wide": 0}.get(shape, int(r.integers(max(0, j - 4), j)))
                self.parents[b, pad + j] = p
                if j:
                    words = q[b, pad + p]
                    self.tokens[b, pad + j] = r.choice(V, p=words / words.sum()) if draft else np.argsort(-words)[
                        min(V - 1, int((self.parents[b, pad:pad + j] == p).sum()))]
        self.uniforms = torch.from_numpy(r.random((B, n)).astype(np.float32)).cuda()

    def run(self, **kw):
        if self.new_lens is not None:
            kw.setdefault("new_lens", torch.tensor(self.new_lens, dtype=torch.int32, device="cuda"))
        return fd.verify_tree(torch.from_numpy(self.tokens).cuda(), torch.from_numpy(self.parents).cuda(),
                              kw.pop("target", self.target), self.uniforms, draft=kw.pop("draft", self.draft), **kw)

    def want(self):
        paths, counts, words = np.full((self.B, self.n), -1), np.zeros(self.B, int), np.zeros(self.B, int)
        t = self.target.float().cpu().numpy()
        d = None if self.draft is None else self.draft.float().cpu().numpy()
        u = self.uniforms.cpu().numpy()
        for b in range(self.B):
            at = slice(self.n - (self.n if self.new_lens is None else self.new_lens[b]), self.n)
            path, words[b] = oracle.tree.verify(self.tokens[b, at], self.parents[b, at], t[b, at], u[b, at],
                                                None if d is None else d[b, at])
            paths[b, :len(path)], counts[b] = path, len(path)
        return paths, counts, words

    def check(self, got):
        for g, w in zip(got, self.want()):
            assert g.dtype == torch.int32 and np.array_equal(g.cpu().numpy(), w), (g.cpu().numpy(), w)


@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 4096, 4097, 20011, 50000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("shape", ["chain", "random", "wide"])
def test_against_the_oracle(V, dtype, draft, shape):
    c = Case(5, 7, V, dtype=dtype, draft=draft, shape=shape, seed=V)
    c.check(c.run())
    assert fd.workspace_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_large_vocabulary(dtype):
    c = Case(2, 9, 300007, dtype=dtype, draft=dtype == "f32", shape="random", seed=1)
    c.check(c.run())
    assert fd.workspace_status() == 0


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("agree", [0.0, 0.95, 1.0])
def test_trees_of_any_size(n, draft, agree):
    r = np.random.default_rng(n)
    c = Case(9, n, 601, draft=draft, agree=agree, new_lens=r.integers(0, n + 1, 9).tolist(), seed=n)
    c.check(c.run())
    c = Case(2, n, 601, draft=draft, agree=agree, shape="wide", seed=n)  # many refusals at one token
    c.check(c.run())


def test_many_sequences():
    c = Case(300, 5, 5003, seed=1)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("draft", [True, False])
def test_strided_rows_and_odd_addresses(dtype, draft):
    """Rows of a padded vocabulary, rows that start anywhere, and one row for all sequences."""
    c = Case(4, 6, 9001, dtype=dtype, draft=draft, seed=2)
    want = c.want()
    for pad, off in ((7, 0), (8, 0), (3, 1), (0, 5)):
        kw = {}
        for name in ("target", "draft"):
            x = getattr(c, name)
            if x is not None:
                flat = torch.full((4 * 6 * (9001 + pad) + off,), float("nan"), dtype=x.dtype, device="cuda")
                view = flat[off:].view(4, 6, 9001 + pad)[..., :9001]
                view.copy_(x)
                kw[name] = view
        for g, w in zip(c.run(**kw), want):
            assert np.array_equal(g.cpu().numpy(), w)
    one = c.target[:1, :1]
    c.target = one.expand(4, 6, 9001)
    c.check(c.run())


def test_uniforms_at_their_ends():
    for u in (0.0, 1.0 - 2.0 ** -24, 1.0):
        for draft in (True, False):
            c = Case(6, 5, 700, draft=draft, seed=3)
            c.uniforms.fill_(u)
            c.check(c.run())


def test_zeros_and_what_is_no_probability():
    """Words of probability 0 are never drawn; NaN and negative entries count as 0; a row without any gives -1."""
    c = Case(4, 4, 5000, draft=False, seed=4)
    c.target[:, :, 100:4900] = 0
    c.check(c.run())
    before = c.run()
    c.target[:, :, 200:300] = float("nan")
    c.target[:, :, 300:400] = -1.0
    for a, b in zip(c.run(), before):
        assert torch.equal(a, b)
    c.target.zero_()
    path, count, word = c.run()
    assert (count == 1).all() and (word == -1).all()


@pytest.mark.parametrize("V", [64, 30000])
def test_the_draft_is_the_target(V):
    """p = q: every child stays for u < 1; refused by u = 1, it leaves nothing, and the target itself is drawn from."""
    c = Case(3, 6, V, shape="wide", seed=5)
    c.draft = c.target.clone()
    c.check(c.run())
    c.uniforms[:, 1:] = 1.0
    c.check(c.run())
    assert (c.run()[1] == 1).all()


def test_words_and_parents_out_of_range_are_left_out():
    c = Case(3, 5, 1000, seed=6, shape="chain")
    want = c.run()
    assert fd.workspace_status() == 0
    for name, bad in (("tokens", 1000), ("tokens", -1), ("tokens", 1 << 30), ("parents", 2), ("parents", -2), ("parents", 1 << 30)):
        old = getattr(c, name).copy()
        getattr(c, name)[0, 2] = bad
        path, count, word = c.run()
        assert fd.workspace_status() == fd.fdecode.FD_ERR_BAD_INDEX
        assert count[0] <= 2 and torch.equal(path[1:], want[0][1:]) and torch.equal(word[1:], want[2][1:])
        setattr(c, name, old)
    assert fd.workspace_status() == 0


@pytest.mark.parametrize("V", [500, 40000])
def test_on_another_stream_and_captured(V):
    c = Case(7, 9, V, seed=7)
    want = c.run()
    tokens, parents = torch.from_numpy(c.tokens).cuda(), torch.from_numpy(c.parents).cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = fd.verify_tree(tokens, parents, c.target, c.uniforms, draft=c.draft, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = fd.Workspace()
    out = dict(path=torch.empty_like(want[0]), count=torch.empty_like(want[1]), next_token=torch.empty_like(want[2]))
    fd.verify_tree(tokens, parents, c.target, c.uniforms, draft=c.draft, workspace=ws, **out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fd.verify_tree(tokens, parents, c.target, c.uniforms, draft=c.draft, workspace=ws, **out)
    for _ in range(3):
        for t in out.values():
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out.values(), want))


def test_the_tokens_have_the_target_distribution():
    """65536 sequences with random numbers of their own: the first new token has the target's probabilities.  Each count is
    binomial, so it is within 6 standard deviations of its mean but with probability 2e-9."""
    B, n, V = 65536, 3, 8
    r = np.random.default_rng(8)
    p, q = r.dirichlet(np.ones(V)), r.dirichlet(np.ones(V))
    tokens = r.choice(V, (B, n), p=q).astype(np.int32)
    target = torch.from_numpy(p.astype(np.float32)).cuda().expand(B, n, V)
    draft = torch.from_numpy(q.astype(np.float32)).cuda().expand(B, n, V)
    parents = torch.tensor([-1, 0, 0], dtype=torch.int32, device="cuda")
    u = torch.from_numpy(r.random((B, n)).astype(np.float32)).cuda()
    path, count, word = fd.verify_tree(torch.from_numpy(tokens).cuda(), parents, target, u, draft=draft)
    first = np.where(count.cpu().numpy() == 1, word.cpu().numpy(), tokens[np.arange(B), path[:, 1].clamp(min=0).cpu().numpy()])
    got = np.bincount(first, minlength=V)
    assert np.all(np.abs(got - B * p) < 6 * np.sqrt(B * p * (1 - p))), (got / B, p)


def test_refusals():
    c = Case(2, 4, 50, seed=9)
    tokens, parents = torch.from_numpy(c.tokens).cuda(), torch.from_numpy(c.parents).cuda()
    call = lambda **kw: fd.verify_tree(**{**dict(tokens=tokens, parents=parents, target=c.target, uniforms=c.uniforms, draft=c.draft), **kw})  # noqa: E731
    call()
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    for kw in (dict(target=c.target.cpu()), dict(target=c.target[0]), dict(target=c.target.half()), dict(draft=c.draft.bfloat16()),
               dict(draft=c.draft[:, :, :49]), dict(draft=c.draft.transpose(1, 2).contiguous().transpose(1, 2)),
               dict(tokens=tokens.long()), dict(tokens=tokens[:, :3]), dict(uniforms=c.uniforms.double()),
               dict(parents=parents[:1]), dict(new_lens=lens[:1]), dict(new_lens=lens.long()), dict(path=lens), dict(count=lens.float()),
               dict(next_token=torch.empty(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            call(**kw)
    z = torch.zeros(1, 65, dtype=torch.int32, device="cuda")
    with pytest.raises(fd.FdError):
        fd.verify_tree(z, z, torch.zeros(1, 65, 8, device="cuda"), z.float())
