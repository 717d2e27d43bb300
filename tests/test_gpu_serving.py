"""Decoding rounds with the target's cache and the emitted tokens' log probabilities:
reserve, append, attend, verify, commit and token_logprobs as a serving loop calls them,
with forks, compaction and exchanged requests between the rounds.

The target is a lookup: a token has fixed queries, keys and values per layer, so the
attention of a request follows in binary64 from the tokens it has kept.  The tolerance
of an attended row is that of the attention's own tests: with u = 2^-24, A = sum w |v|,
B = max scale sum |q k|, n keys of D elements, 2 u ((D + 2) B + 2 B log2 e + 4) A +
(n + 16) u A for scores, exponentials and sums, and for bf16 2^-8 A for the rounded
weights and 2^-8 of the result."""
import math

import numpy as np
import pytest

import test_gpu_logprobs as LP

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24
R, GAMMA, V, LAYERS, HEADS, KV, DIM, PAGE = 5, 4, 1000, 2, 4, 2, 64, 16


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from draft_sampling_verification_w1_amd import dspark
    dspark.lib()
    return dspark


def ints(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Target:
    """Lookup tables of a target, and the tokens that each request's cache should hold."""

    def __init__(self, dev, dtype, max_pages, pages, seed=5):
        import torch
        from draft_sampling_verification_w1_amd.cache import PagedCache
        from draft_sampling_verification_w1_amd.decode import DecodeLoop
        self.dt = torch.float32 if dtype == "f32" else torch.bfloat16
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.q = rand(LAYERS, V, HEADS, DIM).to(self.dt).cuda()
        self.k = rand(LAYERS, V, KV, DIM).to(self.dt).cuda()
        self.v = rand(LAYERS, V, KV, DIM).to(self.dt).cuda()
        self.wo = (rand(HEADS * DIM, V) * 0.05).cuda()
        self.W1 = (rand(V, 256) * 0.1).to(self.dt).cuda()
        self.W2 = (rand(256, V) * 0.1).to(self.dt).cuda()
        self.cache = PagedCache(R, max_pages, pages, PAGE, LAYERS, KV, DIM, self.dt)
        self.cache.K.fill_(math.nan)
        self.cache.V.fill_(math.nan)
        self.gen = g
        self.anchors = torch.randint(0, V, (R,), generator=g, dtype=torch.int32).cuda()
        make = lambda **kw: DecodeLoop(self.W1, dev.pack_w2(self.W2, V), self.anchors, 77, GAMMA, **kw)  # noqa: E731
        self.loop, self.plain = make(cache=self.cache, logprobs=3), make()
        self.kept = [[] for _ in range(R)]
        self.calls = 0

    def forward(self, ids, offsets):
        """Appends and attends the flattened tokens; checks every attended row."""
        import torch
        total = 0
        ids = ids.long()
        for layer in range(LAYERS):
            q, k, v = self.q[layer][ids], self.k[layer][ids], self.v[layer][ids]
            self.cache.append(layer, k, v, offsets)
            out = self.cache.attend(layer, q, offsets)
            self.check(layer, out, ids.tolist(), offsets.tolist())
            total = total + out.float().reshape(len(ids), -1) @ self.wo
        return total

    def check(self, layer, out, ids, offsets):
        import torch
        got = out.double().cpu()
        Q, K, W = (t[layer].double().cpu() for t in (self.q, self.k, self.v))
        bf = self.dt == torch.bfloat16
        scale = DIM ** -0.5
        for s in range(R):
            chunk = ids[offsets[s]:offsets[s + 1]]
            n, old = len(chunk), len(self.kept[s])
            if n == 0:
                continue
            seen = torch.tensor(self.kept[s] + chunk)
            mask = torch.arange(old + n)[None] > old + torch.arange(n)[:, None]
            for h in range(HEADS):
                g = h // (HEADS // KV)
                q, k, v = Q[chunk, h], K[seen, g], W[seen, g]
                w = torch.softmax((scale * q @ k.T).masked_fill(mask, -math.inf), 1)
                B = (scale * q.abs() @ k.abs().T).amax(1, keepdim=True)
                want, A = w @ v, w @ v.abs()
                rel = 2 * U24 * ((DIM + 2) * B + 2 * B * 1.45 + 4) + (old + n + 16) * U24
                tol = A * (rel + (2.0 ** -8 if bf else 0)) + want.abs() * (2.0 ** -8 if bf else U24)
                off = (got[offsets[s]:offsets[s + 1], h] - want).abs()
                assert (off <= tol).all(), (layer, s, h, float((off / tol).max()))

    def prompt(self, prompts):
        """Prefills the given tokens (a list per request) behind what the slots hold."""
        lens = [len(p) for p in prompts]
        self.cache_status(self.cache.reserve(ints(lens)))
        flat = [t for p in prompts for t in p]
        if flat:
            self.forward(ints(flat), ints([0] + np.cumsum(lens).tolist()))
        self.cache.commit(ints(lens))
        for s, p in enumerate(prompts):
            self.kept[s] += p

    def cache_status(self, r):
        assert r["status"].tolist() == [0] * R

    def logits(self, t, tok):
        import torch
        self.calls += 1
        prev = torch.cat([self.loop.anchors[:, None], tok], 1)
        a = self.forward(prev.reshape(-1), self.loop.offsets).reshape(R, GAMMA + 1, V)
        d = self.W1[prev.long()].float() @ self.W2.float()
        return (torch.cat([self.U, self.U[:, :1]], 1).float() + d + 0.3 * a).to(self.dt)

    def round(self):
        """A round of the loop against one without a cache, and its consequences."""
        import torch
        self.U = (torch.randn((R, GAMMA, V), generator=self.gen) * 2).to(self.dt).cuda()
        got = {}

        def target(t, tok):
            got["T"] = self.logits(t, tok)
            return got["T"]

        first = self.loop.anchors.tolist()
        r = self.loop.round(self.U, target)
        self.plain.anchors.copy_(ints(first))
        p = self.plain.round(self.U, lambda t, tok: got["T"])
        for name in ("tokens", "n_accept", "out_token", "cstar", "accept_mask"):
            assert torch.equal(r[name], p[name]), name
        tok, n, last = r["tokens"].tolist(), r["n_accept"].tolist(), r["out_token"].tolist()
        want = [tok[s][:n[s]] + [last[s]] + [-1] * (GAMMA - n[s]) for s in range(R)]
        assert r["emitted"].tolist() == want
        T = got["T"].double().cpu().numpy().reshape(-1, V)
        LP.check({x: r[x] for x in ("logprob", "entropy", "top_ids", "top_logprobs")},
                 LP.reference(T, np.array(want).reshape(-1), 3))
        for s in range(R):
            self.kept[s] += [first[s]] + tok[s][:n[s]]
        assert self.cache.lens.tolist() == [len(x) for x in self.kept]
        return n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rounds(dev, dtype):
    t = Target(dev, dtype, max_pages=12, pages=48)
    rng = np.random.default_rng(9)
    some = lambda n: rng.integers(0, V, n).tolist()  # noqa: E731
    t.prompt([some(n) for n in (37, 0, 1, 16, 15)])
    accepted = t.round() + t.round()
    # request 3 becomes a second continuation of request 0
    t.cache.free(ints([3]))
    assert t.cache.fork(ints([0]), ints([3])).tolist() == [0]
    t.loop.anchors[3] = t.loop.anchors[0]
    t.kept[3] = list(t.kept[0])
    accepted += t.round() + t.round()
    # request 1 ends, the pages move together, a new request takes its place
    t.cache.free(ints([1]))
    t.kept[1] = []
    t.cache.compact()
    t.prompt([[], some(50), [], [], []])
    for _ in range(3):
        accepted += t.round()
    # both continuations back to where request 0's cache ended long ago
    back = [20 - len(t.kept[0]), -2 ** 31, -2 ** 31, 20 - len(t.kept[3]), -2 ** 31]
    t.cache.commit(ints(back))
    t.kept[0], t.kept[3] = t.kept[0][:20], t.kept[3][:20]
    accepted += t.round()
    assert 0 < np.mean(accepted) < GAMMA  # rounds of every kind


def test_round_without_pages(dev):
    """A request without pages ends the round before the target runs; the round is
    repeated once a slot was freed.  (12 pages: prompts take 2 + 3 + 2 + 2 + 2.)"""
    t = Target(dev, "bf16", max_pages=4, pages=12)
    rng = np.random.default_rng(3)
    t.prompt([rng.integers(0, V, n).tolist() for n in (30, 40, 30, 30, 20)])
    before = t.cache.lens.tolist()
    with pytest.raises(RuntimeError, match=r"requests \[2, 3\]"):
        t.U = t.W1.new_zeros((R, GAMMA, V))
        t.loop.round(t.U, t.logits)
    assert t.calls == 0 and t.loop.t == 0 and t.cache.lens.tolist() == before
    t.cache.free(ints([1]))
    t.kept[1] = []
    t.round()
    assert t.calls == 1


def test_loop_refusals(dev):
    import torch
    from draft_sampling_verification_w1_amd.cache import PagedCache
    from draft_sampling_verification_w1_amd.decode import DecodeLoop
    t = Target(dev, "bf16", max_pages=4, pages=12)
    small = PagedCache(R - 1, 2, 8, PAGE, 1, KV, DIM)
    args = (t.W1, dev.pack_w2(t.W2, V), t.anchors, 1, GAMMA)
    with pytest.raises(ValueError):
        DecodeLoop(*args, cache=small)
    for n in (-1, 65):
        with pytest.raises(ValueError):
            DecodeLoop(*args, logprobs=n)
    U = torch.zeros((R, GAMMA, V), dtype=t.dt, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        U.zero_()
        with pytest.raises(RuntimeError, match="captured"):
            t.loop.round(U, t.logits)


def test_binding_refusals(dev):
    """Shapes, types, strides, devices and workspaces that the Python calls turn down."""
    import torch
    from draft_sampling_verification_w1_amd.cache import PagedCache
    c = PagedCache(3, 4, 9, 16, 1, 2, 64)
    q = torch.zeros((6, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((6, 2, 64), dtype=torch.bfloat16, device="cuda")
    off = ints([0, 2, 4, 6])
    z, ids = torch.zeros((4, 30000), device="cuda"), ints([0, 1, 2, 3])
    ws = c.attend_workspace(6, 4)
    bad = [
        lambda: c.attend(0, q.float(), off), lambda: c.attend(0, q[:, :, :32], off),
        lambda: c.attend(0, q[::2], off), lambda: c.attend(0, q, off[:3]),
        lambda: c.attend(0, q, off.long()), lambda: c.attend(0, q, off.cpu()),
        lambda: c.attend(0, q, off, out=q[:3]), lambda: c.attend(0, q, off, ws=ws.cpu()),
        lambda: c.append(0, k, q, off), lambda: c.append(0, k[:5], k, off),
        lambda: c.append(0, k, k.transpose(0, 1).contiguous().transpose(0, 1), off),
        lambda: c.reserve(ints([1, 1])), lambda: c.commit(off), lambda: c.fork(ints([0]), ints([1, 2])),
        lambda: c.free(torch.zeros(1, device="cuda")), lambda: c.copy_pages(ints([0]), ints([1]), count=off),
        lambda: dev.token_logprobs(z, ids[:3]), lambda: dev.token_logprobs(z.half(), ids),
        lambda: dev.token_logprobs(z.t(), ids), lambda: dev.token_logprobs(z[:, ::2], ids),
        lambda: dev.token_logprobs(z[:1].expand(4, -1), ids), lambda: dev.token_logprobs(z[0], ids),
        lambda: dev.token_logprobs(z, ids.cpu()),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    refused = [
        lambda: c.attend(1, q, off), lambda: c.attend(0, q, off, scale=0.0), lambda: c.attend(0, q, off, out=q),
        lambda: c.attend(0, q, off, max_chunk=0), lambda: c.attend(0, q, off, ws=ws[:-256]),
        lambda: c.attend(0, q[:, :3].contiguous(), off), lambda: c.append(-1, k, k, off),
        lambda: dev.token_logprobs(z, ids, 65), lambda: dev.token_logprobs(z, ids, ws=ws[:256]),
    ]
    for call in refused:
        with pytest.raises(RuntimeError):
            call()
