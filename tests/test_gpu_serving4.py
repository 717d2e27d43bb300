"""Decoding rounds of a target whose keys and queries are rotated by their positions, over a
cache in 4 bits and over one of whole elements: reserve, append with a rotation, attend, read, verify and
commit as a serving loop calls them, with forks, compaction and rollback between the rounds.

The target of test_gpu_serving.py; what its cache holds is read back after every append: tokens kept from
earlier rounds must be bit for bit what they were, and the attention follows in binary64 from them.
The tolerance is that of test_gpu_attend4.py."""
import math

import numpy as np
import pytest

import mx_model as M
import test_gpu_serving as TS
from test_gpu_serving import DIM, GAMMA, HEADS, KV, LAYERS, PAGE, R, V, dev, ints  # noqa: F401

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24


class Target(TS.Target):
    def __init__(self, dev, dtype, max_pages, pages, four):
        from draft_sampling_verification_w1_amd import cache
        from draft_sampling_verification_w1_amd.decode import DecodeLoop
        super().__init__(dev, dtype, max_pages, pages)
        self.four = four
        if four:
            self.cache = cache.PagedCache(R, max_pages, pages, PAGE, LAYERS, KV, DIM, cache.FOUR_BITS)
            self.cache.K.fill_(255)
            self.cache.V.fill_(255)
            self.loop = DecodeLoop(self.W1, dev.pack_w2(self.W2, V), self.anchors, 77, GAMMA, cache=self.cache,
                                   logprobs=3)
        self.rotation = cache.Rotation(cache.rope_frequencies(DIM), interleaved=four)
        self.held = [[(np.zeros((0, KV, DIM)),) * 2 for _ in range(R)] for _ in range(LAYERS)]

    def forward(self, ids, offsets):
        total = 0
        ids, off = ids.long(), offsets.tolist()
        for layer in range(LAYERS):
            q, k, v = self.q[layer][ids], self.k[layer][ids], self.v[layer][ids]
            turned = self.cache.append(layer, k, v, offsets, rotation=self.rotation, q=q)
            out = self.cache.attend(layer, turned, offsets)
            self.check_layer(layer, turned, v, out, off)
            total = total + out.float().reshape(len(ids), -1) @ self.wo
        return total

    def check_layer(self, layer, turned, values, out, off):
        """Everything the slots hold, against what they held before, and the attention over it."""
        import torch
        old = [len(x) for x in self.kept]
        n = [b - a for a, b in zip(off, off[1:])]
        every = [0] + np.cumsum([a + b for a, b in zip(old, n)]).tolist()
        K, W = (t.double().cpu().numpy() for t in
                self.cache.read(layer, ints(every), first=ints([0] * R), N=max(1, every[-1])))
        bf = self.dt == torch.bfloat16
        Q, got, scale = turned.double().cpu().numpy(), out.double().cpu().numpy(), DIM ** -0.5
        given = values.double().cpu().numpy()
        for s in range(R):
            k, w = K[every[s]:every[s + 1]], W[every[s]:every[s + 1]]
            before = self.held[layer][s]
            assert np.array_equal(k[:old[s]], before[0][:old[s]]) and np.array_equal(w[:old[s]], before[1][:old[s]])
            self.held[layer][s] = (k, w)
            if n[s] == 0:
                continue
            x = given[off[s]:off[s + 1]]
            assert np.array_equal(w[old[s]:], M.values(x) if self.four else x)
            mask = np.arange(old[s] + n[s])[None] > old[s] + np.arange(n[s])[:, None]
            for h in range(HEADS):
                g, q = h // (HEADS // KV), Q[off[s]:off[s + 1], h]
                z = np.where(mask, -math.inf, scale * q @ k[:, g].T)
                p = np.exp(z - z.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                B = (scale * np.abs(q) @ np.abs(k[:, g]).T).max(1, keepdims=True)
                want, A = p @ w[:, g], p @ np.abs(w[:, g])
                rel = 2 * U24 * ((DIM + 2) * B + 2 * B * 1.45 + 4) + (old[s] + n[s] + 16) * U24
                tol = A * (rel + (2.0 ** -8 if bf else 0)) + np.abs(want) * (2.0 ** -8 if bf else U24) + \
                    (old[s] + n[s]) * 2.0 ** -126 * np.abs(w).max()
                assert (np.abs(got[off[s]:off[s + 1], h] - want) <= tol).all(), (layer, s, h)


@pytest.mark.parametrize("dtype,four", [("bf16", True), ("f32", True), ("bf16", False), ("f32", False)])
def test_rounds(dev, dtype, four):  # noqa: F811
    t = Target(dev, dtype, 12, 48, four)
    rng = np.random.default_rng(9)
    some = lambda n: rng.integers(0, V, n).tolist()  # noqa: E731
    t.prompt([some(n) for n in (37, 0, 1, 16, 15)])
    accepted = t.round() + t.round()
    # request 3 becomes a second continuation of request 0
    t.cache.free(ints([3]))
    assert t.cache.fork(ints([0]), ints([3])).tolist() == [0]
    t.loop.anchors[3] = t.loop.anchors[0]
    t.kept[3] = list(t.kept[0])
    for held in t.held:
        held[3] = held[0]
    accepted += t.round() + t.round()
    # request 1 ends, the pages move together, a new request takes its place
    t.cache.free(ints([1]))
    t.kept[1] = []
    t.cache.compact()
    t.prompt([[], some(50), [], [], []])
    for _ in range(2):
        accepted += t.round()
    # both continuations back to where request 0's cache ended long ago
    t.cache.commit(ints([20 - len(t.kept[0]), -2 ** 31, -2 ** 31, 20 - len(t.kept[3]), -2 ** 31]))
    t.kept[0], t.kept[3] = t.kept[0][:20], t.kept[3][:20]
    accepted += t.round()
    assert 0 < np.mean(accepted) < GAMMA  # rounds of every kind


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_moved_into_four_bits(dev, dtype):  # noqa: F811
    """A request's tokens read out of a cache of whole elements go into a 4-bit cache: what that holds is
    what the same rows give directly."""
    import torch
    from draft_sampling_verification_w1_amd import cache
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    a = cache.PagedCache(2, 5, 12, 16, 1, KV, DIM, dt)
    b = cache.PagedCache(2, 5, 12, 32, 1, KV, DIM, cache.FOUR_BITS)
    lens, off, zero = ints([50, 21]), ints([0, 50, 71]), ints([0, 0])
    k, v = (torch.randn((71, KV, DIM), device="cuda").to(dt) for _ in range(2))
    for c in (a, b):
        c.reserve(lens)
    rot = cache.Rotation(cache.rope_frequencies(DIM))
    a.append(0, k, v, off, rotation=rot)
    moved = a.read(0, off, first=zero, N=71)
    b.append(0, *moved, off)
    got = b.read(0, off, N=71, dtype=dt)
    for x, y in zip(moved, got):
        assert np.array_equal(y.double().cpu().numpy(), M.values(x.double().cpu().numpy()))


def test_binding_refusals(dev):  # noqa: F811
    """Shapes, types, strides, devices and combinations that the Python calls turn down."""
    import torch
    from draft_sampling_verification_w1_amd import cache
    c = cache.PagedCache(3, 4, 9, 16, 1, 2, 64, cache.FOUR_BITS)
    w = cache.PagedCache(3, 4, 9, 16, 1, 2, 64)
    q = torch.zeros((6, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((6, 2, 64), dtype=torch.bfloat16, device="cuda")
    off, ws = ints([0, 2, 4, 6]), c.attend_workspace(6, 4)
    rot = cache.Rotation(cache.rope_frequencies(64))
    bad = [
        lambda: c.attend(0, q.half(), off), lambda: c.attend(0, q[::2], off), lambda: c.attend(0, q, off, out=q.float()),
        lambda: c.attend(0, q, off, ws=ws.cpu()), lambda: c.append(0, k, k.float(), off),
        lambda: c.append(0, k.half(), k.half(), off), lambda: c.append(0, k, k, off, q=q),
        lambda: w.append(0, k, k, off, q=q), lambda: w.append(0, k, k, off, q_out=q),
        lambda: c.append(0, k, k, off, rotation=rot, q=q.float()), lambda: c.append(0, k, k, off, rotation=rot, q_out=q),
        lambda: c.append(0, k, k, off, rotation=rot, q=q, q_out=q[:5]), lambda: w.append(0, k.float(), k.float(), off, rotation=rot),
        lambda: c.read(0, off), lambda: c.read(0, off, out=(k, k.float())), lambda: c.read(0, off, first=off, out=(k, k.clone())),
        lambda: c.read(0, off[:3], N=6), lambda: w.read(0, off, N=6, dtype=torch.float32), lambda: c.read(0, off, N=6, dtype=torch.half),
        lambda: cache.Rotation(rot.freqs.float()), lambda: cache.Rotation(rot.freqs.cpu()), lambda: cache.Rotation([1.0]),
        lambda: cache.Rotation(rot.freqs.view(2, -1)),
        lambda: cache.PagedCache.of(c.K, c.V, **c.tables()), lambda: cache.PagedCache.of(c.K, c.V, **c.tables(), shape=(16, 2, 128)),
        lambda: cache.PagedCache.of(w.K, w.V, **w.tables(), shape=(16, 2, 64)),
        lambda: cache.PagedCache.of(c.K, c.V[:, 1:], **c.tables(), shape=(16, 2, 64)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i}")
    refused = [
        lambda: c.attend(1, q, off), lambda: c.attend(0, q, off, scale=0.0), lambda: c.attend(0, q, off, out=q),
        lambda: c.attend(0, q, off, ws=ws[:-256]), lambda: c.append(-1, k, k, off), lambda: c.read(1, off, N=6),
        lambda: c.append(0, k, k, off, rotation=cache.Rotation(cache.rope_frequencies(80))),
        lambda: c.append(0, k, k, off, rotation=cache.Rotation(cache.rope_frequencies(24))),
        lambda: c.append(0, k, k, off, rotation=rot, q=q[:, :3].contiguous()), lambda: c.read(0, off, out=(k, k)),
    ]
    for call in refused:
        with pytest.raises(RuntimeError):
            call()
    same = cache.PagedCache.of(c.K, c.V, **c.tables(), shape=(16, 2, 64))
    assert same.dtype == cache.FOUR_BITS and same.head_dim == 64 and same.page_size == 16
