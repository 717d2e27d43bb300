"""Chunk attention over a 4-bit cache (dspark_attend4) against binary64 over what the codes stand for.

Tolerance per element, u = 2^-24, A = sum_p w_p |v_p| with the weights w of the row,
B = max_p scale sum_d |q_d k_d|, as of the attention over whole elements (test_gpu_attend.py): a score is a sum of
head_dim products in binary32, off by at most (head_dim + 2) u B; the exponential adds u (|s - m| log2 e + 4) with
|s - m| <= 2B; both change a weight relatively, numerator and denominator alike.  Sums over n keys add n u.  bf16
rounds each weight (2^-8) for the product with v; the result is rounded once (2^-8 bf16, 2^-24 fp32).
A weight below 2^-126 of the largest is no normal number of binary32 and counts as 0, and so may a part's
factor: that is off by up to 2^-126 max|v| per key (4-bit values are often 0 where the large weights are, so that A
itself can be as small)."""
import math

import numpy as np
import pytest

import mx_model as M
import test_gpu_attend as TA

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
C = TA.C
ints = TA.ints


class Batch(TA.Batch):
    """As for whole elements; the tokens' keys and values are those that 4 bits stand for."""

    def __init__(self, C, dtype, page, heads, kv, dim, lens, chunks, seed=0, layers=2, extra=3,
                 scale=1.0, pages=None):
        import torch
        self.dt = torch.float32 if dtype == "f32" else torch.bfloat16
        g = torch.Generator().manual_seed(seed)
        S = len(lens)
        self.lens, self.chunks, self.page, self.dim, self.heads, self.kv = lens, chunks, page, dim, heads, kv
        need = [-(-(ln + c) // page) for ln, c in zip(lens, chunks)]
        width = max(max(need), 1) + 1
        total = sum(need) + 7 if pages is None else pages
        c = C.PagedCache(S, width, total, page, layers, kv, dim, C.FOUR_BITS)
        if pages is None:  # codes and scales outside the tokens: all bits set, NaN
            c.K.fill_(255)
            c.V.fill_(255)
        order = torch.randperm(total, generator=g)[:sum(need)] if pages is None else \
            total - 1 - torch.arange(sum(need))
        table = torch.full((S, width), -1, dtype=torch.int32)
        at = 0
        for s in range(S):
            table[s, :need[s]] = order[at:at + need[s]].to(torch.int32)
            at += need[s]
        c.table.copy_(table)
        c.lens.zero_()
        c.held.copy_(ints(need))
        self.c, self.off = c, [0] + np.cumsum(chunks).tolist()
        self.layer = layers - 1
        old = [0] + np.cumsum(lens).tolist()
        rand = lambda n, h: (torch.randn((n, h, dim), generator=g) * scale).to(self.dt)  # noqa: E731
        held = lambda t: torch.from_numpy(M.values(t.double().numpy()))  # noqa: E731
        old_k, old_v = rand(max(1, old[-1]), kv), rand(max(1, old[-1]), kv)
        old_k[..., 5::16] *= 4
        self.old = old
        c.append(self.layer, old_k.cuda(), old_v.cuda(), ints(old))
        c.lens.copy_(ints(lens))
        N = self.off[-1] + extra
        self.q, k, v = rand(N, heads), rand(N, kv), rand(N, kv)
        self.offsets = ints(self.off)
        c.append(self.layer, k.cuda(), v.cuda(), self.offsets)
        self.old_k, self.old_v, self.k, self.v = held(old_k), held(old_v), held(k), held(v)


    def check(self, out, scale=None, hidden=()):
        """hidden: {(slot, page column)} that count as absent."""
        import torch
        scale = self.dim ** -0.5 if scale is None else scale
        got = out.double().cpu().numpy()
        G = self.heads // self.kv
        bf = self.dt == torch.bfloat16
        for s, (ln, n) in enumerate(zip(self.lens, self.chunks)):
            a, o = self.off[s], self.old[s]
            if n == 0:
                continue
            keys = torch.cat([self.old_k[o:o + ln], self.k[a:a + n]]).double()
            vals = torch.cat([self.old_v[o:o + ln], self.v[a:a + n]]).double()
            gone = torch.tensor([(s, p // self.page) in hidden for p in range(ln + n)], dtype=torch.bool)
            mask = torch.arange(ln + n)[None] > ln + torch.arange(n)[:, None]
            mask = mask | gone[None]
            for h in range(self.heads):
                q = self.q[a:a + n, h].double()
                kk, vv = keys[:, h // G], vals[:, h // G]
                B = (scale * q.abs() @ kk.abs().T).amax(1)
                w = torch.softmax((scale * q @ kk.T).masked_fill(mask, -math.inf), 1)
                w = torch.where(mask.all(1, keepdim=True), 0.0, w)
                want, A = (w @ vv).numpy(), (w @ vv.abs()).numpy()
                rel = U * ((self.dim + 2) * B + 2 * B * 1.45 + 4) * 2 + (ln + n + 16) * U
                tol = A * (rel.numpy()[:, None] + (2.0 ** -8 if bf else 0)) + \
                    np.abs(want) * (2.0 ** -8 if bf else U) + (ln + n) * 2.0 ** -126 * float(vv.abs().max())
                off = np.abs(got[a:a + n, h] - want)
                at = np.unravel_index(np.argmax(off / (tol + 1e-300)), off.shape)
                assert (off <= tol).all(), (s, h, at, got[a:a + n, h][at], want[at], A[at], tol[at])
        assert (got[self.off[-1]:] == 7.5).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("heads,kv,dim", [(4, 4, 64), (8, 2, 128), (2, 1, 256)])
def test_ragged(C, dtype, page, heads, kv, dim):
    """Lengths around the pages' and tiles' ends, chunks of 0 to 40 tokens."""
    lens = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 100, 255, 256, 300, 0]
    chunks = [1, 1, 2, 0, 17, 9, 1, 32, 1, 16, 5, 1, 3, 40, 0]
    b = Batch(C, dtype, page, heads, kv, dim, lens, chunks)
    b.check(b.run(max_chunk=40))
    b.check(b.run(max_chunk=1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,dim", [(7, 1, 64), (28, 4, 128), (32, 8, 128), (16, 2, 256), (24, 8, 64),
                                          (5, 5, 128), (64, 1, 128)])
@pytest.mark.parametrize("chunk", [1, 5, 9, 17])
def test_groups(C, dtype, heads, kv, dim, chunk):
    b = Batch(C, dtype, 16, heads, kv, dim, [37, 250], [chunk, chunk], seed=chunk)
    b.check(b.run(max_chunk=chunk))


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("heads,kv,dim", [(4, 1, 64), (4, 1, 128), (3, 1, 128), (2, 1, 256)])
@pytest.mark.parametrize("chunk", [4, 8, 12, 16, 20, 24, 32, 48, 64, 96, 130])
def test_tiles(C, page, heads, kv, dim, chunk):
    """Every tile, full and cut."""
    b = Batch(C, "bf16", page, heads, kv, dim, [700, 33], [chunk, chunk - 1], seed=chunk)
    b.check(b.run(max_chunk=chunk))


@pytest.mark.parametrize("dtype,dim,ctx,chunk", [
    ("bf16", 128, 20000, 1), ("bf16", 64, 9000, 17), ("f32", 128, 5000, 3), ("bf16", 256, 7001, 5),
    ("bf16", 128, 0, 700), ("bf16", 128, 1500, 333), ("f32", 64, 100, 200)])
def test_long(C, dtype, dim, ctx, chunk):
    """Key ranges split over workgroups, and chunks longer than a tile."""
    b = Batch(C, dtype, 16 if ctx % 2 else 64, 4, 2, dim, [ctx, ctx // 3], [chunk, max(1, chunk // 2)])
    b.check(b.run(max_chunk=chunk))
    b.check(b.run())


@pytest.mark.parametrize("slots", [257, 4096])
def test_many_slots(C, slots):
    rng = np.random.default_rng(slots)
    lens, chunks = rng.integers(0, 20, slots).tolist(), rng.integers(0, 4, slots).tolist()
    b = Batch(C, "bf16", 16, 2, 1, 64, lens, chunks)
    b.check(b.run(max_chunk=3))


@pytest.mark.parametrize("dtype,heads,kv,dim", [("bf16", 4, 1, 64), ("bf16", 8, 4, 128), ("bf16", 12, 1, 256),
                                                ("f32", 6, 3, 128)])
@pytest.mark.parametrize("chunk", [1, 9, 60])
def test_short_beside_long(C, dtype, heads, kv, dim, chunk):
    """Groups of one key step next to groups of a hundred, slots without rows between."""
    lens = [0, 0, 3300, 1, 40, 5, 1200, 31, 0, 64, 2]
    chunks = [1, chunk, chunk, 0, 1, chunk, 1, min(chunk, 2), 0, chunk, 1]
    b = Batch(C, dtype, 32, heads, kv, dim, lens, chunks, seed=chunk)
    b.check(b.run(max_chunk=chunk))
    b.check(b.run(max_chunk=1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.5, 30.0])
def test_large_scores(C, dtype, scale):
    """Scores far apart: the running maximum moves often and by much."""
    b = Batch(C, dtype, 16, 8, 2, 128, [700, 90], [5, 17], scale=4.0)
    b.check(b.run(max_chunk=17, scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("chunk", [3, 130])
def test_far_scores(C, dtype, chunk):
    """One key's score lies so far from zero that the others' weights vanish: the result is its value."""
    import torch
    b = Batch(C, dtype, 32, 4, 1, 128, [150], [chunk])
    k = torch.zeros((150 + chunk, 1, 128))
    k[:, 0, 0] = -1.0
    k[77, 0, 0] = 4.0
    v = torch.randn((150 + chunk, 1, 128)).to(b.dt)
    b.c.lens.zero_()
    b.c.append(b.layer, k.to(b.dt).cuda(), v.cuda(), ints([0, 150 + chunk]))
    b.c.lens.copy_(ints([150]))
    q = torch.zeros_like(b.q)
    q[..., 0] = 2.0 ** 60
    out = b.c.attend(b.layer, q.cuda(), b.offsets, scale=2.0 ** 30, max_chunk=chunk)
    want = torch.from_numpy(M.values(v[77:78].double().numpy()))
    assert torch.equal(out[:chunk].double().cpu(), want.expand(chunk, 4, 128))


def test_absent_pages(C):
    """A hole in a slot's table, ids outside the pool and a slot without any page:
    their keys are not there; a token that sees none gives 0."""
    for chunk, dtype in ((3, "bf16"), (3, "f32"), (40, "bf16")):
        b = Batch(C, dtype, 16, 4, 2, 64, [100, 64, 5], [chunk, 2, 1])
        t = b.c.table.cpu()
        t[0, 2], t[0, 5], t[1, 0], t[2, 0] = -1, b.c.pages, 2 ** 31 - 1, -7
        b.c.table.copy_(t)
        b.check(b.run(max_chunk=chunk), hidden={(0, 2), (0, 5), (1, 0), (2, 0)})


def test_far_pages(C):
    """Byte offsets past 2^32 in K and V."""
    import torch
    free, _ = torch.cuda.mem_get_info()
    pages = 2 ** 32 // (8 * 16 * 128 * 17 // 32) + 200
    if free < 3 * pages * 8 * 16 * 128:
        pytest.skip("not enough memory")
    b = Batch(C, "bf16", 16, 8, 8, 128, [300, 41], [5, 1], layers=1, pages=pages)
    b.check(b.run(max_chunk=5))


def test_zero_and_tiny_scales(C):
    """Blocks whose scale is the smallest there is, next to ordinary ones."""
    import torch
    b = Batch(C, "bf16", 16, 4, 2, 64, [64], [2])
    k, v = torch.randn((66, 2, 64)).bfloat16(), torch.randn((66, 2, 64)).bfloat16()
    k[10:20], v[15:25] = 0, 0
    k[30, :, 32:] = 1e-38
    v[31, :, :32] = 1e-39
    b.c.lens.zero_()
    b.c.append(b.layer, k.cuda(), v.cuda(), ints([0, 66]))
    b.c.lens.copy_(ints([64]))
    held = lambda t: torch.from_numpy(M.values(t.double().numpy()))  # noqa: E731
    b.old_k, b.old_v, b.k, b.v = held(k[:64]), held(v[:64]), held(k[64:]), held(v[64:])
    b.check(b.run(max_chunk=2))


def test_replayed_graph_and_streams(C):
    """attend inside a graph, replayed with other queries and lengths between eager calls;
    two graphs on one workspace; a stream of its own."""
    import torch
    b = Batch(C, "bf16", 16, 8, 2, 128, [300, 2000, 40], [5, 1, 9])
    c, q = b.c, b.q.cuda()
    ws = c.attend_workspace(q.shape[0], 8)
    out, out2 = torch.zeros_like(q), torch.zeros_like(q)
    c.attend(b.layer, q, b.offsets, out=out, ws=ws)
    torch.cuda.synchronize()
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attend(b.layer, q, b.offsets, max_chunk=9, out=out, ws=ws)
    with torch.cuda.graph(g2):
        c.attend(b.layer, q, b.offsets, max_chunk=9, out=out2, ws=ws)
    side = torch.cuda.Stream()
    for i in range(4):
        q.normal_()
        c.lens.copy_(ints([300 - i, 2000 - 17 * i, 40 - 40 * (i == 3)]))
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        eager = c.attend(b.layer, q, b.offsets, max_chunk=9, out=torch.zeros_like(q))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            other = c.attend(b.layer, q, b.offsets, max_chunk=9, out=torch.zeros_like(q))
        side.synchronize()
        assert torch.equal(out, eager) and torch.equal(out2, eager) and torch.equal(other, eager)
