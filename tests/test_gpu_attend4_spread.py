"""Attention over a 4-bit cache where the elements of a bf16 query lie further apart than the two 8-bit operands of a
row reach, and the keys have their weight where the query is small.

Tolerance: that of test_gpu_attend4.py (the bound of a score goes by the products that are there, sum |q k|) and the score's
error by the operands, up to 2^-11 of a binary logarithm for each weight, numerator and denominator alike."""
import math

import numpy as np
import pytest
import torch

import test_gpu_attend4 as TQ
from test_gpu_attend4 import C, ints  # noqa: F401

pytestmark = pytest.mark.gpu

U = TQ.U
SPLIT = 2.0 ** -11 * math.log(2) * 1.01


def change(b, keys, queries):
    """The same tokens and rows with other keys and queries; keys(x) and queries(x) get [n, heads, dim] in binary64."""
    def put(x, v, off):
        x = keys(x).to(b.dt)
        b.c.append(b.layer, x.cuda(), v.to(b.dt).cuda(), ints(off))
        return torch.from_numpy(TQ.M.values(x.double().numpy()))
    b.c.lens.zero_()
    b.old_k = put(b.old_k, b.old_v, b.old)
    b.c.lens.copy_(ints(b.lens))
    b.k = put(b.k, b.v, b.off)
    b.q = queries(b.q.double()).to(b.dt)


def check(b, out):
    got = out.double().cpu().numpy()
    G, scale = b.heads // b.kv, b.dim ** -0.5
    for s, (ln, n) in enumerate(zip(b.lens, b.chunks)):
        a, o = b.off[s], b.old[s]
        keys, vals = torch.cat([b.old_k[o:o + ln], b.k[a:a + n]]), torch.cat([b.old_v[o:o + ln], b.v[a:a + n]])
        mask = torch.arange(ln + n)[None] > ln + torch.arange(n)[:, None]
        for h in range(b.heads):
            q, kk, vv = b.q[a:a + n, h].double(), keys[:, h // G], vals[:, h // G]
            B = (scale * q.abs() @ kk.abs().T).amax(1).numpy()[:, None]
            w = torch.softmax((scale * q @ kk.T).masked_fill(mask, -math.inf), 1)
            want, A = (w @ vv).numpy(), (w @ vv.abs()).numpy()
            rel = U * ((b.dim + 2) * B + 2 * B * 1.45 + 4) * 2 + (ln + n + 16) * U + 2 * SPLIT
            tol = A * (rel + 2.0 ** -8) + np.abs(want) * 2.0 ** -8 + (ln + n) * 2.0 ** -126 * float(vv.abs().max())
            off = np.abs(got[a:a + n, h] - want)
            at = np.unravel_index(np.argmax(off / (tol + 1e-300)), off.shape)
            assert (off <= tol).all(), (s, h, at, got[a:a + n, h][at], want[at], A[at], tol[at])
    assert (got[b.off[-1]:] == 7.5).all()


SHAPES = [(4, 4, 64), (8, 2, 128), (3, 1, 256)]


@pytest.mark.parametrize("heads,kv,dim", SHAPES)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("chunk", [1, 9, 20, 60, 130])
@pytest.mark.parametrize("far", [10, 14, 18, 22, 40, 80])
def test_outliers_where_keys_are_zero(C, heads, kv, dim, page, chunk, far):  # noqa: F811
    """A few query elements 2^far above the others; odd rows have none."""
    b = TQ.Batch(C, "bf16", page, heads, kv, dim, [300, 37], [chunk, max(1, chunk // 3)], seed=chunk)
    at = [5, 40, dim - 1]

    def keys(x):
        x = x.clone()
        x[..., at] = 0
        return x

    def queries(x):
        x[0::2, :, at] *= 2.0 ** far
        return x
    change(b, keys, queries)
    check(b, b.run(max_chunk=chunk))


@pytest.mark.parametrize("heads,kv,dim", SHAPES)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("chunk", [1, 9, 20, 60, 130])
@pytest.mark.parametrize("far", [10, 14, 18, 22, 40])
def test_large_keys_where_queries_are_small(C, heads, kv, dim, page, chunk, far):  # noqa: F811
    """Keys of one block of 32 elements alone, 2^far times a normal variate, where the query's are 2^-far."""
    b = TQ.Batch(C, "bf16", page, heads, kv, dim, [300, 37], [chunk, max(1, chunk // 3)], seed=chunk)
    block = (torch.arange(dim) // 32 == 1).double()

    def keys(x):
        return x * block * 2.0 ** far

    def queries(x):
        return x * torch.where(block > 0, 2.0 ** -far, 1.0)
    change(b, keys, queries)
    check(b, b.run(max_chunk=chunk))


@pytest.mark.parametrize("heads,kv,dim", SHAPES)
@pytest.mark.parametrize("size", [-30, -12, 0, 12, 30])
def test_large_and_small_keys(C, heads, kv, dim, size):  # noqa: F811
    """Normal variates, the keys' size against the queries': scores as always."""
    b = TQ.Batch(C, "bf16", 32, heads, kv, dim, [300, 37], [20, 7])
    change(b, lambda x: x * 2.0 ** size, lambda x: x * 2.0 ** -size)
    check(b, b.run(max_chunk=20))


def test_a_few_tokens_with_large_keys(C):  # noqa: F811
    """Steps that need the exact products beside steps that don't, in one row."""
    b = TQ.Batch(C, "bf16", 16, 8, 2, 128, [700, 90], [5, 17])
    at = torch.arange(128) % 32 == 3

    def keys(x):
        x = x.clone()
        x[..., at] = 0
        x[::50] = torch.where(at, 2.0 ** 20, 0.0) * torch.randn_like(x[::50])
        return x

    def queries(x):
        x[..., at] *= 2.0 ** -20
        x[..., ~at] *= 2.0
        return x
    change(b, keys, queries)
    check(b, b.run(max_chunk=17))
