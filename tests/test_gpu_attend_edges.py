"""Chunk attention (dspark_attend) where its tiling and its numbers have their ends,
against binary64 with the bounds of test_gpu_attend.py."""
import pytest

from test_gpu_attend import U, Batch, C, ints  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,heads,kv,dim,chunk", [
    ("bf16", 2, 2, 128, 1153),    # three tiles of 384 rows and one row
    ("bf16", 3, 1, 64, 385),
    ("bf16", 8, 2, 128, 290),
    ("bf16", 7, 1, 64, 220),
    ("bf16", 2, 2, 256, 400), ("bf16", 3, 1, 256, 129), ("bf16", 4, 1, 256, 97),
    ("f32", 3, 3, 64, 97), ("f32", 4, 1, 128, 25), ("f32", 7, 1, 256, 14)])
@pytest.mark.parametrize("before", [False, True])
def test_short_last_tile(C, dtype, heads, kv, dim, chunk, before):  # noqa: F811
    """Four tiles or more, the last one almost empty, at the end of the batch's work and
    in front of another slot's."""
    lens, chunks = ([30, 77], [chunk, 5]) if before else ([0, 30], [3, chunk])
    b = Batch(C, dtype, 32, heads, kv, dim, lens, chunks, seed=chunk)
    b.check(b.run(max_chunk=chunk))
    b.check(b.run(max_chunk=max(1, chunk // 4)))


@pytest.mark.parametrize("dtype,heads,kv,dim,chunk", [("bf16", 2, 2, 128, 1600), ("f32", 2, 1, 64, 150)])
def test_table_shorter_than_the_chunk(C, dtype, heads, kv, dim, chunk):  # noqa: F811
    """Tokens behind the table's last position are dropped; every row sees the others."""
    import torch
    b = Batch(C, dtype, 16, heads, kv, dim, [20, 40], [chunk, 2])
    c, width = b.c, 4
    table, held = c.table[:, :width].contiguous(), c.held.clamp(max=width)
    b.c = C.PagedCache.of(c.K, c.V, table, c.lens, held, c.refs, c.free_bits, c.n_free)
    columns = range(width, -(-(20 + chunk) // 16))
    b.check(b.run(max_chunk=chunk), hidden={(0, j) for j in columns})
    assert torch.equal(c.lens, ints([20, 40]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("exponent", [8, 20, 24, 25, 31, 33, 40, 60, 97])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("heads,kv,dim,chunk", [(4, 2, 64, 1), (2, 2, 128, 40), (8, 1, 128, 40), (2, 1, 256, 17)])
def test_far_scores(C, dtype, exponent, sign, heads, kv, dim, chunk):  # noqa: F811
    """Scaled scores of up to 2^98 = 3.2e29 in magnitude.

    A score is exact: one dimension of query and key holds a power of two (times 65/64 or
    66/64), the others nothing.  Its product with log2 e is not.  Every third key has the
    largest score x, the others lie |x| / 65 and about |x| behind it.  From 2^20 on only the
    largest have a weight, all the same; at 2^8 the next ones have e^-4: an exponent of 4
    log2 e costs two roundings and that of log2 e, the exponential two more: (3 * 5.8 + 2) u.
    Sums of n keys add n u; bf16 rounds the weights and the result (2^-8 each)."""
    import torch
    lens, chunks = [70, 333], [chunk, chunk]
    b = Batch(C, dtype, 16, heads, kv, dim, lens, chunks, seed=exponent)
    low, far = (1.0, 0.0) if sign > 0 else (66 / 64, 2.0)

    def keys(n):
        k = torch.zeros((n, kv, dim))
        i = torch.arange(n)[:, None]
        k[..., 3] = torch.where(i % 3 == 0, 65 / 64, torch.where(i % 3 == 1, low, far))
        return (k * (sign * 2.0 ** (exponent - exponent // 2))).to(b.dt)

    b.q = torch.zeros_like(b.q)
    b.q[..., 3] = 2.0 ** (exponent // 2)
    b.old_k, b.k = keys(len(b.old_k)), keys(len(b.k))
    b.c.lens.zero_()
    b.c.append(b.layer, b.old_k.cuda(), b.old_v.cuda(), ints(b.old))
    b.c.lens.copy_(ints(lens))
    b.c.append(b.layer, b.k.cuda(), b.v.cuda(), b.offsets)
    bf = dtype == "bf16"
    for most in (chunk, 1):
        got = b.run(max_chunk=most, scale=1.0).double().cpu()
        for s, (ln, n) in enumerate(zip(lens, chunks)):
            a, o = b.off[s], b.old[s]
            kk = torch.cat([b.old_k[o:o + ln], b.k[a:a + n]]).double()
            vv = torch.cat([b.old_v[o:o + ln], b.v[a:a + n]]).double()
            mask = torch.arange(ln + n)[None] > ln + torch.arange(n)[:, None]
            for h in range(heads):
                sc = b.q[a:a + n, h].double() @ kk[:, h // (heads // kv)].T
                w = torch.softmax(sc.masked_fill(mask, -torch.inf), 1)
                v = vv[:, h // (heads // kv)]
                want, A = w @ v, w @ v.abs()
                tol = A * ((ln + n + 36) * U + (2.0 ** -8 if bf else 0)) + want.abs() * (2.0 ** -8 if bf else U)
                off = (got[a:a + n, h] - want).abs()
                assert (off <= tol).all(), (most, s, h, float((off / tol).max()))
