"""Chunk attention (dspark_attend) where its tiling and its numbers have their ends,
against binary64 with the bounds of test_gpu_attend.py."""

import pytest

from test_gpu_attend import Batch, C, ints  # noqa: F401

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
