"""Attention over a 4-bit cache: tokens without a value (an infinity or NaN among their keys or values) behind
some rows.  Rows that don't see them are what they are without them, to the tolerance
of test_gpu_attend4.py; the others are NaN, of values in the block's 32 elements."""
import math

import pytest

import test_gpu_attend4 as TQ
from test_gpu_attend4 import C, ints  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,heads,kv,dim", [("bf16", 4, 2, 64), ("bf16", 8, 2, 128), ("bf16", 4, 2, 256), ("f32", 4, 2, 64),
                                                ("f32", 4, 2, 128), ("f32", 2, 2, 256)])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("chunk,at", [(2, 1), (9, 3), (17, 16), (70, 33), (300, 1)])
@pytest.mark.parametrize("what", ["keys", "values"])
def test_nothing_seen_of_later_tokens(C, dtype, heads, kv, dim, page, chunk, at, what):  # noqa: F811
    import torch
    lens, chunks = [45, 0, 500], [chunk, chunk, 1]
    b = TQ.Batch(C, dtype, page, heads, kv, dim, lens, chunks)
    out = b.run(max_chunk=chunk)
    b.check(out)
    # tokens `at` of the first two slots, of kv head 1 alone, in one block of 32 each
    k, v = (torch.randn((2, kv, dim)).to(b.dt) for _ in range(2))
    bad = k if what == "keys" else v
    bad[0, 1, 3], bad[1, 1, dim - 1] = math.nan, math.inf
    for s in range(2):
        b.c.lens.copy_(ints([n + at for n in lens]))
        one = [0] * (s + 1) + [1] * (3 - s)
        b.c.append(b.layer, k[s:s + 1].cuda(), v[s:s + 1].cuda(), ints(one))
    b.c.lens.copy_(ints(lens))
    # the tokens' other heads have other numbers now, too
    held = lambda t: torch.from_numpy(TQ.M.values(t.double().numpy()))  # noqa: E731
    for s in range(2):
        row = b.off[s] + at
        b.k[row, 0], b.v[row, 0] = held(k[s:s + 1])[0, 0], held(v[s:s + 1])[0, 0]
    got = b.run(max_chunk=chunk)
    for s in range(2):  # rows that see kv head 1's token
        rows = slice(b.off[s] + at, b.off[s] + chunk)
        block = slice(0, dim) if what == "keys" else (slice(0, 32) if s == 0 else slice(dim - 32, dim))
        assert got[rows, heads // 2:, block].isnan().all()
        got[rows, heads // 2:] = out[rows, heads // 2:]
    assert not got[:b.off[-1]].isnan().any()
    b.check(got)
