"""Attention over a 4-bit cache with a token without a value (an infinity or NaN in a block of its keys or values) among
the cached ones, which every row sees: the rows of that kv head are NaN, of values in the block's elements, wherever
the token lies on the key axis; the other heads are what they are."""
import math

import pytest

import test_gpu_attend4 as TQ
from test_gpu_attend4 import C, ints  # noqa: F401

pytestmark = pytest.mark.gpu


def spoil(b, slot, at, what, block, x):
    """Token `at` of a slot again, of the last kv head with an element x in `block`."""
    k, v = (t[b.old[slot] + at:b.old[slot] + at + 1].to(b.dt) for t in (b.old_k, b.old_v))
    (k if what == "keys" else v)[0, -1, 32 * block + 7] = x
    lens = list(b.lens)
    lens[slot] = at
    b.c.lens.copy_(ints(lens))
    one = [0] * (slot + 1) + [1] * (len(lens) - slot)
    b.c.append(b.layer, k.cuda(), v.cuda(), ints(one))
    b.c.lens.copy_(ints(b.lens))


@pytest.mark.parametrize("dtype,heads,kv,dim", [("bf16", 4, 2, 64), ("bf16", 8, 2, 128), ("bf16", 4, 2, 256),
                                                ("f32", 4, 2, 64), ("f32", 4, 2, 128), ("f32", 2, 2, 256)])
@pytest.mark.parametrize("chunk", [1, 17, 70])
@pytest.mark.parametrize("at", [0, 31, 500, 2999])
@pytest.mark.parametrize("what,x", [("keys", math.nan), ("keys", -math.inf), ("values", math.inf)])
def test_seen_by_every_row(C, dtype, heads, kv, dim, chunk, at, what, x):  # noqa: F811
    b = TQ.Batch(C, dtype, 16 if at % 2 else 64, heads, kv, dim, [3000, 40], [chunk, 2], seed=chunk)
    out = b.run(max_chunk=chunk)
    b.check(out)
    block = dim // 32 - 1
    spoil(b, 0, at, what, block, x)
    got = b.run(max_chunk=chunk)
    where = slice(0, dim) if what == "keys" else slice(32 * block, dim)
    bad = got[:chunk, heads // 2:]
    assert bad[..., where].isnan().all()
    got[:chunk, heads // 2:] = out[:chunk, heads // 2:]
    b.check(got)


@pytest.mark.parametrize("chunk", [1, 20])
def test_beside_queries_multiplied_in_bf16(C, chunk):  # noqa: F811
    """The same where the rows' elements lie far apart."""
    b = TQ.Batch(C, "bf16", 32, 8, 2, 128, [700, 40], [chunk, 2])
    b.q[..., 9] *= 2.0 ** 30
    spoil(b, 0, 333, "keys", 2, math.nan)
    got = b.run(max_chunk=chunk)
    assert got[:chunk, 4:].isnan().all() and not got[:chunk, :4].isnan().any()


def test_only_nan(C):  # noqa: F811
    """A row whose only key has no value, and a row without any key beside it."""
    b = TQ.Batch(C, "bf16", 16, 4, 2, 128, [1, 0], [1, 1])
    spoil(b, 0, 0, "keys", 1, math.nan)
    table = b.c.table.cpu()
    table[1, 0] = -1
    b.c.table.copy_(table)
    got = b.run(max_chunk=1)
    assert got[0, 2:].isnan().all() and not got[0, :2].isnan().any() and not got[1].any()
