"""Rotated keys in 4 bits, and rotated queries, follow from the definition bit for bit (c and s rounded to binary32, then
every product and sum): at small positions and near 10^6, with pages there.  The model's sines and cosines come from
numpy in binary64; with these seeds none is close enough to a rounding border to matter."""
import numpy as np
import pytest

import mx_model as M
from test_gpu_cache_store import C, host, ints  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,dim", [(4, 4, 64), (8, 2, 128), (2, 1, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("start", [0, 1000, 999_990, (1 << 20) + 5])
def test_bit_for_bit(C, rows, heads, kv, dim, interleaved, start):  # noqa: F811
    import torch
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[rows]
    page, n = 256, 40
    lens, chunks = [start, start + 133], [n, n - 9]
    width = (lens[1] + n) // page + 1
    c = C.PagedCache(2, width, 6, page, 1, kv, dim, C.FOUR_BITS)
    table, free = torch.full((2, width), -1, dtype=torch.int32), [4, 1, 5, 0]
    for s in range(2):
        for j in range(lens[s] // page, (lens[s] + chunks[s] - 1) // page + 1):
            table[s, j] = free.pop()
    c.table.copy_(table)
    c.lens.copy_(ints(lens))
    c.held.fill_(width)
    g = torch.Generator().manual_seed(start + dim)
    N = sum(chunks)
    q, k, v = ((torch.randn((N, h, dim), generator=g) * 2.0 ** torch.randint(-3, 4, (N, 1, 1), generator=g)).to(dt)
               for h in (heads, kv, kv))
    freqs = C.rope_frequencies(dim, 1e4)
    got = c.append(0, k.cuda(), v.cuda(), ints([0, n, N]), rotation=C.Rotation(freqs, interleaved), q=q.cuda())
    pos = np.concatenate([np.arange(a, a + b) for a, b in zip(lens, chunks)])
    f = freqs.cpu().numpy()
    want = M.rotate(host(q), pos, f, interleaved)
    assert want.dtype == np.float32
    assert torch.equal(got.cpu(), torch.from_numpy(want).to(dt))
    # sums of unrounded products give other results: the comparison would see one
    apart = M.rotate(host(q), pos, f, interleaved, exact=True).astype(np.float32)
    assert start == 0 or not np.array_equal(apart, want)
    turned = M.rotate(host(k), pos, f, interleaved)
    scales, seen = M.scale_bytes(turned), {}
    codes = M.values(turned, scales)
    pool = c.K[0].cpu().numpy()
    row = 0
    for s in range(2):
        for p in range(lens[s], lens[s] + chunks[s]):
            at = int(table[s, p // page])
            if at not in seen:
                seen[at] = M.unpack(pool[at], "K", kv, page, dim)
            x, sc = (t[p % page] for t in seen[at])
            assert np.array_equal(sc, scales[row])
            assert np.array_equal(x * np.repeat(np.exp2(sc.astype(float) - 127), 32, -1), codes[row])
            row += 1
