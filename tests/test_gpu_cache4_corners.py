"""Calls that the documents allow and other tests do not make: rotations of every permitted number of dimensions, and pages
whose scale bytes somebody else laid down."""
import numpy as np
import pytest

import mx_model as M
from test_gpu_cache_store import C, host, ints  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bits", [False, True])
def test_every_number_of_dimensions(C, dim, interleaved, bits):  # noqa: F811
    """Multiples of 16 that are no powers of two: elements behind them stay, queries and keys alike."""
    import torch
    g = torch.Generator().manual_seed(dim)
    N, pos = 11, np.arange(37, 48)
    q, k, v = (torch.randn((N, h, dim), generator=g) for h in (4, 2, 2))
    for rot in range(16, dim + 1, 16):
        c = C.PagedCache(1, 4, 4, 16, 1, 2, dim, C.FOUR_BITS if bits else torch.float32)
        c.table.copy_(torch.tensor([[2, 0, 3, 1]], dtype=torch.int32))
        c.lens.fill_(37)
        c.held.fill_(4)
        freqs = C.rope_frequencies(rot, 1e4)
        got = c.append(0, k.cuda(), v.cuda(), ints([0, N]), rotation=C.Rotation(freqs, interleaved), q=q.cuda())
        f = freqs.cpu().numpy()
        assert np.array_equal(got.cpu().numpy(), M.rotate(host(q), pos, f, interleaved))
        turned = M.rotate(host(k), pos, f, interleaved)
        back, values = c.read(0, ints([0, N]), N=N, dtype=torch.float32)
        assert np.array_equal(host(back), M.values(turned) if bits else turned)
        assert np.array_equal(host(values), M.values(host(v)) if bits else host(v))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_scale_byte_and_code(C, dtype):  # noqa: F811
    """256 tokens of a page, each with a scale byte of its own and all codes: what read makes of them."""
    import torch
    dim, page = 64, 256
    c = C.PagedCache(1, 1, 1, page, 1, 1, dim, C.FOUR_BITS)
    c.table.zero_()
    c.held.fill_(1)
    codes = page * dim // 2
    for pool in (c.K, c.V):
        pool[0, 0, :codes] = (torch.arange(codes, device="cuda") * 37 % 256).to(torch.uint8)
        pool[0, 0, codes:] = torch.arange(page, device="cuda").repeat(dim // 32).to(torch.uint8)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    k, v = c.read(0, ints([0, page]), N=page, dtype=dt)
    for name, pool, got in (("K", c.K, k), ("V", c.V, v)):
        x, scales = M.unpack(pool[0, 0].cpu().numpy(), name, 1, page, dim)
        want = torch.from_numpy(x * np.repeat(np.exp2(scales.astype(float) - 127), 32, -1))
        want = want.to(dt)  # 254: 4 and 6 are beyond the type, infinite
        assert got[255].isnan().all()
        assert torch.equal(got[:255].cpu(), want[:255])


@pytest.mark.parametrize("heads,kv,dim", [(4, 4, 64), (8, 2, 128), (3, 1, 256)])
@pytest.mark.parametrize("size", [-110, -60, 60, 110])
@pytest.mark.parametrize("far", [0, 20])
def test_keys_and_queries_far_from_one(C, heads, kv, dim, size, far):  # noqa: F811
    """Keys of 2^size and queries of 2^-size, some of them with an element 2^far above the others where keys are zero."""
    import test_gpu_attend4 as TQ
    import test_gpu_attend4_spread as TS
    b = TQ.Batch(C, "bf16", 32, heads, kv, dim, [300, 37], [20, 7])

    def keys(x):
        x = x * 2.0 ** size
        x[..., 11] = 0
        return x

    def queries(x):
        x = x * 2.0 ** -size
        x[::2, :, 11] *= 2.0 ** (far if size >= 0 else min(far, 10))
        return x
    TS.change(b, keys, queries)
    TS.check(b, b.run(max_chunk=20))
