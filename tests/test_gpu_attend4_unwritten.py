"""Attention over a 4-bit cache does not depend, in any bit, on what its pages hold where no token was written, nor on pages
of no slot."""
import pytest
import torch

import test_gpu_attend4 as TQ
from test_gpu_attend4 import C, ints  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,dim", [(4, 4, 64), (8, 2, 128), (2, 1, 256)])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("chunk", [1, 9, 40, 130])
def test_same_bits(C, dtype, heads, kv, dim, page, chunk):  # noqa: F811
    b = TQ.Batch(C, dtype, page, heads, kv, dim, [300, 3, 0, 70, 900], [chunk, chunk, 0, 1, max(1, chunk // 2)])
    b.q[..., 3] *= 64.0  # some elements lie further from the largest
    t = b.c.table.cpu()
    t[3, 1 if page < 64 else 0] = -1  # a hole
    b.c.table.copy_(t)
    outs = []
    for byte in (0x00, 0xFF, 0x9C, 0x7F):
        b.c.K.fill_(byte)
        b.c.V.fill_(byte)
        b.c.lens.zero_()
        b.c.append(b.layer, b.old_k.to(b.dt).cuda(), b.old_v.to(b.dt).cuda(), ints(b.old))
        b.c.lens.copy_(ints(b.lens))
        b.c.append(b.layer, b.k.to(b.dt).cuda(), b.v.to(b.dt).cuda(), b.offsets)
        outs.append(b.run(max_chunk=chunk))
    assert not outs[0].isnan().any()
    assert all(torch.equal(o.view(torch.uint8), outs[0].view(torch.uint8)) for o in outs)
