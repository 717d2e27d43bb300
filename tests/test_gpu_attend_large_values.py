"""Chunk attention over values just inside what the contract allows (below 2^90): weighted sums stay inside binary32 before
they are divided, to the tolerances of test_gpu_attend.py and test_gpu_attend4.py, which go with the values' size."""
import pytest
import torch

import test_gpu_attend as TA
import test_gpu_attend4 as TQ
from test_gpu_attend4 import C, ints  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["whole", "4bit"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("chunk", [1, 17, 130])
@pytest.mark.parametrize("scale", [0.01, 1.0])
def test_large_values(C, kind, dtype, chunk, scale):  # noqa: F811
    b = (TA if kind == "whole" else TQ).Batch(C, dtype, 64, 8, 2, 128, [20000, 40], [chunk, 1])
    k, v = b.old_k.to(b.dt), (b.old_v * 2.0 ** 87).to(b.dt)
    assert float(v.abs().max()) < 2.0 ** 90
    b.c.lens.zero_()
    b.c.append(b.layer, k.cuda(), v.cuda(), ints(b.old))
    b.c.lens.copy_(ints(b.lens))
    b.old_v = torch.from_numpy(TQ.M.values(v.double().numpy())) if kind == "4bit" else v
    b.check(b.run(max_chunk=chunk, scale=scale), scale=scale)
