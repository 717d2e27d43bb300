"""Token log probabilities (dspark_token_logprobs) of logits that lie at the ends of their
types, at zero, and tied, against binary64 with the bounds of test_gpu_logprobs.py.  The
reference takes the row's maximum off first (exact or far below a bound here), as a sum of
1e10 and a logarithm would lose more in binary64 than the bounds allow.  The bounds hold
for far logits too: a difference z - m that matters there is exact, and its product with
log2 e is rounded once, as the fma elsewhere is."""
import math

import numpy as np
import pytest

from test_gpu_logprobs import check, dev, reference  # noqa: F401

pytestmark = pytest.mark.gpu

# whole rows, rows shared by several workgroups, many short rows
SHAPES = [(3, 20011), (3, 40009), (2051, 300)]


def expect(z, ids, n_top):
    z = z.double().numpy()
    m = z.max(1, keepdims=True)
    r = reference(z - np.where(np.isfinite(m), m, 0.0), ids.numpy(), n_top)
    for name in ("logprob", "top_logprobs"):
        # from here on a difference rounds to -inf in binary32
        r[name] = np.where(r[name] <= -2.0 ** 128 * (1 - 2.0 ** -25), -np.inf, r[name])
    return r


def rand(N, V, seed, scale=4.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return torch.randn((N, V), generator=g) * scale, torch.randint(0, V, (N,), generator=g).to(torch.int32), g


def dtype_of(name):
    import torch
    return torch.float32 if name == "f32" else torch.bfloat16


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mask", [-1e6, -1e10, -1e20, -1e30, "lowest bf16", "lowest"])
@pytest.mark.parametrize("N,V", SHAPES)
@pytest.mark.parametrize("n_top", [0, 20])
def test_finite_masks(dev, dtype, mask, N, V, n_top):  # noqa: F811
    """Masked entries that are finite: whole threads' first entries, nearly all of a row,
    a whole row (then a uniform distribution)."""
    import torch
    dt = dtype_of(dtype)
    value = {"lowest": torch.finfo(dt).min, "lowest bf16": torch.finfo(torch.bfloat16).min}.get(mask, mask)
    z, ids, g = rand(N, V, 3)
    z[0, :V * 2 // 3] = value
    z[1, torch.rand(V, generator=g) < 0.99] = value
    z[2] = value
    if N > 3:
        z[torch.rand((N, V), generator=g) < 0.5] = value
    ids[0], ids[2] = V - 1, V // 2
    z = z.to(dt)
    check(dev.token_logprobs(z.cuda(), ids.cuda(), n_top), expect(z, ids, n_top))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift,scale", [(1e5, 4), (3e6, 4), (-3e6, 4), (1e7, 4), (1e10, 4096), (-1e10, 4096),
                                         (1e20, 0), (0, 1e6), (0, 1e10), (0, 1e30), (0, 5e37), (3.2e38, 0),
                                         (-3.2e38, 0)])
@pytest.mark.parametrize("N,V", SHAPES)
def test_far_logits(dev, dtype, shift, scale, N, V):  # noqa: F811
    z, ids, g = rand(N, V, 5, 1.0)
    z = (z * scale + shift).to(dtype_of(dtype))
    check(dev.token_logprobs(z.cuda(), ids.cuda(), 8), expect(z, ids, 8))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gone", [(5, 512), (1, 1), (3, 2049), (0, 1024), (7, 4100), (2, 16390)])
@pytest.mark.parametrize("N,V", [(2, 20000), (2, 57345)])
@pytest.mark.parametrize("n_top", [1, 4, 8, 20, 64])
def test_ties_over_waves(dev, dtype, gone, N, V, n_top):  # noqa: F811
    """All entries equal but for a masked range: the lowest tokens lie in several waves'
    shares.  The second row has few values, in no order."""
    import torch
    z, ids, g = rand(N, V, 9)
    z[0] = 1.5
    z[1] = torch.randint(-1, 2, (V,), generator=g).float()
    z[:, gone[0]:gone[1]] = -math.inf
    ids[:] = V - 1
    z = z.to(dtype_of(dtype))
    check(dev.token_logprobs(z.cuda(), ids.cuda(), n_top), expect(z, ids, n_top))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["zeros", "both zeros", "negative zeros", "largest is 0", "falls from 0", "tiny"])
@pytest.mark.parametrize("N,V", SHAPES + [(5, 7)])
@pytest.mark.parametrize("n_top", [1, 2, 3, 4, 5, 64])
def test_zero(dev, dtype, kind, N, V, n_top):  # noqa: F811
    """The n-th best entry is zero: the entries that equal it, of either sign, count."""
    import torch
    z, ids, g = rand(N, V, 7)
    if kind == "zeros":
        z = torch.zeros((N, V))
    elif kind == "both zeros":
        z = torch.where(torch.rand((N, V), generator=g) < 0.5, 0.0, -0.0)
    elif kind == "negative zeros":
        z = -torch.zeros((N, V))
    elif kind == "largest is 0":
        z -= z.amax(1, keepdim=True)
    elif kind == "falls from 0":
        z = -torch.arange(V).float().repeat(N, 1) / 64
    else:                        # below the smallest normal number, of both signs
        z = torch.randint(-3, 4, (N, V), generator=g).float() * 2.0 ** -130
    z = z.to(dtype_of(dtype))
    check(dev.token_logprobs(z.cuda(), ids.cuda(), n_top), expect(z, ids, n_top))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("what", [math.nan, -math.nan, math.inf])
@pytest.mark.parametrize("N,V", [(6, 20011), (6, 40009), (2051, 300), (6, 5)])
@pytest.mark.parametrize("n_top", [0, 3])
def test_rows_without_a_distribution(dev, dtype, what, N, V, n_top):  # noqa: F811
    """A NaN or +inf among the entries: NaN and no alternatives, the other rows as ever."""
    import torch
    z, ids, g = rand(N, V, 13)
    z[0, V - 1] = what
    z[1, 0] = what
    z[2, V // 2] = what
    z[3, ids[3].item()] = what
    z[3, :V // 3] = -math.inf
    z = z.to(dtype_of(dtype))
    none = ~(z < math.inf).all(1, keepdim=True)
    assert none[:3].all()
    want = expect(z.double().masked_fill(none, -math.inf), ids, n_top)
    check(dev.token_logprobs(z.cuda(), ids.cuda(), n_top), want)


def test_most_rows(dev):  # noqa: F811
    """As many rows as a call takes, of two entries.  The bounds of test_gpu_logprobs.py with
    |z - m| <= 6: (2 * 6 + 9) u, and (21 + (21 + 7) * 7) u for the entropy."""
    import torch
    N = 2 ** 24 - 1
    a = torch.arange(N, device="cuda")
    z = torch.stack([a % 5, (a + 3) % 7 - 2], 1).to(torch.bfloat16)
    got = dev.token_logprobs(z, (a % 2).to(torch.int32), 1)
    p = torch.log_softmax(z.double(), 1)
    best = (z[:, 1] > z[:, 0]).to(torch.int32)
    u = 2.0 ** -24
    assert torch.equal(got["top_ids"].view(-1), best)
    for name, want, tol in (("logprob", p.gather(1, (a % 2).view(-1, 1)), 21 * u),
                            ("top_logprobs", p.gather(1, best.long().view(-1, 1)), 21 * u),
                            ("entropy", -(p.exp() * p).sum(1, keepdim=True), 217 * u)):
        off = (got[name].double().view(-1, 1) - want).abs()
        assert (off <= tol + u * want.abs()).all(), name
