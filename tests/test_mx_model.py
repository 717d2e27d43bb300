"""The plain model of the 4-bit pages: closed forms, so that what the GPU tests compare with is pinned."""
import numpy as np
import pytest

import mx_model as M


def test_levels_are_kept():
    x = np.zeros((1, 32))
    x[0, :8], x[0, 8:16] = M.LEVELS * 4, -M.LEVELS * 4
    assert M.scale_bytes(x)[0, 0] == 127 + 2
    assert np.array_equal(M.values(x), x)


@pytest.mark.parametrize("top,e", [(7.0, 0), (7.000001, 1), (6.0, 0), (3.5, -1), (3.4999, -1), (3.5001, 0), (1.75, -2),
                                   (1e-40, -120), (0.0, -120), (3e38, 125)])
def test_scale_is_the_smallest(top, e):
    x = np.zeros((1, 32))
    x[0, 9] = -top
    assert M.scale_bytes(x)[0, 0] == 127 + e


def test_ties_go_to_even_codes():
    x = np.zeros((1, 32))
    x[0, :9] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 0.7500001]
    assert M.values(x)[0, :9].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 1]


def test_no_value_is_nearer():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 64)) * np.exp2(rng.integers(-20, 20, (200, 1)))
    b = M.scale_bytes(x)
    s = np.repeat(np.exp2(b.astype(float) - 127), 32, -1)
    every = np.concatenate([M.LEVELS, -M.LEVELS])[:, None, None] * s
    assert np.array_equal(np.abs(every - x).min(0), np.abs(M.values(x) - x))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_relative_positions(interleaved):
    """The product of a query at p and a key at q depends on p - q alone."""
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    f = 1e4 ** (-np.arange(0, 48, 2) / 48)
    dot = lambda p, r: float((M.rotate(q, [p], f, interleaved, True) * M.rotate(k, [r], f, interleaved, True)).sum())  # noqa: E731
    assert abs(dot(1000, 993) - dot(7, 0)) < 1e-10
    assert np.array_equal(M.rotate(q, [5], f, interleaved, True)[..., 48:], q[..., 48:])
    assert np.allclose(M.rotate(q, [0], f, interleaved), q.astype(np.float32), rtol=0, atol=0)
