"""A plain model of the rotation and of the 4-bit pages (include/dspark.h) in numpy: element by
element, in the order of the definition."""
import numpy as np

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def rotate(x, pos, freqs, interleaved, exact=False):
    """Rows x [n, heads, d] at positions pos [n].  Binary32 as defined (c and s rounded, then every
    product and sum), or in binary64."""
    f = np.float64 if exact else np.float32
    dim = 2 * len(freqs)
    angle = np.asarray(pos, np.float64)[:, None] * np.asarray(freqs, np.float64)[None]
    c, s = np.cos(angle).astype(f)[:, None], np.sin(angle).astype(f)[:, None]
    out = np.array(x, f)
    a, b = (slice(0, dim, 2), slice(1, dim, 2)) if interleaved else (slice(0, dim // 2), slice(dim // 2, dim))
    xa, xb = out[..., a].copy(), out[..., b].copy()
    out[..., a] = xa * c - xb * s
    out[..., b] = xb * c + xa * s
    return out


def scale_bytes(x):
    """Of blocks of 32 elements x [..., d]: the smallest power of two of which the largest is at most 7."""
    top = np.abs(np.asarray(x, np.float64)).reshape(*x.shape[:-1], -1, 32).max(-1)
    m, e = np.frexp(top)
    e = np.where(m > 0.875, e - 2, e - 3)
    e = np.clip(np.where(top == 0, -120, e), -120, 125)
    return np.where(np.isfinite(top), e + 127, 255).astype(np.uint8)


def nearest(x, bytes_):
    """Signed places among LEVELS (code without its sign bit, sign apart) for given scale bytes."""
    y = np.abs(np.asarray(x, np.float64)) * np.repeat(np.exp2(127.0 - bytes_.astype(np.float64)), 32, -1)
    code = np.zeros(y.shape, np.uint8)
    for i in range(7):
        mid = (LEVELS[i] + LEVELS[i + 1]) / 2
        code = np.where(y >= mid if i % 2 else y > mid, i + 1, code)
    return code.astype(np.uint8)


def values(x, bytes_=None):
    """What 4 bits make of x [..., d] (finite), in binary64."""
    b = scale_bytes(x) if bytes_ is None else bytes_
    size = LEVELS[nearest(x, b)] * np.repeat(np.exp2(b.astype(np.float64) - 127), 32, -1)
    return np.where(np.asarray(x) < 0, -size, size)


def unpack(blob, name, heads, page, d):
    """A page's bytes as (signed values before scaling [page, heads, d], scale bytes [page, heads, d / 32])."""
    t, h, e = np.indices((page, heads, d))
    if name == "K":
        at = ((h * (d // 32) + e // 32) * page + t) * 16 + e % 32 // 2
    else:
        n, r = e // (d // 16), e % (d // 16)
        at = h * page * d // 2 + (((t // 8 * (d // 64) + r // 4) * 16 + n) * 2 + r % 4 // 2) * 8 + t % 8
    code = blob[at].astype(int) >> 4 * (e % 2) & 15
    t, h, b = np.indices((page, heads, d // 32))
    scales = blob[heads * page * d // 2 + (h * (d // 32) + b) * page + t]
    return np.where(code > 7, -LEVELS[code & 7], LEVELS[code & 7]), scales
