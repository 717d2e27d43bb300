"""dspark_cache_store, dspark_cache_read and dspark_attend4 reject bad arguments on the host before anything
is enqueued.  No GPU needed: every call here fails validation, with addresses that nothing reads."""
import ctypes

import pytest

from test_abi_serving import CACHES, D, ERR_ARG, ERR_DTYPE, ERR_RANGE, ERR_SHAPE, ERR_WS, P, cache, refused, tables  # noqa: F401


def rotation(D, freqs=P, dim=128, interleaved=0):  # noqa: F811
    return ctypes.byref(D.CacheRotation(freqs, dim, interleaved))


def test_four_bits_is_a_cache_type(D):  # noqa: F811
    L = D.lib()
    assert L.dspark_cache_compact_workspace_bytes(ctypes.byref(cache(D, dtype=2))) > 0
    assert L.dspark_attend_workspace_bytes(ctypes.byref(cache(D, dtype=2)), 40, 4) > 0
    # the calls for whole elements do not take it
    c, t = ctypes.byref(cache(D, dtype=2)), ctypes.byref(tables(D))
    refused(D, ERR_DTYPE, L.dspark_cache_append(c, t, 0, P, P, 1, P, P, P, None))
    refused(D, ERR_DTYPE, L.dspark_attend(c, t, 0, P, P, 1, 4, P, P, 0.1, 1, P, P, 1 << 30, None))


@pytest.mark.parametrize("kw,code", [x for x in CACHES if x[1] is not None])
def test_cache_shapes(D, kw, code):  # noqa: F811
    L = D.lib()
    c, t = ctypes.byref(cache(D, **{"dtype": 2, **kw})), ctypes.byref(tables(D))
    refused(D, code, L.dspark_cache_store(c, t, 0, P, P, 1, 1, P, P, P, None, 0, None, None, None))
    refused(D, code, L.dspark_cache_read(c, t, 0, P, P, 1, 1, P, None, P, P + (1 << 20), None))
    refused(D, code, L.dspark_attend4(c, t, 0, P, P, 1, 4, 1, P, P, 0.1, 1, P, P, 1 << 30, None))


@pytest.mark.parametrize("name", ["table", "lens", "held", "refs", "free_bits", "n_free"])
@pytest.mark.parametrize("value", [None, P + 2])
def test_cache_tables(D, name, value):  # noqa: F811
    L = D.lib()
    c, t = ctypes.byref(cache(D, dtype=2)), ctypes.byref(tables(D, **{name: value}))
    refused(D, ERR_ARG, L.dspark_cache_store(c, t, 0, P, P, 1, 1, P, P, P, None, 0, None, None, None))
    refused(D, ERR_ARG, L.dspark_cache_read(c, t, 0, P, P, 1, 1, P, None, P, P + (1 << 20), None))
    refused(D, ERR_ARG, L.dspark_attend4(c, t, 0, P, P, 1, 4, 1, P, P, 0.1, 1, P, P, 1 << 30, None))


@pytest.mark.parametrize("pool,dtype", [(2, 2), (2, -1), (0, 1), (1, 0), (1, 2)])
def test_row_types(D, pool, dtype):  # noqa: F811
    L = D.lib()
    c, t = ctypes.byref(cache(D, dtype=pool)), ctypes.byref(tables(D))
    refused(D, ERR_DTYPE, L.dspark_cache_store(c, t, 0, P, P, 1, dtype, P, P, P, None, 0, None, None, None))
    refused(D, ERR_DTYPE, L.dspark_cache_read(c, t, 0, P, P, 1, dtype, P, None, P, P + (1 << 20), None))
    refused(D, ERR_DTYPE, L.dspark_attend4(c, t, 0, P, P, 1, 4, dtype, P, P, 0.1, 1, P, P, 1 << 30, None))


def test_attend4_needs_four_bits(D):  # noqa: F811
    c, t = ctypes.byref(cache(D, dtype=1)), ctypes.byref(tables(D))
    refused(D, ERR_DTYPE, D.lib().dspark_attend4(c, t, 0, P, P, 1, 4, 1, P, P, 0.1, 1, P, P, 1 << 30, None))


@pytest.mark.parametrize("pool", [1, 2])
def test_store_arguments(D, pool):  # noqa: F811
    L = D.lib()
    c, t = ctypes.byref(cache(D, dtype=pool)), ctypes.byref(tables(D))
    far = P + (1 << 24)

    def store(layer=0, K=P, V=P, N=40, k=P, v=P, off=P, rot=None, heads=0, q=P, q_out=far):
        return L.dspark_cache_store(c, t, layer, K, V, N, 1, k, v, off, rot, heads, q, q_out, None)

    for layer in (-1, 2):
        refused(D, ERR_RANGE, store(layer=layer))
    for n in (0, -5, 2 ** 22 + 1):
        refused(D, ERR_SHAPE, store(N=n))
    for heads in (-2, 3, 2 ** 26):
        refused(D, ERR_SHAPE, store(heads=heads, rot=rotation(D)))
    for name in ("K", "V", "k", "v"):
        for value in (None, P + 8):
            refused(D, ERR_ARG, store(**{name: value}))
    refused(D, ERR_ARG, store(off=None))
    for dim in (0, -16, 8, 24, 144, 256):
        refused(D, ERR_SHAPE, store(rot=rotation(D, dim=dim)))
    for freqs in (None, P + 4):
        refused(D, ERR_ARG, store(rot=rotation(D, freqs=freqs)))
    for flag in (2, -1):
        refused(D, ERR_RANGE, store(rot=rotation(D, interleaved=flag)))
    refused(D, ERR_ARG, store(heads=4))  # queries without a rotation
    for name in ("q", "q_out"):
        for value in (None, P + 8):
            refused(D, ERR_ARG, store(heads=4, rot=rotation(D), **{name: value}))
    size = 40 * 4 * 128 * 2
    for off in (16, size - 16):
        refused(D, ERR_ARG, store(heads=4, rot=rotation(D), q=P, q_out=P + off))
        refused(D, ERR_ARG, store(heads=4, rot=rotation(D), q=P + off, q_out=P))


@pytest.mark.parametrize("pool", [1, 2])
@pytest.mark.parametrize("name", ["k", "v"])
def test_turned_queries_beside_keys_and_values(D, pool, name):  # noqa: F811
    """Turned queries [40, 8, 128] over keys or values [40, 2, 128] are refused: from the last byte of one to the
    first of the other."""
    L = D.lib()
    c, t = ctypes.byref(cache(D, dtype=pool)), ctypes.byref(tables(D))
    rows, queries = 40 * 2 * 128 * 2, 40 * 8 * 128 * 2
    out = P + (1 << 24)
    for at in (out, out + queries - 16, out - rows + 16):
        kv = {"k": P, "v": P, name: at}
        refused(D, ERR_ARG, L.dspark_cache_store(c, t, 0, P, P, 40, 1, kv["k"], kv["v"], P, rotation(D), 8, P, out, None))


@pytest.mark.parametrize("pool", [1, 2])
def test_read_arguments(D, pool):  # noqa: F811
    L = D.lib()
    c, t = ctypes.byref(cache(D, dtype=pool)), ctypes.byref(tables(D))
    far = P + (1 << 24)

    def read(layer=0, K=P, V=P, N=40, off=P, first=None, k=P, v=far):
        return L.dspark_cache_read(c, t, layer, K, V, N, 1, off, first, k, v, None)

    for layer in (-1, 2):
        refused(D, ERR_RANGE, read(layer=layer))
    for n in (-5, 2 ** 22 + 1):
        refused(D, ERR_SHAPE, read(N=n))
    assert read(N=0, off=None, k=None, v=None) == 0  # no rows: nothing to do
    refused(D, ERR_RANGE, read(N=0, layer=2))
    for name in ("K", "V", "k", "v"):
        for value in (None, P + 8):
            refused(D, ERR_ARG, read(**{name: value}))
    refused(D, ERR_ARG, read(off=None))
    size = 40 * 2 * 128 * 2
    for off in (0, 16, size - 16):
        refused(D, ERR_ARG, read(k=P, v=P + off))
        refused(D, ERR_ARG, read(k=P + off, v=P))


@pytest.mark.parametrize("dtype", [0, 1])
def test_attend4_arguments(D, dtype):  # noqa: F811
    L = D.lib()
    c, t = ctypes.byref(cache(D, dtype=2)), ctypes.byref(tables(D))
    need = L.dspark_attend_workspace_bytes(c, 40, 4)

    def attend(layer=0, K=P, V=P, N=40, heads=4, q=P, off=P, scale=0.1, chunk=5, out=P, ws=P, nb=need):
        return L.dspark_attend4(c, t, layer, K, V, N, heads, dtype, q, off, scale, chunk, out, ws, nb, None)

    for layer in (-1, 2):
        refused(D, ERR_RANGE, attend(layer=layer))
    for n in (0, -5, 2 ** 22 + 1):
        refused(D, ERR_SHAPE, attend(N=n))
    for heads in (0, 3, 2 ** 26):
        refused(D, ERR_SHAPE, attend(heads=heads))
    refused(D, ERR_SHAPE, attend(chunk=0))
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        refused(D, ERR_RANGE, attend(scale=scale))
    for name in ("K", "V", "q", "out"):
        for value in (None, P + 8):
            refused(D, ERR_ARG, attend(**{name: value}))
    refused(D, ERR_ARG, attend(off=None))
    for kw in (dict(ws=None), dict(ws=P + 16), dict(nb=0)):
        refused(D, ERR_WS, attend(**kw))
    for off in (0, 16, 40 * 4 * 128 * (2 if dtype else 4) - 16):  # out over q
        refused(D, ERR_ARG, attend(q=P + off))
        refused(D, ERR_ARG, attend(out=P + off))


def test_binding_refuses_cpu_tensors(D):  # noqa: F811
    import torch
    from draft_sampling_verification_w1_amd.cache import FOUR_BITS, PagedCache, Rotation, rope_frequencies, table_shapes
    t = {n: torch.zeros(s, dtype=torch.int32) for n, s in table_shapes(2, 2, 4).items()}
    pool = torch.zeros((1, 4, 16 * 2 * 64 * 17 // 32), dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        PagedCache.of(pool, pool, **t, shape=(16, 2, 64))
    with pytest.raises(ValueError, match="3-dimensional"):
        PagedCache.of(pool[0], pool, **t, shape=(16, 2, 64))
    with pytest.raises(ValueError, match="last dimension"):
        PagedCache.of(pool, pool, **t, shape=(32, 2, 64))
    with pytest.raises(ValueError, match="GPU"):
        PagedCache(2, 2, 4, 16, 1, 2, 64, FOUR_BITS, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        Rotation(rope_frequencies(64, device="cpu"))
