"""The serving entry points (emitted tokens, log probabilities, cache, attention)
reject bad arguments on the host before anything is enqueued.  No GPU needed: every
call here fails validation, with addresses that nothing reads."""
import ctypes

import pytest

ERR_ARG, ERR_SHAPE, ERR_DTYPE, ERR_WS, ERR_RANGE = -1, -2, -3, -4, -5
P = 0x10000  # aligned, never read


@pytest.fixture(scope="module")
def D():
    import os
    from draft_sampling_verification_w1_amd import dspark
    if not os.path.exists(dspark.LIB_PATH):
        from draft_sampling_verification_w1_amd import build
        build.build()
    return dspark


def cache(D, **kw):
    d = dict(slots=8, max_pages=16, pages=64, page_size=16, layers=2, kv_heads=2, head_dim=128, dtype=1)
    d.update(kw)
    return D.Cache(*d.values())


def tables(D, **kw):
    return D.CacheTables(*(kw.get(n, P) for n in ("table", "lens", "held", "refs", "free_bits", "n_free")))


def refused(D, code, status):
    assert status == code
    assert D.lib().dspark_last_error()


def test_emitted_tokens(D):
    f = D.lib().dspark_emitted_tokens
    for R, gamma in ((0, 4), (65537, 4), (1, 0), (1, 65), (-1, -1)):
        refused(D, ERR_SHAPE, f(R, gamma, P, P, P, P, None))
    for i in range(4):
        refused(D, ERR_ARG, f(2, 4, *[None if i == j else P for j in range(4)], None))


def test_token_logprobs(D):
    L = D.lib()
    f = L.dspark_token_logprobs

    def call(dtype=1, N=4, V=100000, ld=100000, logits=P, ids=P, top=2, lp=P, h=P, ti=P, tl=P, ws=P,
             nb=1 << 30):
        return f(dtype, N, V, ld, logits, ids, top, lp, h, ti, tl, ws, nb, None)

    refused(D, ERR_DTYPE, call(dtype=2))
    for kw in (dict(N=0), dict(N=2 ** 24 + 1), dict(V=0), dict(V=2 ** 26, ld=2 ** 26), dict(top=-1),
               dict(top=65), dict(ld=99999)):
        refused(D, ERR_SHAPE, call(**kw))
    for name in ("logits", "ids", "lp", "h", "ti", "tl"):
        refused(D, ERR_ARG, call(**{name: None}))
    refused(D, ERR_ARG, call(logits=P + 1))
    refused(D, ERR_ARG, call(dtype=0, logits=P + 2))
    need = L.dspark_logprobs_workspace_bytes(4, 100000, 2)
    assert need > 0
    for kw in (dict(ws=None), dict(ws=P + 16), dict(nb=need - 1)):
        refused(D, ERR_WS, call(**kw))
    assert L.dspark_logprobs_workspace_bytes(1 << 20, 4096, 2) == 0  # whole rows
    for args in ((0, 10, 0), (1, 0, 0), (1, 10, 65), (1, 1 << 26, 0)):
        assert L.dspark_logprobs_workspace_bytes(*args) == 0


CACHES = [(dict(slots=0), ERR_SHAPE), (dict(slots=4097), ERR_SHAPE), (dict(pages=0), ERR_SHAPE),
          (dict(pages=2 ** 24 + 1), ERR_SHAPE), (dict(page_size=8), ERR_SHAPE), (dict(page_size=48), ERR_SHAPE),
          (dict(page_size=512), ERR_SHAPE), (dict(max_pages=0), ERR_SHAPE), (dict(max_pages=2 ** 20 + 1), ERR_SHAPE),
          (dict(slots=2048, max_pages=2 ** 20), ERR_SHAPE), (dict(max_pages=2 ** 20, page_size=256, slots=1, pages=9),
                                                             None),
          (dict(layers=0), ERR_SHAPE), (dict(layers=1025), ERR_SHAPE), (dict(kv_heads=0), ERR_SHAPE),
          (dict(kv_heads=1025), ERR_SHAPE), (dict(head_dim=96), ERR_SHAPE), (dict(dtype=3), ERR_DTYPE)]


@pytest.mark.parametrize("kw,code", CACHES)
def test_cache_shapes(D, kw, code):
    L = D.lib()
    c, t = ctypes.byref(cache(D, **kw)), ctypes.byref(tables(D))
    if code is None:  # the widest table that is allowed
        assert L.dspark_cache_compact_workspace_bytes(c) > 0
        return
    refused(D, code, L.dspark_cache_init(c, t, None))
    refused(D, code, L.dspark_cache_fork(c, t, 1, P, P, P, None))
    refused(D, code, L.dspark_cache_reserve(c, t, P, P, P, P, None))
    refused(D, code, L.dspark_cache_commit(c, t, P, 1, None))
    refused(D, code, L.dspark_cache_free(c, t, 1, P, None))
    refused(D, code, L.dspark_cache_compact(c, t, t, P, P, P, P, 1 << 30, None))
    refused(D, code, L.dspark_cache_copy_pages(c, P, P, 1, P, P, None, None))
    refused(D, code, L.dspark_cache_append(c, t, 0, P, P, 1, P, P, P, None))
    refused(D, code, L.dspark_attend(c, t, 0, P, P, 1, 4, P, P, 0.1, 1, P, P, 1 << 30, None))
    assert L.dspark_cache_compact_workspace_bytes(c) == 0
    assert L.dspark_attend_workspace_bytes(c, 1, 4) == 0


def test_cache_null(D):
    L = D.lib()
    t = ctypes.byref(tables(D))
    refused(D, ERR_ARG, L.dspark_cache_init(None, t, None))
    refused(D, ERR_ARG, L.dspark_attend(None, t, 0, P, P, 1, 4, P, P, 0.1, 1, P, P, 1 << 30, None))
    assert L.dspark_attend_workspace_bytes(None, 1, 4) == 0


@pytest.mark.parametrize("name", ["table", "lens", "held", "refs", "free_bits", "n_free"])
@pytest.mark.parametrize("value", [None, P + 2])
def test_cache_tables(D, name, value):
    L = D.lib()
    c, t, good = ctypes.byref(cache(D)), ctypes.byref(tables(D, **{name: value})), ctypes.byref(tables(D))
    refused(D, ERR_ARG, L.dspark_cache_init(c, t, None))
    refused(D, ERR_ARG, L.dspark_cache_fork(c, t, 1, P, P, P, None))
    refused(D, ERR_ARG, L.dspark_cache_reserve(c, t, P, P, P, P, None))
    refused(D, ERR_ARG, L.dspark_cache_commit(c, t, P, 1, None))
    refused(D, ERR_ARG, L.dspark_cache_free(c, t, 1, P, None))
    refused(D, ERR_ARG, L.dspark_cache_compact(c, t, good, P, P, P, P, 1 << 30, None))
    refused(D, ERR_ARG, L.dspark_cache_compact(c, good, t, P, P, P, P, 1 << 30, None))
    refused(D, ERR_ARG, L.dspark_cache_append(c, t, 0, P, P, 1, P, P, P, None))
    refused(D, ERR_ARG, L.dspark_attend(c, t, 0, P, P, 1, 4, P, P, 0.1, 1, P, P, 1 << 30, None))


def test_bookkeeping_arguments(D):
    L = D.lib()
    c, t = ctypes.byref(cache(D)), ctypes.byref(tables(D))
    for n in (0, -1, 4097):
        refused(D, ERR_SHAPE, L.dspark_cache_fork(c, t, n, P, P, P, None))
        refused(D, ERR_SHAPE, L.dspark_cache_free(c, t, n, P, None))
    for n in (0, 2 ** 24 + 1):
        refused(D, ERR_SHAPE, L.dspark_cache_copy_pages(c, P, P, n, P, P, None, None))
    for i in range(3):
        refused(D, ERR_ARG, L.dspark_cache_fork(c, t, 1, *[None if i == j else P for j in range(3)], None))
        refused(D, ERR_ARG, L.dspark_cache_compact(c, t, t, *[None if i == j else P for j in range(3)], P,
                                                   1 << 30, None))
    for i in range(4):
        ps = [None if i == j else P for j in range(4)]
        refused(D, ERR_ARG, L.dspark_cache_reserve(c, t, *ps, None))
        refused(D, ERR_ARG, L.dspark_cache_copy_pages(c, ps[0], ps[1], 1, ps[2], ps[3], None, None))
    refused(D, ERR_ARG, L.dspark_cache_copy_pages(c, P + 8, P, 1, P, P, None, None))
    refused(D, ERR_ARG, L.dspark_cache_copy_pages(c, P, P + 8, 1, P, P, None, None))
    refused(D, ERR_ARG, L.dspark_cache_commit(c, t, None, 1, None))
    refused(D, ERR_ARG, L.dspark_cache_free(c, t, 1, None, None))
    need = L.dspark_cache_compact_workspace_bytes(c)
    for ws, nb in ((None, need), (P + 16, need), (P, need - 1)):
        refused(D, ERR_WS, L.dspark_cache_compact(c, t, t, P, P, P, ws, nb, None))


def test_append_and_attend_arguments(D):
    L = D.lib()
    c, t = ctypes.byref(cache(D)), ctypes.byref(tables(D))
    need = L.dspark_attend_workspace_bytes(c, 40, 4)
    assert need > 0

    def append(layer=0, K=P, V=P, N=40, k=P, v=P, off=P):
        return L.dspark_cache_append(c, t, layer, K, V, N, k, v, off, None)

    def attend(layer=0, K=P, V=P, N=40, heads=4, q=P, off=P, scale=0.1, chunk=5, out=P, ws=P, nb=need):
        return L.dspark_attend(c, t, layer, K, V, N, heads, q, off, scale, chunk, out, ws, nb, None)

    for layer in (-1, 2):
        refused(D, ERR_RANGE, append(layer=layer))
        refused(D, ERR_RANGE, attend(layer=layer))
    for n in (0, -5, 2 ** 22 + 1):
        refused(D, ERR_SHAPE, append(N=n))
        refused(D, ERR_SHAPE, attend(N=n))
        assert L.dspark_attend_workspace_bytes(c, n, 4) == 0
    for heads in (0, 3, 2 ** 26):
        refused(D, ERR_SHAPE, attend(heads=heads))
        assert L.dspark_attend_workspace_bytes(c, 40, heads) == 0
    refused(D, ERR_SHAPE, attend(chunk=0))
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        refused(D, ERR_RANGE, attend(scale=scale))
    for name in ("K", "V"):
        for value in (None, P + 8):
            refused(D, ERR_ARG, append(**{name: value}))
            refused(D, ERR_ARG, attend(**{name: value}))
    for value in (None, P + 8):
        refused(D, ERR_ARG, append(k=value))
        refused(D, ERR_ARG, append(v=value))
        refused(D, ERR_ARG, attend(q=value))
        refused(D, ERR_ARG, attend(out=value))
    refused(D, ERR_ARG, append(off=None))
    refused(D, ERR_ARG, attend(off=None))
    for kw in (dict(ws=None), dict(ws=P + 16), dict(nb=need - 1)):
        refused(D, ERR_WS, attend(**kw))
    for off in (0, 16, 40 * 4 * 128 * 2 - 16):  # out over q
        refused(D, ERR_ARG, attend(q=P + off))
        refused(D, ERR_ARG, attend(out=P + off))


def test_binding_refuses_cpu_tensors(D):
    import torch
    from draft_sampling_verification_w1_amd.cache import PagedCache, table_shapes
    K = torch.zeros((1, 4, 2, 8, 16, 8), dtype=torch.bfloat16)
    V = torch.zeros((1, 4, 2, 2, 64, 8), dtype=torch.bfloat16)
    t = {n: torch.zeros(s, dtype=torch.int32) for n, s in table_shapes(2, 2, 4).items()}
    with pytest.raises(ValueError, match="GPU"):
        PagedCache.of(K, V, **t)
    with pytest.raises(ValueError):
        PagedCache.of(K[0], V, **t)
    with pytest.raises(ValueError):
        PagedCache.of(K.half(), V, **t)
    with pytest.raises(ValueError):
        PagedCache(2, 2, 4, 16, 1, 2, 64, torch.float16, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        D.token_logprobs(torch.zeros((2, 8)), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        D.emitted_tokens(torch.zeros((2, 4), dtype=torch.int32), None, None)
