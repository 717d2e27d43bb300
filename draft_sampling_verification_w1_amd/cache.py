"""Paged key/value cache over the C ABI (include/dspark.h): what the target's
verify forward pass keeps between rounds.  A round reserves pages for the chunk
that it verifies, appends the chunk's keys and values layer by layer, attends over
them, and commits the accepted tokens; slots fork, roll back and are freed without
the host learning a length.  Summary page §5.3 (the verify batch is flattened over
requests of different verify lengths).

A cache may hold its keys and values in 4 bits (dtype torch.float4_e2m1fn_x2): a quarter of
the bytes that attention reads and that a token takes.  append then converts, read gives back
what the codes stand for.

Argument marshalling only: every step runs in the HIP library.
"""
from __future__ import annotations

import ctypes

import torch

from . import dspark

FOUR_BITS = torch.float4_e2m1fn_x2
_TYPES = {**dspark._DTYPES, FOUR_BITS: dspark.MXFP4}
TABLES = ("table", "lens", "held", "refs", "free_bits", "n_free")


def table_shapes(slots: int, max_pages: int, pages: int) -> dict:
    """Shapes of the int32 tables of a cache."""
    return {"table": (slots, max_pages), "lens": (slots,), "held": (slots,), "refs": (pages,),
            "free_bits": ((pages + 31) // 32,), "n_free": (1,)}


def rope_frequencies(dim: int, base: float = 10000.0, device="cuda"):
    """Radians per position of the dim / 2 pairs: base^(-2 j / dim), float64."""
    return base ** (torch.arange(0, dim, 2, dtype=torch.float64, device=device) / -dim)


class Rotation:
    """Rotation of keys and queries by their positions (dspark_rotation): freqs [dim / 2]
    float64, radians per position, the first dim elements of a head rotate; pairs are (j,
    j + dim / 2), or (2 j, 2 j + 1) if interleaved."""

    def __init__(self, freqs, interleaved: bool = False):
        if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
            raise ValueError("freqs must be a 1-dimensional float64 tensor")
        dspark._need(freqs, "freqs", dtype=torch.float64)
        self.freqs, self.interleaved, self.dim = freqs, bool(interleaved), 2 * freqs.numel()
        self._index = freqs.get_device()
        self._r = dspark.CacheRotation(freqs.data_ptr(), self.dim, int(self.interleaved))
        self._p = ctypes.byref(self._r)


class PagedCache:
    """A pool of pages and the tables of its slots.

    K [layers, pages, kv_heads, head_dim / E, page_size, E] and V [layers, pages,
    kv_heads, page_size / E, head_dim, E] (E = 16 bytes of elements) hold the tokens, in 4 bits
    K and V [layers, pages, bytes of a page] uint8 (laid out as in dspark.h);
    table, lens, held, refs, free_bits and n_free say which page is whose.  Calls go
    to the current stream of the cache's device."""

    def __init__(self, slots: int, max_pages: int, pages: int, page_size: int, layers: int,
                 kv_heads: int, head_dim: int, dtype=torch.bfloat16, device="cuda"):
        if dtype not in _TYPES:
            raise ValueError(f"dtype must be float32, bfloat16 or float4_e2m1fn_x2, got {dtype}")
        shape = None
        if dtype == FOUR_BITS:
            shape = (page_size, kv_heads, head_dim)
            K, V = (torch.empty((layers, pages, kv_heads * page_size * head_dim * 17 // 32), dtype=torch.uint8,
                                device=device) for _ in range(2))
        else:
            e = 16 // dtype.itemsize
            K = torch.empty((layers, pages, kv_heads, head_dim // e, page_size, e), dtype=dtype, device=device)
            V = torch.empty((layers, pages, kv_heads, page_size // e, head_dim, e), dtype=dtype, device=device)
        tables = {n: torch.empty(s, dtype=torch.int32, device=device)
                  for n, s in table_shapes(slots, max_pages, pages).items()}
        self._adopt(K, V, tables, shape)
        self.clear()

    @classmethod
    def of(cls, K, V, table, lens, held, refs, free_bits, n_free, shape=None):
        """A cache over tensors that exist already (laid out as the class says).  shape: of a
        4-bit cache (page_size, kv_heads, head_dim), which its bytes do not show."""
        self = cls.__new__(cls)
        self._adopt(K, V, dict(zip(TABLES, (table, lens, held, refs, free_bits, n_free))), shape)
        return self

    def _adopt(self, K, V, tables, shape):
        if shape is not None:
            page, heads, dim = shape
            if not isinstance(K, torch.Tensor) or K.dim() != 3 or K.dtype != torch.uint8:
                raise ValueError("K of a 4-bit cache must be a 3-dimensional uint8 tensor")
            layers, pages, held = K.shape
            if held * 32 != heads * page * dim * 17:
                raise ValueError(f"K's last dimension must be {heads * page * dim * 17 // 32}, got {held}")
            dtype = FOUR_BITS
            dspark._need(K, "K")
            dspark._need(V, "V", dtype=torch.uint8, shape=K.shape)
        else:
            if not isinstance(K, torch.Tensor) or K.dim() != 6 or K.dtype not in dspark._DTYPES:
                raise ValueError("K must be a 6-dimensional float32 or bfloat16 tensor")
            layers, pages, heads, chunks, page, e = K.shape
            if e != 16 // K.dtype.itemsize:
                raise ValueError(f"K's last dimension must be {16 // K.dtype.itemsize}, got {e}")
            dim, dtype = chunks * e, K.dtype
            dspark._need(K, "K")
            dspark._need(V, "V", dtype=K.dtype, shape=(layers, pages, heads, page // e, dim, e))
        if not isinstance(tables["table"], torch.Tensor) or tables["table"].dim() != 2:
            raise ValueError("table must have shape [slots, max_pages]")
        slots, max_pages = tables["table"].shape
        self._shapes = table_shapes(slots, max_pages, pages)
        self.K, self.V, self.device = K, V, K.device
        self.slots, self.max_pages, self.pages, self.page_size = slots, max_pages, pages, page
        self.layers, self.kv_heads, self.head_dim, self.dtype = layers, heads, dim, dtype
        self._index = K.get_device()
        self._tables = self._table_ptrs(tables)
        self._t = ctypes.byref(self._tables)
        for n in TABLES:
            setattr(self, n, tables[n])
        self._c = dspark.Cache(slots, max_pages, pages, page, layers, heads, dim, _TYPES[dtype])
        self._p = ctypes.byref(self._c)
        if dspark.lib().dspark_cache_compact_workspace_bytes(self._p) == 0:
            dspark._check(-2)

    def _table_ptrs(self, tables):
        for n in TABLES:
            self._need(tables[n], n, torch.int32, self._shapes[n])
        return dspark.CacheTables(*(tables[n].data_ptr() for n in TABLES))

    def _need(self, t, name, dtype, shape):
        dspark._need_on(self._index, t, name, dtype, shape)

    def _ints(self, *shape):
        return torch.empty(shape, dtype=torch.int32, device=self.device)

    def tables(self) -> dict:
        return {n: getattr(self, n) for n in TABLES}

    def _call(self, fn, *args):
        dspark._call_on(self._index, fn, self._p, *args)

    def clear(self):
        """Empty tables (dspark_cache_init)."""
        self._call(dspark.lib().dspark_cache_init, self._t)

    def fork(self, src, dst):
        """Slots dst [n] get the tokens of slots src [n] by sharing the pages that hold
        them, not those reserved behind (dspark_cache_fork).  Returns status [n] (1: the pair was refused)."""
        n = src.numel()
        self._need(src, "src", torch.int32, (n,))
        self._need(dst, "dst", torch.int32, (n,))
        status = self._ints(n)
        self._call(dspark.lib().dspark_cache_fork, self._t, n, src.data_ptr(),
                   dst.data_ptr(), status.data_ptr())
        return status

    def reserve(self, add, out=None):
        """Pages for add [slots] more tokens (dspark_cache_reserve), with the copies
        of shared pages that it asks for made in every layer.  Returns a dict of
        status, cow_src and cow_dst [slots]; ``out`` may supply it."""
        self._need(add, "add", torch.int32, (self.slots,))
        if out is None:
            out = dict(zip(("status", "cow_src", "cow_dst"), self._ints(3, self.slots).unbind(0)))
        else:
            for name in ("status", "cow_src", "cow_dst"):
                self._need(out[name], name, torch.int32, (self.slots,))
        self._call(dspark.lib().dspark_cache_reserve, self._t, add.data_ptr(),
                   out["status"].data_ptr(), out["cow_src"].data_ptr(), out["cow_dst"].data_ptr())
        self._copy(self.slots, out["cow_src"], out["cow_dst"], None)
        return out

    def commit(self, keep, plus: int = 0):
        """lens += keep + plus, pages behind the new lengths released
        (dspark_cache_commit)."""
        self._need(keep, "keep", torch.int32, (self.slots,))
        self._call(dspark.lib().dspark_cache_commit, self._t, keep.data_ptr(), plus)

    def free(self, slots):
        """Releases the listed slots (dspark_cache_free)."""
        n = slots.numel()
        self._need(slots, "slots", torch.int32, (n,))
        self._call(dspark.lib().dspark_cache_free, self._t, n, slots.data_ptr())

    def copy_pages(self, src, dst, count=None):
        """Copies pages src [n] to dst [n] in every layer (dspark_cache_copy_pages);
        count: device int32 [1], the pairs that count."""
        n = src.numel()
        self._need(src, "src", torch.int32, (n,))
        self._need(dst, "dst", torch.int32, (n,))
        if count is not None:
            self._need(count, "count", torch.int32, (1,))
        self._copy(n, src, dst, count)

    def _copy(self, n, src, dst, count):
        self._call(dspark.lib().dspark_cache_copy_pages, self.K.data_ptr(), self.V.data_ptr(), n,
                   src.data_ptr(), dst.data_ptr(), None if count is None else count.data_ptr())

    def compact(self, into=None, ws=None):
        """Moves the used pages to the front of the pool (dspark_cache_compact) and
        copies them.  ``into``: a dict of other tables that receive the new state, while
        this cache's own stay valid for rounds in flight; by default its own change.
        Returns a dict of the moves: src, dst [pages], n_moves [1]."""
        new = self._t if into is None else ctypes.byref(self._table_ptrs(into))
        if ws is None:
            n = dspark.lib().dspark_cache_compact_workspace_bytes(self._p)
            ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        src, dst = self._ints(2, self.pages).unbind(0)
        out = {"src": src, "dst": dst, "n_moves": self._ints(1)}
        self._call(dspark.lib().dspark_cache_compact, self._t, new,
                   out["src"].data_ptr(), out["dst"].data_ptr(), out["n_moves"].data_ptr(),
                   *dspark._ws_on(self._index, ws))
        self._copy(self.pages, src, dst, out["n_moves"])
        return out

    def _row_type(self, t, name):
        """The type of token rows: the cache's, or the given tensor's beside 4 bits."""
        if self.dtype != FOUR_BITS:
            return self.dtype
        if not isinstance(t, torch.Tensor) or t.dtype not in dspark._DTYPES:
            raise ValueError(f"{name} must be a float32 or bfloat16 tensor")
        return t.dtype

    def append(self, layer: int, k, v, offsets, rotation: Rotation | None = None, q=None, q_out=None):
        """Writes a chunk's keys and values into the pages: k, v [N, kv_heads, head_dim],
        slot s has rows offsets[s] .. offsets[s + 1] - 1.  With a rotation the keys, and
        queries q [N, heads, head_dim] if given, are rotated by their positions on the way
        (dspark_cache_store); the rotated queries are returned, in q_out if given, which may be q.
        A 4-bit cache takes float32 or bfloat16 rows.  Without a rotation, and for a
        cache of whole elements, the call is dspark_cache_append."""
        N = k.shape[0]
        dt = self._row_type(k, "k")
        self._need(k, "k", dt, (N, self.kv_heads, self.head_dim))
        self._need(v, "v", dt, (N, self.kv_heads, self.head_dim))
        self._need(offsets, "offsets", torch.int32, (self.slots + 1,))
        if rotation is None and q is None and q_out is None and self.dtype != FOUR_BITS:
            self._call(dspark.lib().dspark_cache_append, self._t, layer, self.K.data_ptr(),
                       self.V.data_ptr(), N, k.data_ptr(), v.data_ptr(), offsets.data_ptr())
            return None
        heads, turn = 0, None
        if q is None and q_out is not None:
            raise ValueError("q_out needs q")
        if rotation is not None:
            if rotation._index != self._index:
                raise ValueError(f"rotation must be on device {self._index}, got {rotation.freqs.device}")
            turn = rotation._p
        if q is not None:
            if rotation is None:
                raise ValueError("q needs a rotation")
            heads = q.shape[1]
            self._need(q, "q", dt, (N, heads, self.head_dim))
            if q_out is None:
                q_out = torch.empty_like(q)
            else:
                self._need(q_out, "q_out", dt, q.shape)
        self._call(dspark.lib().dspark_cache_store, self._t, layer, self.K.data_ptr(), self.V.data_ptr(), N,
                   dspark._DTYPES[dt], k.data_ptr(), v.data_ptr(), offsets.data_ptr(), turn, heads,
                   q.data_ptr() if heads else None, q_out.data_ptr() if heads else None)
        return q_out

    def read(self, layer: int, offsets, first=None, out=None, N: int | None = None, dtype=None):
        """Tokens out of the pages as dense rows (dspark_cache_read): rows offsets[s] ..
        offsets[s + 1] - 1 of k and v [N, kv_heads, head_dim] are slot s's tokens from position
        first[s] on (first [slots] int32; by default lens, the chunk behind the committed tokens).
        Returns (k, v), or ``out``; without it N rows of dtype (the cache's, bfloat16 of a 4-bit
        cache)."""
        if out is None:
            if N is None:
                raise ValueError("read needs out or N")
            if dtype is None:
                dtype = torch.bfloat16 if self.dtype == FOUR_BITS else self.dtype
            # rows behind the last token are nobody's
            out = tuple(torch.zeros((N, self.kv_heads, self.head_dim), dtype=dtype, device=self.device)
                        for _ in range(2))
        k, v = out
        N, dt = k.shape[0], self._row_type(k, "k")
        self._need(k, "k", dt, (N, self.kv_heads, self.head_dim))
        self._need(v, "v", dt, (N, self.kv_heads, self.head_dim))
        self._need(offsets, "offsets", torch.int32, (self.slots + 1,))
        if first is not None:
            self._need(first, "first", torch.int32, (self.slots,))
        self._call(dspark.lib().dspark_cache_read, self._t, layer, self.K.data_ptr(), self.V.data_ptr(), N,
                   dspark._DTYPES[dt], offsets.data_ptr(), None if first is None else first.data_ptr(),
                   k.data_ptr(), v.data_ptr())
        return out

    def attend_workspace(self, N: int, heads: int):
        """Workspace of attend for N rows of q."""
        n = dspark.lib().dspark_attend_workspace_bytes(self._p, N, heads)
        if n == 0:
            dspark._check(-2)
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def attend(self, layer: int, q, offsets, scale: float | None = None,
               max_chunk: int | None = None, out=None, ws=None):
        """Attention of the chunk's tokens over their slots' pages (dspark_attend, of a 4-bit
        cache dspark_attend4).  q [N, heads, head_dim]; scale: 1 / sqrt(head_dim) by default; max_chunk: the
        longest chunk expected (N by default).  Rows behind offsets[slots] of ``out``
        are left as they were."""
        N, heads = q.shape[0], q.shape[1]
        dt = self._row_type(q, "q")
        self._need(q, "q", dt, (N, heads, self.head_dim))
        self._need(offsets, "offsets", torch.int32, (self.slots + 1,))
        if out is None:
            out = torch.empty_like(q)
        else:
            self._need(out, "out", dt, q.shape)
        if ws is None:
            ws = self.attend_workspace(N, heads)
        fn, own = dspark.lib().dspark_attend, ()
        if self.dtype == FOUR_BITS:
            fn, own = dspark.lib().dspark_attend4, (dspark._DTYPES[dt],)
        self._call(fn, self._t, layer, self.K.data_ptr(),
                   self.V.data_ptr(), N, heads, *own, q.data_ptr(), offsets.data_ptr(),
                   self.head_dim ** -0.5 if scale is None else scale, N if max_chunk is None else max_chunk,
                   out.data_ptr(), *dspark._ws_on(self._index, ws))
        return out
