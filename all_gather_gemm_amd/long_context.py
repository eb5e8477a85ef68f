"""Long contexts over the paged key-value cache: Python binding of the functions of include/agmm_long.h
(libagmm.so).

`PrefixAttention` attends with one new token of every sequence where sequences share prefixes, which are
read once for every 128 rows (q heads of one kv head) of all that share one. `PageIndex` keeps bounds of every page's keys, and selects for each
sequence and kv head the pages whose score is highest; DecodeAttention.run takes the table that it makes.
`AttentionMass` adds up the weight that each cached token gets, `Evictor` keeps the tokens that got the
most and moves their rows together. As in all of the package's modules, arguments are marshalled only: tensors'
pointers and strides and torch's current stream (or `stream`, as all_gather_gemm_amd.attention describes)
go to the library's kernels, error codes come back as AgmmError, and there is no fallback path.

No gradient passes through these: they serve.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import lib
from .attention import (_DTYPES, _STORAGES, DecodeAttention, PagedCache, _checked, _empty, _like, _pick,
                        _stream, _tensor, ag_attn_desc, ag_kv_cache)

EXPORTED = [
    "ag_prefix_scratch_bytes", "ag_prefix_run", "ag_index_update", "ag_index_scratch_bytes",
    "ag_index_select", "ag_attn_run_heads", "ag_mass_add", "ag_evict_choose", "ag_evict_move",
]


class ag_page_index(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


def _declare():
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    cache, attn, index = (ctypes.POINTER(t) for t in (ag_kv_cache, ag_attn_desc, ag_page_index))
    lib.ag_prefix_scratch_bytes.argtypes = [attn, i64, i64]
    lib.ag_prefix_scratch_bytes.restype = i64
    lib.ag_prefix_run.argtypes = [vp, cache, vp, i64, i64, vp, i64, i64, vp, vp, i64, vp, i64, i64, vp, i64,
                                  vp, i64, i64, vp, vp, i64, vp]
    lib.ag_index_update.argtypes = [cache, index, vp, i64, i64, vp, vp, i64, vp]
    lib.ag_index_scratch_bytes.argtypes = [cache, i64, i64]
    lib.ag_index_scratch_bytes.restype = i64
    lib.ag_index_select.argtypes = [cache, index, vp, i64, i64, i64, vp, i64, i64, vp, i64, i64, i64, i64, vp,
                                    vp, vp, i64, vp]
    lib.ag_mass_add.argtypes = [attn, cache, vp, i64, i64, vp, vp, i64, i64, vp, i64, vp, i64, i64, vp, i64,
                                i64, i64, ctypes.c_float, vp]
    lib.ag_evict_choose.argtypes = [cache, vp, i64, i64, i64, vp, i64, i64, vp, i64, i64, i64, i64, vp, vp, vp,
                                    vp]
    lib.ag_evict_move.argtypes = [cache, vp, i64, i64, cache, vp, i64, i64, vp, i64, vp, i64, vp]


_declare()


# Arguments' checks are most of a small call's time: what is right is seen with few attributes, and whatever is not goes
# to attention._tensor, which says why.
def _is(t, name, dtype, shape, cache):
    """A tensor of this type and shape on the cache's GPU whose last dimension is dense."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == cache.index and t.stride(-1) == 1:
        return t
    return _tensor(t, name, dtype, shape, cache.device)


def _table(t, name, rows, cache):
    shape = t.shape
    if t.dtype is torch.int32 and len(shape) == 2 and shape[0] == rows and t.get_device() == cache.index and \
            t.stride(1) == 1:
        return t
    return _tensor(t, name, torch.int32, (rows, shape[1] if len(shape) == 2 else None), cache.device)


def _dense(t, name):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


class PrefixAttention(DecodeAttention):
    """Attention of one new token of every sequence over the prefix that its group shares and its own tokens.

    run(q, cache, prefix_table, prefix_lens, page_table, lens): q [batch, q_heads, head_dim]; prefix_table
    int32 [groups, pages] and prefix_lens int32 [groups]; page_table int32 [batch, pages] and lens int32
    [batch] of the sequences' own tokens, the new one counted in (no window). Group g has the sequences starts[g] to
    starts[g + 1] - 1 (starts int32 [groups + 1]); without starts there is one group, the whole batch.
    Returns out like q, or (out, lse) with lse float32 [batch, q_heads]. A handle serves one stream at a time."""

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, dtype: str = "bf16",
                 storage: str = "16bit", scale: float = 0.0, soft_cap: float = 0.0, num_wgs: int = 0):
        super().__init__(q_heads, kv_heads, head_dim, dtype=dtype, storage=storage, scale=scale,
                         soft_cap=soft_cap, num_wgs=num_wgs)
        self._scratch = {}

    def _scratch_bytes(self, batch, groups):
        n = self._scratch.get((batch, groups))
        if n is None:
            n = lib.ag_prefix_scratch_bytes(ctypes.byref(self.desc), batch, groups)
            _checked(min(n, 0), "ag_prefix_scratch_bytes")
            if len(self._scratch) >= 4096:
                self._scratch.clear()
            self._scratch[batch, groups] = n
        return n

    def run(self, q, cache: PagedCache, prefix_table, prefix_lens, page_table, lens, starts=None, out=None,
            return_lse: bool = False, stream=None):
        batch = q.shape[0]
        _is(q, "q", self.torch_dtype, (batch, self.q_heads, self.head_dim), cache)
        groups = prefix_lens.shape[0]
        _is(prefix_lens, "prefix_lens", torch.int32, (groups,), cache)
        _table(prefix_table, "prefix_table", groups, cache)
        _table(page_table, "page_table", batch, cache)
        _is(lens, "lens", torch.int32, (batch,), cache)
        if starts is not None:
            _is(starts, "starts", torch.int32, (groups + 1,), cache)
        elif groups != 1:
            raise ValueError("several groups need starts")
        where = _stream(stream, cache.index)
        if out is None:
            out = _like(q, stream)
        else:
            _is(out, "out", self.torch_dtype, q.shape, cache)
        lse = _empty(q, (batch, self.q_heads), torch.float32, stream) if return_lse else None
        n = self._scratch_bytes(batch, groups)
        scratch = _empty(q, (n,), torch.uint8, stream)
        qs, os = q.stride(), out.stride()
        rc = lib.ag_prefix_run(
            self.handle, cache._ref, q.data_ptr(), qs[0], qs[1], prefix_table.data_ptr(),
            prefix_table.stride(0), prefix_table.shape[1], prefix_lens.data_ptr(),
            None if starts is None else starts.data_ptr(), groups, page_table.data_ptr(), page_table.stride(0),
            page_table.shape[1], lens.data_ptr(), batch, out.data_ptr(), os[0], os[1],
            lse.data_ptr() if return_lse else None, scratch.data_ptr(), n, where)
        _checked(rc, "ag_prefix_run")
        return (out, lse) if return_lse else out


class PageIndex:
    """Bounds of the keys of a cache's pages, and the pages that they select (ag_page_index).

    codes int8 [pages, kv_heads, 2, head_dim]: for each element the largest of a page's keys and the least, in
    units of 2^(scale byte - 127), rounded outwards; scales uint8 [pages, kv_heads]. New ones are made
    where none are given."""

    def __init__(self, cache: PagedCache, codes=None, scales=None):
        pages = cache.desc.num_pages
        shape = (pages, cache.kv_heads, 2, cache.head_dim)
        if (codes is None) != (scales is None):
            raise ValueError("codes and scales are given both or neither")
        if codes is None:
            codes = torch.zeros(shape, dtype=torch.int8, device=cache.device)
            scales = torch.zeros(shape[:2], dtype=torch.uint8, device=cache.device)
        self.codes = _dense(_tensor(codes, "codes", torch.int8, shape, cache.device), "codes")
        self.scales = _dense(_tensor(scales, "scales", torch.uint8, shape[:2], cache.device), "scales")
        self.cache, self._scratch = cache, {}
        self.desc = ag_page_index(codes.data_ptr(), scales.data_ptr())
        self._ref = ctypes.byref(self.desc)

    def update(self, page_table, lens, starts=None, stream=None):
        """Makes the entries of the pages that hold tokens starts[b] (0 without starts) to lens[b] - 1 of
        the sequences of page_table int32 [batch, pages]; starts and lens int32 [batch]. A page in several of
        those places gets the entry of the one with the most of its tokens."""
        cache, batch = self.cache, lens.shape[0]
        _table(page_table, "page_table", batch, cache)
        _is(lens, "lens", torch.int32, (batch,), cache)
        if starts is not None:
            _is(starts, "starts", torch.int32, (batch,), cache)
        rc = lib.ag_index_update(cache._ref, self._ref, page_table.data_ptr(), page_table.stride(0),
                                 page_table.shape[1], None if starts is None else starts.data_ptr(),
                                 lens.data_ptr(), batch, _stream(stream, cache.index))
        _checked(rc, "ag_index_update")

    def select(self, q, page_table, lens, budget: int, sink: int = 1, recent: int = 2, stream=None):
        """(table, tokens): table int32 [batch, kv_heads, budget], the pages that the new tokens q [batch,
        q_heads, head_dim] attend to (the sequence's first `sink`, its last `recent`, and those with the
        highest scores), in order, and -1 behind them; tokens int32 [batch], how many they hold.
        DecodeAttention.run takes both as its page table and lengths."""
        cache, batch = self.cache, q.shape[0]
        _is(q, "q", cache.torch_dtype, (batch, q.shape[1] if q.dim() == 3 else None, cache.head_dim), cache)
        _table(page_table, "page_table", batch, cache)
        _is(lens, "lens", torch.int32, (batch,), cache)
        if budget < 1:
            raise ValueError("budget must be at least 1")
        where = _stream(stream, cache.index)
        pages = page_table.shape[1]
        n = self._scratch.get((batch, pages))
        if n is None:
            n = lib.ag_index_scratch_bytes(cache._ref, pages, batch)
            _checked(min(n, 0), "ag_index_scratch_bytes")
            if len(self._scratch) >= 4096:
                self._scratch.clear()
            self._scratch[batch, pages] = n
        scratch = _empty(q, (n,), torch.uint8, stream) if n else None
        table = _empty(lens, (batch, cache.kv_heads, budget), torch.int32, stream)
        tokens = _like(lens, stream)
        rc = lib.ag_index_select(cache._ref, self._ref, q.data_ptr(), q.stride(0), q.stride(1), q.shape[1],
                                 page_table.data_ptr(), page_table.stride(0), pages, lens.data_ptr(), batch,
                                 budget, sink, recent, table.data_ptr(), tokens.data_ptr(),
                                 scratch.data_ptr() if n else None, n, where)
        _checked(rc, "ag_index_select")
        return table, tokens


class AttentionMass:
    """Adds up the attention weight of cached tokens (ag_mass_add), for the geometry, scale, window and cap of
    a DecodeAttention.

    add(mass, q, lse, cache, page_table, lens) returns decay * mass plus, for each token, the softmax weights
    of the kv head's q heads: mass float32 [batch, kv_heads, tokens], q and lse [batch, q_heads] as the attention
    took and gave them, over one page table for all heads (not behind a shared prefix, nor over selected pages). Entries from lens on are copied. out may be mass itself."""

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, dtype: str = "bf16",
                 storage: str = "16bit", scale: float = 0.0, window: int = 0, soft_cap: float = 0.0):
        d = ag_attn_desc()
        lib.ag_attn_desc_init(ctypes.byref(d))
        d.dtype, self.torch_dtype = _pick(_DTYPES, dtype, "dtype")
        d.storage = _pick(_STORAGES, storage, "storage")
        d.head_dim, d.q_heads, d.kv_heads = head_dim, q_heads, kv_heads
        d.scale, d.window, d.soft_cap = scale, window, soft_cap
        n = lib.ag_attn_workspace_bytes(ctypes.byref(d))   # refuses what create would
        _checked(min(n, 0), "AttentionMass")
        self.desc, self._ref = d, ctypes.byref(d)
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim

    def add(self, mass, q, lse, cache: PagedCache, page_table, lens, decay: float = 1.0, out=None,
            stream=None):
        batch = q.shape[0]
        _is(q, "q", self.torch_dtype, (batch, self.q_heads, self.head_dim), cache)
        shape = (batch, self.kv_heads, mass.shape[2] if mass.dim() == 3 else None)
        _is(mass, "mass", torch.float32, shape, cache)
        _dense(_is(lse, "lse", torch.float32, (batch, self.q_heads), cache), "lse")
        _table(page_table, "page_table", batch, cache)
        _is(lens, "lens", torch.int32, (batch,), cache)
        where = _stream(stream, cache.index)
        if out is None:
            out = _empty(mass, mass.shape, torch.float32, stream)
        else:
            _is(out, "out", torch.float32, mass.shape, cache)
        ms, os, qs = mass.stride(), out.stride(), q.stride()
        rc = lib.ag_mass_add(self._ref, cache._ref, q.data_ptr(), qs[0], qs[1], lse.data_ptr(),
                             page_table.data_ptr(), page_table.stride(0), page_table.shape[1],
                             lens.data_ptr(), batch, mass.data_ptr(), ms[0], ms[1], out.data_ptr(), os[0],
                             os[1], mass.shape[2], decay, where)
        _checked(rc, "ag_mass_add")
        return out


class Evictor:
    """Keeps `budget` tokens of each sequence and kv head: the first `sink`, the last `recent`, and of the others
    those with the most mass (ag_evict_choose), and moves their rows together (ag_evict_move)."""

    def __init__(self, budget: int, sink: int = 4, recent: int = 64):
        if budget < 1 or sink < 0 or recent < 0 or sink + recent > budget:
            raise ValueError("sink + recent must be within 0 .. budget, and budget at least 1")
        self.budget, self.sink, self.recent = budget, sink, recent

    def choose(self, cache: PagedCache, page_table, lens, mass, stream=None):
        """(lens, kept, mass): kept int32 [batch, kv_heads, budget], the tokens that are kept, in order, and -1
        behind them; their masses, float32, and 0 behind them; lens int32 [batch], how many they are."""
        return self._choose(cache, page_table, lens, mass, stream, self._where(cache, page_table, lens, stream))

    def move(self, cache: PagedCache, page_table, kept, lens, to_table, to: Optional[PagedCache] = None,
             stream=None):
        """Row j of each sequence and kv head in the pages of to_table int32 [batch, pages] of `to` (the same
        cache if None) becomes the row of token kept[..., j]. No page may be both read and written, nor be in
        two places of to_table."""
        to = self._destination(cache, page_table, lens, to_table, to)
        where = self._where(cache, page_table, lens, stream)
        _dense(_tensor(kept, "kept", torch.int32, (lens.shape[0], cache.kv_heads, kept.shape[2] if kept.dim() == 3
                                                   else None), cache.device), "kept")
        self._move(cache, page_table, kept, lens, to_table, to, where)

    def run(self, cache: PagedCache, page_table, lens, mass, to_table, to: Optional[PagedCache] = None,
            stream=None):
        """choose and move in one call: (lens, kept, mass) of the moved sequences."""
        to = self._destination(cache, page_table, lens, to_table, to)
        where = self._where(cache, page_table, lens, stream)
        tokens, kept, new = self._choose(cache, page_table, lens, mass, stream, where)
        self._move(cache, page_table, kept, tokens, to_table, to, where)
        return tokens, kept, new

    @staticmethod
    def _where(cache, page_table, lens, stream):
        _table(page_table, "page_table", lens.shape[0], cache)
        _is(lens, "lens", torch.int32, (lens.shape[0],), cache)
        return _stream(stream, cache.index)

    @staticmethod
    def _destination(cache, page_table, lens, to_table, to):
        to = cache if to is None else to
        _table(to_table, "to_table", lens.shape[0], cache)
        if to.device != cache.device:
            raise ValueError("both caches must be on one GPU")
        if to.desc.k == cache.desc.k and to_table.data_ptr() == page_table.data_ptr() and lens.shape[0]:
            raise ValueError("rows cannot be moved within the pages that they are read from")
        return to

    def _choose(self, cache, page_table, lens, mass, stream, where):
        batch = lens.shape[0]
        shape = (batch, cache.kv_heads, mass.shape[2] if mass.dim() == 3 else None)
        _is(mass, "mass", torch.float32, shape, cache)
        kept = _empty(lens, (batch, cache.kv_heads, self.budget), torch.int32, stream)
        new = _empty(mass, kept.shape, torch.float32, stream)
        tokens = _like(lens, stream)
        ms = mass.stride()
        rc = lib.ag_evict_choose(cache._ref, mass.data_ptr(), ms[0], ms[1], mass.shape[2], page_table.data_ptr(),
                                 page_table.stride(0), page_table.shape[1], lens.data_ptr(), batch, self.budget,
                                 self.sink, self.recent, kept.data_ptr(), new.data_ptr(), tokens.data_ptr(), where)
        _checked(rc, "ag_evict_choose")
        return tokens, kept, new

    @staticmethod
    def _move(cache, page_table, kept, lens, to_table, to, where):
        rc = lib.ag_evict_move(cache._ref, page_table.data_ptr(), page_table.stride(0), page_table.shape[1],
                               to._ref, to_table.data_ptr(), to_table.stride(0), to_table.shape[1],
                               kept.data_ptr(), kept.shape[2], lens.data_ptr(), lens.shape[0], where)
        _checked(rc, "ag_evict_move")
