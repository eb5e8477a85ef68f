"""Rotary positions, the paged key-value cache and single-token attention: Python binding of the
functions of include/agmm_attn.h (libagmm.so).

What stands between the two sharded products of an attention block when it serves: `Rope` turns q
and k, `PagedCache` writes keys and values (quantised on the way where the cache is stored in 8 or 4
bits) and reads them back, `DecodeAttention` attends with one new token of every sequence. As in the
package's main module, this one only marshals arguments: tensors' pointers and strides and torch's
current stream go to the library's kernels, error codes come back as AgmmError, and there is no
fallback path.

With `stream`, a run is launched there instead: what it reads has to be ready on that stream, and
whoever reads its results waits for that stream (`wait_stream`). Results that a run allocates are
safe on the stream that was current as well; its inputs the caller keeps, or records on `stream`.

`Rope` takes part in autograd. The cache and the attention serve: no gradient passes through them.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import BF16, F16, AgmmError, AGMM_OK, _result, lib

AGMM_ERR_WRONG_DEVICE = -6

ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_NONE, ROPE_LINEAR, ROPE_BASE, ROPE_TURNS, ROPE_INDEX = range(5)
KV_16BIT, KV_MXFP8, KV_MXFP4 = range(3)

EXPORTED = [
    "ag_rope_desc_init", "ag_rope_thetas", "ag_rope_create", "ag_rope_destroy", "ag_rope_run",
    "ag_kv_append", "ag_kv_append_rope", "ag_kv_read", "ag_attn_desc_init",
    "ag_attn_workspace_bytes", "ag_attn_create", "ag_attn_destroy", "ag_attn_run",
]

_DTYPES = {"f16": (F16, torch.float16), "bf16": (BF16, torch.bfloat16)}
_PAIRINGS = {"half": ROPE_HALF, "interleaved": ROPE_INTERLEAVED}
_SCALINGS = {"none": ROPE_NONE, "linear": ROPE_LINEAR, "base": ROPE_BASE, "turns": ROPE_TURNS,
             "index": ROPE_INDEX}
_STORAGES = {"16bit": KV_16BIT, "mxfp8": KV_MXFP8, "mxfp4": KV_MXFP4}


class ag_rope_desc(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
        ("rot_start", ctypes.c_int32), ("pairing", ctypes.c_int32), ("scaling", ctypes.c_int32),
        ("base", ctypes.c_double), ("factor", ctypes.c_double), ("original_len", ctypes.c_double),
        ("low", ctypes.c_double), ("high", ctypes.c_double), ("magnitude", ctypes.c_double),
        ("thetas", ctypes.POINTER(ctypes.c_double)),
    ]


class ag_kv_cache(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("storage", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("num_pages", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
        ("row_stride", ctypes.c_int64), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("scale_page", ctypes.c_int64), ("scale_head", ctypes.c_int64),
        ("scale_row", ctypes.c_int64),
    ]


class ag_attn_desc(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("storage", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("num_wgs", ctypes.c_int32),
        ("window", ctypes.c_int64), ("scale", ctypes.c_float), ("soft_cap", ctypes.c_float),
    ]


def _declare():
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    rope, cache, attn = (ctypes.POINTER(t) for t in (ag_rope_desc, ag_kv_cache, ag_attn_desc))
    lib.ag_rope_desc_init.argtypes = [rope]
    lib.ag_rope_desc_init.restype = None
    lib.ag_rope_thetas.argtypes = [rope, ctypes.POINTER(ctypes.c_double)]
    lib.ag_rope_create.argtypes = [rope, ctypes.POINTER(vp)]
    lib.ag_rope_destroy.argtypes = [vp]
    lib.ag_rope_run.argtypes = [vp, vp, i64, i64, i64, vp, i64, i64, i64, vp, i64, i64, i64, i64,
                                i32, vp]
    lib.ag_kv_append.argtypes = [cache, vp, i64, i64, vp, i64, i64, vp, i64, vp]
    lib.ag_kv_append_rope.argtypes = [cache, vp, vp, i64, i64, i64, vp, i64, i64, vp, i64, i64, vp,
                                      i64, i64, vp, vp, i64, vp]
    lib.ag_kv_read.argtypes = [cache, vp, i64, vp, i64, i64, vp, i64, i64, vp]
    lib.ag_attn_desc_init.argtypes = [attn]
    lib.ag_attn_desc_init.restype = None
    lib.ag_attn_workspace_bytes.argtypes = [attn]
    lib.ag_attn_workspace_bytes.restype = i64
    lib.ag_attn_create.argtypes = [attn, vp, ctypes.c_size_t, ctypes.POINTER(vp)]
    lib.ag_attn_destroy.argtypes = [vp]
    lib.ag_attn_run.argtypes = [vp, cache, vp, i64, i64, vp, i64, i64, vp, i64, vp, i64, i64, vp,
                                vp]
    # of agmm_long.h: the attention with a page table for each kv head
    lib.ag_attn_run_heads.argtypes = [vp, cache, vp, i64, i64, vp, i64, i64, i64, vp, i64, vp, i64, i64, vp,
                                      vp]


_declare()


def _checked(rc: int, where: str):
    if rc != AGMM_OK:
        raise AgmmError(rc, where)


# The current stream's handle without a torch.cuda.Stream object made for it (2 us of a call's 7).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream, index: int) -> int:
    """The stream of a launch on the tensors' device. That has to be the current one: a kernel is launched
    on the current device, whatever its pointers and its stream belong to."""
    if index == _current():
        if stream is None:
            return _raw_stream(index)
        if getattr(stream, "device_index", index) == index:
            return stream.cuda_stream
    raise AgmmError(AGMM_ERR_WRONG_DEVICE, f"tensors on device {index}")


def _like(x, stream):
    return torch.empty_like(x) if stream is None else \
        _result(lambda: torch.empty_like(x), stream, x.device)


def _empty(x, shape, dtype, stream):
    return x.new_empty(shape, dtype=dtype) if stream is None else \
        _result(lambda: x.new_empty(shape, dtype=dtype), stream, x.device)


def _pick(table, key, what):
    if key not in table:
        raise ValueError(f"{what} is one of {', '.join(table)}: got {key!r}")
    return table[key]


def _tensor(t, name, dtype, shape, device=None):
    """A device tensor of this type and shape (None: any size) whose last dimension is dense."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_cuda and \
            (t.stride(-1) == 1 or t.shape[-1] == 1):
        return t
    if t.dtype != dtype or not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a {dtype} tensor on the GPU of the others")
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name} must have the shape {tuple(shape)}: got {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t


class _Rotation(torch.autograd.Function):
    """R x or R^T x, and the other one as its gradient."""

    @staticmethod
    def forward(ctx, x, rope, positions, gradient):
        ctx.rope, ctx.gradient = rope, gradient
        ctx.save_for_backward(positions)
        return rope._run(x.detach(), positions, None, None, gradient)

    @staticmethod
    def backward(ctx, dy):
        if dy.stride(-1) != 1:      # as that of a sum, which is one expanded element
            dy = dy.contiguous()
        return ctx.rope._run(dy, ctx.saved_tensors[0], None, None, 1 - ctx.gradient), None, None, None


class Rope:
    """Rotary positions of one head geometry and set of frequencies (ag_rope_desc).

    run(x, positions) returns R x for x [tokens, heads, head_dim] and positions [tokens], or with
    a batch in front of both ([batch, tokens, heads, head_dim]; positions [tokens] are then
    shared); any strides but the last dimension's. grad(dy, positions) returns R^T dy: the
    gradient of x, which autograd takes by itself where x requires it. out may be x itself; an
    x that requires a gradient takes none."""

    def __init__(self, head_dim: int, rot_dim: Optional[int] = None, rot_start: int = 0,
                 pairing: str = "half", dtype: str = "bf16", scaling: str = "none",
                 base: float = 10000.0, factor: float = 1.0, original_len: float = 0.0,
                 low: float = 1.0, high: float = 4.0, magnitude: float = 1.0,
                 thetas: Optional[Sequence[float]] = None):
        self.handle = None
        d = ag_rope_desc()
        lib.ag_rope_desc_init(ctypes.byref(d))
        d.dtype, self.torch_dtype = _pick(_DTYPES, dtype, "dtype")
        d.head_dim, d.rot_start = head_dim, rot_start
        d.rot_dim = head_dim if rot_dim is None else rot_dim
        d.pairing = _pick(_PAIRINGS, pairing, "pairing")
        d.scaling = _pick(_SCALINGS, scaling, "scaling")
        d.base, d.factor, d.original_len = base, factor, original_len
        d.low, d.high, d.magnitude = low, high, magnitude
        if thetas is not None:
            if len(thetas) != d.rot_dim // 2:
                raise ValueError(f"expected {d.rot_dim // 2} thetas, got {len(thetas)}")
            self._thetas = (ctypes.c_double * len(thetas))(*thetas)
            d.thetas = self._thetas
        self.desc, self.head_dim = d, head_dim
        h = ctypes.c_void_p()
        _checked(lib.ag_rope_create(ctypes.byref(d), ctypes.byref(h)), "ag_rope_create")
        self.handle = h.value

    def thetas(self):
        """The angles per position, in radians, as the handle was made with."""
        out = (ctypes.c_double * (self.desc.rot_dim // 2))()
        _checked(lib.ag_rope_thetas(ctypes.byref(self.desc), out), "ag_rope_thetas")
        return list(out)

    def close(self):
        if self.handle:
            lib.ag_rope_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def run(self, x, positions, out=None, stream=None):
        return self._run(x, positions, out, stream, 0)

    def grad(self, dy, positions, out=None, stream=None):
        return self._run(dy, positions, out, stream, 1)

    def _run(self, x, positions, out, stream, gradient):
        if x.requires_grad and torch.is_grad_enabled():
            if out is not None:
                raise ValueError("out takes no part in autograd: x must not require a gradient")
            run = lambda: _Rotation.apply(x, self, positions, gradient)  # noqa: E731
            return _result(run, stream, x.device)   # (backward runs on the same stream)
        shape, xs, device = x.shape, x.stride(), x.device
        dims = len(shape)
        if dims not in (3, 4):
            raise ValueError("x must be [tokens, heads, head_dim] or [batch, tokens, heads, head_dim]")
        _tensor(x, "x", self.torch_dtype, shape[:-1] + (self.head_dim,), device)
        shared = positions.dim() == 1
        _tensor(positions, "positions", torch.int64, shape[-3:-2] if shared else shape[:-2], device)
        where = _stream(stream, device.index)
        if out is None:
            out = _like(x, stream)
        else:
            _tensor(out, "out", self.torch_dtype, shape, device)
        ys, batch, xb, yb, pb = out.stride(), 1, 0, 0, 0
        if dims == 4:
            batch, xb, yb = shape[0], xs[0], ys[0]
        if not shared:
            pb = positions.stride(0)
        rc = lib.ag_rope_run(self.handle, x.data_ptr(), xb, xs[-3], xs[-2], out.data_ptr(), yb,
                             ys[-3], ys[-2], positions.data_ptr(), pb, batch, shape[-3], shape[-2],
                             gradient, where)
        _checked(rc, "ag_rope_run")
        return out


class PagedCache:
    """A paged key-value cache over the caller's tensors (ag_kv_cache).

    k and v: [pages, kv_heads, page_size, row], with any strides (equal for both, multiples of 16
    bytes) but the last dimension's, so a pool laid out [pages, page_size, kv_heads, row] is passed
    as its transposed view. row: head_dim values of the 16-bit type (storage "16bit"), or uint8
    codes, head_dim ("mxfp8") or head_dim / 2 ("mxfp4") of them, with k_scale and v_scale [pages,
    kv_heads, page_size, scale bytes] beside them. `empty` makes the tensors."""

    def __init__(self, k, v, k_scale=None, v_scale=None, dtype: str = "bf16",
                 storage: str = "16bit"):
        c = ag_kv_cache()
        c.dtype, self.torch_dtype = _pick(_DTYPES, dtype, "dtype")
        c.storage = _pick(_STORAGES, storage, "storage")
        kind = self.torch_dtype if storage == "16bit" else torch.uint8
        _tensor(k, "k", kind, (None,) * 4)
        _tensor(v, "v", kind, k.shape, k.device)
        if k.stride() != v.stride():
            raise ValueError("k and v must have the same strides")
        c.num_pages, c.kv_heads, c.page_size = k.shape[:3]
        c.head_dim = k.shape[3] * (2 if storage == "mxfp4" else 1)
        c.k, c.v = k.data_ptr(), v.data_ptr()
        c.page_stride, c.head_stride, c.row_stride = (s * k.element_size() for s in k.stride()[:3])
        if storage == "16bit":
            if k_scale is not None or v_scale is not None:
                raise ValueError("a 16-bit cache has no scales")
        else:
            if k_scale is None or v_scale is None:
                raise ValueError(f"a cache in {storage} needs k_scale and v_scale")
            shape = tuple(k.shape[:3]) + (self.scale_bytes(c.head_dim),)
            _tensor(k_scale, "k_scale", torch.uint8, shape, k.device)
            _tensor(v_scale, "v_scale", torch.uint8, shape, k.device)
            if k_scale.stride() != v_scale.stride():
                raise ValueError("k_scale and v_scale must have the same strides")
            c.k_scale, c.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
            c.scale_page, c.scale_head, c.scale_row = k_scale.stride()[:3]
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.desc, self._ref = c, ctypes.byref(c)
        self.storage, self.device, self.index = storage, k.device, k.device.index
        self.kv_heads, self.head_dim, self.page_size = c.kv_heads, c.head_dim, c.page_size

    @staticmethod
    def scale_bytes(head_dim: int) -> int:
        """Bytes of a row's scales: one for each 32 values, filled up to whole words."""
        return (head_dim // 32 + 3) // 4 * 4

    @classmethod
    def empty(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int,
              dtype: str = "bf16", storage: str = "16bit", device="cuda"):
        """A cache of new tensors, laid out [pages, kv_heads, page_size, row]: a page of one head is
        contiguous, which is what the attention reads together."""
        shape = (num_pages, kv_heads, page_size)
        if _pick(_STORAGES, storage, "storage") == KV_16BIT:
            kind, row = _pick(_DTYPES, dtype, "dtype")[1], head_dim
        else:
            kind, row = torch.uint8, head_dim // (2 if storage == "mxfp4" else 1)
        t = [torch.zeros(shape + (row,), dtype=kind, device=device) for _ in "kv"]
        if storage != "16bit":
            t += [torch.zeros(shape + (cls.scale_bytes(head_dim),), dtype=torch.uint8,
                              device=device) for _ in "kv"]
        return cls(*t, dtype=dtype, storage=storage)

    def append(self, k, v, slots, stream=None):
        """Writes k and v [tokens, kv_heads, head_dim] to slots [tokens] (int64; page * page_size +
        row; a slot out of range leaves its token out, one that two tokens share leaves its row
        undefined)."""
        tokens = slots.shape[0]
        shape, td, device = (tokens, self.kv_heads, self.head_dim), self.torch_dtype, self.device
        _tensor(k, "k", td, shape, device)
        _tensor(v, "v", td, shape, device)
        _tensor(slots, "slots", torch.int64, (tokens,), device)
        ks, vs = k.stride(), v.stride()
        rc = lib.ag_kv_append(self._ref, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
                              slots.data_ptr(), tokens, _stream(stream, device.index))
        _checked(rc, "ag_kv_append")

    def append_rope(self, rope: Rope, q, k, v, positions, slots, q_out=None, stream=None):
        """One launch for what comes before the attention: returns q [tokens, q_heads, head_dim]
        rotated, and writes k, rotated, and v to their slots."""
        tokens = slots.shape[0]
        shape, td, device = (tokens, self.kv_heads, self.head_dim), self.torch_dtype, self.device
        _tensor(q, "q", td, (tokens, q.shape[1] if q.dim() == 3 else None, self.head_dim), device)
        _tensor(k, "k", td, shape, device)
        _tensor(v, "v", td, shape, device)
        _tensor(slots, "slots", torch.int64, (tokens,), device)
        _tensor(positions, "positions", torch.int64, (tokens,), device)
        where = _stream(stream, device.index)
        if q_out is None:
            q_out = _like(q, stream)
        else:
            _tensor(q_out, "q_out", td, q.shape, device)
        qs, os, ks, vs = q.stride(), q_out.stride(), k.stride(), v.stride()
        rc = lib.ag_kv_append_rope(self._ref, rope.handle, q.data_ptr(), qs[0], qs[1], q.shape[1],
                                   q_out.data_ptr(), os[0], os[1], k.data_ptr(), ks[0], ks[1],
                                   v.data_ptr(), vs[0], vs[1], positions.data_ptr(),
                                   slots.data_ptr(), tokens, where)
        _checked(rc, "ag_kv_append_rope")
        return q_out

    def read(self, slots, k_out=None, v_out=None, stream=None):
        """(k, v) [tokens, kv_heads, head_dim] of the rows at slots, as values of the 16-bit type;
        zeros for a slot out of range."""
        tokens = slots.shape[0]
        shape, td, device = (tokens, self.kv_heads, self.head_dim), self.torch_dtype, self.device
        _tensor(slots, "slots", torch.int64, (tokens,), device)
        where = _stream(stream, device.index)
        k = _empty(slots, shape, td, stream) if k_out is None else \
            _tensor(k_out, "k_out", td, shape, device)
        v = _like(k, stream) if v_out is None else _tensor(v_out, "v_out", td, shape, device)
        ks, vs = k.stride(), v.stride()
        rc = lib.ag_kv_read(self._ref, slots.data_ptr(), tokens, k.data_ptr(), ks[0], ks[1],
                            v.data_ptr(), vs[0], vs[1], where)
        _checked(rc, "ag_kv_read")
        return k, v


class DecodeAttention:
    """Attention of one new token of every sequence over a PagedCache (ag_attn_desc).

    run(q, cache, page_table, lens): q [batch, q_heads, head_dim]; page_table int32 [batch,
    pages], or [batch, kv_heads, pages], a table for each kv head; lens int32 [batch], the new token
    counted in. Returns out like q, or (out, lse) with lse float32 [batch, q_heads]. A handle serves
    one stream at a time."""

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, dtype: str = "bf16",
                 storage: str = "16bit", scale: float = 0.0, window: int = 0,
                 soft_cap: float = 0.0, num_wgs: int = 0):
        self.handle = None
        d = ag_attn_desc()
        lib.ag_attn_desc_init(ctypes.byref(d))
        d.dtype, self.torch_dtype = _pick(_DTYPES, dtype, "dtype")
        d.storage = _pick(_STORAGES, storage, "storage")
        d.head_dim, d.q_heads, d.kv_heads = head_dim, q_heads, kv_heads
        d.scale, d.window, d.soft_cap, d.num_wgs = scale, window, soft_cap, num_wgs
        self.desc, self.q_heads, self.head_dim = d, q_heads, head_dim
        h = ctypes.c_void_p()
        _checked(lib.ag_attn_create(ctypes.byref(d), None, 0, ctypes.byref(h)), "ag_attn_create")
        self.handle = h.value

    def close(self):
        if self.handle:
            lib.ag_attn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def run(self, q, cache: PagedCache, page_table, lens, out=None, return_lse: bool = False,
            stream=None):
        batch, device = q.shape[0], cache.device
        _tensor(q, "q", self.torch_dtype, (batch, self.q_heads, self.head_dim), device)
        heads = page_table.dim() == 3
        _tensor(page_table, "page_table", torch.int32,
                (batch, self.desc.kv_heads, page_table.shape[2]) if heads else
                (batch, page_table.shape[1] if page_table.dim() == 2 else None), device)
        _tensor(lens, "lens", torch.int32, (batch,), device)
        where = _stream(stream, device.index)
        if out is None:
            out = _like(q, stream)
        else:
            _tensor(out, "out", self.torch_dtype, q.shape, device)
        lse = _empty(q, (batch, self.q_heads), torch.float32, stream) if return_lse else None
        qs, os = q.stride(), out.stride()
        if heads:
            ts = page_table.stride()
            rc = lib.ag_attn_run_heads(self.handle, cache._ref, q.data_ptr(), qs[0], qs[1],
                                       page_table.data_ptr(), ts[0], ts[1], page_table.shape[2],
                                       lens.data_ptr(), batch, out.data_ptr(), os[0], os[1],
                                       lse.data_ptr() if return_lse else None, where)
            _checked(rc, "ag_attn_run_heads")
            return (out, lse) if return_lse else out
        rc = lib.ag_attn_run(self.handle, cache._ref, q.data_ptr(), qs[0], qs[1],
                             page_table.data_ptr(), page_table.stride(0), page_table.shape[1],
                             lens.data_ptr(), batch, out.data_ptr(), os[0], os[1],
                             lse.data_ptr() if return_lse else None, where)
        _checked(rc, "ag_attn_run")
        return (out, lse) if return_lse else out
