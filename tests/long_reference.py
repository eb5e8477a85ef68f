"""What the tests of include/agmm_long.h share: runs of tokens in a paged cache, and plain 64-bit references
from the header's definitions (numpy on the CPU)."""
from __future__ import annotations

import math

import numpy as np
import torch

import attention_reference as ref

DEV = "cuda"
ABSENT = [-1, 0x7FFFFFFF, -(1 << 31)]


class Pool:
    """Runs of tokens (of these lengths) in one paged cache, in pages of a random order. What no token owns (rows
    past a length, unused pages, unused table entries) holds NaN bit patterns and page numbers far out
    of range. holes: pages of each run that its table does not have."""

    def __init__(self, T, lens, kv_heads, dim, page, storage, dtype, seed=1, holes=(), transposed=False,
                 k=None, v=None, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.dtype, self.storage, self.dim = list(lens), page, dtype, storage, dim
        self.kv_heads = kv_heads
        td = ref.TORCH[dtype]
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        self.order = torch.randperm(pages, generator=g).tolist()
        shape = (pages, page, kv_heads) if transposed else (pages, kv_heads, page)
        row = dim if storage != "mxfp4" else dim // 2
        kind = td if storage == "16bit" else torch.uint8
        t = [torch.empty(shape + (row,), dtype=kind, device=DEV) for _ in "kv"]
        if storage != "16bit":
            t += [torch.empty(shape + (T.PagedCache.scale_bytes(dim),), dtype=torch.uint8, device=DEV)
                  for _ in "kv"]
        for x in t:
            x.view(torch.uint8).fill_(0xFF)      # NaN in every type
        if transposed:
            t = [x.transpose(1, 2) for x in t]
        self.cache = T.PagedCache(*t, dtype=dtype, storage=storage)
        tokens = sum(lens)
        draw = lambda: torch.randn((tokens, kv_heads, dim), generator=g)  # noqa: E731
        k = (draw() if k is None else k).to(td)
        v = (draw() if v is None else v).to(td)
        slots, self.pages, self.gone, at = [], [], [], 0
        for n, m in zip(lens, need):
            mine = self.order[at:at + m]
            at += m
            slots += [mine[i // page] * page + i % page for i in range(n)]
            self.gone.append([j for j in holes if j < m])
            self.pages.append(mine)
        self.free = self.order[at:]
        if tokens:
            slots = torch.tensor(slots, dtype=torch.int64, device=DEV)
            self.cache.append(k.to(DEV), v.to(DEV), slots)
            k, v = self.cache.read(slots)       # what the cache stands for
        k, v = ref.f64(k), ref.f64(v)
        ends = np.cumsum([0] + self.lens)
        self.k = [k[a:b] for a, b in zip(ends, ends[1:])]
        self.v = [v[a:b] for a, b in zip(ends, ends[1:])]

    def table(self, runs, extra=1):
        """The page table of some runs: rows further apart than they are long, entries past each run's pages
        far out of range."""
        wide = max([len(self.pages[r]) for r in runs] + [0]) + extra
        t = torch.full((len(runs), wide + 3), 0x7FFFFFFF, dtype=torch.int32)
        for i, r in enumerate(runs):
            t[i, :len(self.pages[r])] = torch.tensor(self.pages[r], dtype=torch.int32)
            for j, x in zip(self.gone[r], ABSENT * len(self.gone[r])):
                t[i, j] = x
        return t.to(DEV)[:, :wide]

    def lengths(self, runs):
        return torch.tensor([self.lens[r] for r in runs], dtype=torch.int32, device=DEV)

    def there(self, r):
        """Whether each token of a run is in a page that its table has."""
        return np.array([t // self.page not in self.gone[r] for t in range(self.lens[r])], dtype=bool)

    def q(self, batch, q_heads, seed=2, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        q = spread * torch.randn((batch, q_heads + 1, self.dim), generator=g)
        return q.to(ref.TORCH[self.dtype]).to(DEV)[:, 1:]        # strided


def check_attention(dtype, q, out, lse, keys, values, scale, cap=0.0):
    """out and lse of each sequence against the reference over keys[b] and values[b] [tokens, kv_heads, dim].

    Tolerances, with w = sum |q k| * scale at its largest token, A = sum p |v|: scores are 32-bit sums of exact
    products over dim elements (dim * 2^-24 * w off at most, and a few roundings of |s|), weights carry that and
    the hardware's exponential (2^-22), and enter the product with 11 bits (f16) or 16 (bf16, in two parts), the
    sums over tokens 2^-20 of A, and each joining of two parts four roundings of 2^-24. So out is within half an
    ulp of |out| + A * (2 * (dim + 8) * 2^-24 * w + 2^-11 [f16] or 2^-15 + 2^-18), and lse within (dim + 8) *
    2^-24 * w + 2^-21 * (1 + |lse|)."""
    q, out, lse = ref.f64(q), ref.f64(out), ref.f64(lse)
    dim = q.shape[-1]
    part = 2.0 ** -11 if dtype == "f16" else 2.0 ** -15
    for b, (k, v) in enumerate(zip(keys, values)):
        o, s, a, w = ref.attention(q[b], k, v, scale, cap)
        if not len(k):
            assert (out[b] == 0).all() and np.isneginf(lse[b]).all(), b
            continue
        err = (dim + 8) * 2.0 ** -24 * w
        tol = ref.HALF_ULP[dtype] * np.abs(o) + a * (2 * err + part + 2.0 ** -18)[:, None] + ref.TINY[dtype]
        assert (np.abs(out[b] - o) <= tol).all(), (b, len(k), np.abs(out[b] - o).max())
        assert (np.abs(lse[b] - s) <= err + 2.0 ** -21 * (1 + np.abs(s))).all(), (b, len(k))


# ---- the index ----

def least_exponent(most):
    e = -126
    if most > 127 * 2.0 ** -126:
        e = max(-126, math.frexp(most)[1] - 8)
        while most > 127 * 2.0 ** e:
            e += 1
    return e


def entry(k):
    """(codes [kv_heads, 2, dim], scale bytes [kv_heads]) of a page's keys [tokens, kv_heads, dim]; None for
    the codes of a head with a key that is not finite."""
    codes, scales = [], []
    for h in range(k.shape[1]):
        x = k[:, h]
        if not np.isfinite(x).all():
            codes.append(None)
            scales.append(255)
            continue
        e = least_exponent(np.abs(x).max())
        codes.append(np.stack((np.ceil(x.max(0) / 2.0 ** e), np.floor(x.min(0) / 2.0 ** e))).astype(np.int64))
        scales.append(e + 127)
    return codes, scales


def scores(q, codes, scales):
    """Scores of pages: q [heads, dim] of one kv head, codes [pages, 2, dim], scale bytes [pages]."""
    x = np.where(np.isfinite(q), q, 0.0)
    c = np.rint(x / 2.0 ** least_exponent(np.abs(x).max())).astype(np.int64)     # halves to even
    a, b = np.maximum(c, 0).sum(0), np.minimum(c, 0).sum(0)
    total = codes[:, 0] @ a + codes[:, 1] @ b
    with np.errstate(over="ignore"):
        got = total.astype(np.float32) * (2.0 ** (np.minimum(scales, 254).astype(np.float64) - 127)).astype(np.float32)
    return np.where(scales == 255, np.inf, got.astype(np.float64))


def highest(keys, there, sink, recent, budget):
    """The items that are kept, in order: the first `sink` and last `recent` of those there, then the highest keys
    (NaN above all), the earlier where equal."""
    n = len(keys)
    forced = [i for i in range(n) if there[i] and (i < sink or i >= n - recent)]
    rest = [i for i in range(n) if there[i] and not (i < sink or i >= n - recent)]
    rest.sort(key=lambda i: (not math.isnan(keys[i]), -keys[i] if not math.isnan(keys[i]) else 0.0, i))
    return sorted(forced + rest[:max(0, budget - len(forced))])
