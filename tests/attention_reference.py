"""Plain 64-bit references for the rotary positions, the paged cache and the single-token attention
(numpy on the CPU, from the definitions in include/agmm_attn.h)."""
from __future__ import annotations

import math

import numpy as np
import torch

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}   # of a result, times its magnitude's bound
TINY = {"f16": 2.0 ** -24, "bf16": 2.0 ** -133}     # half the least subnormal is below this


def f64(t) -> np.ndarray:
    return t.detach().cpu().double().numpy()


# ---- rotary positions ----

def thetas(rot, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=4.0):
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    th = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [t / factor for t in th]
    if scaling == "turns":
        out = []
        for t in th:
            g = (original_len * t / (2 * math.pi) - low) / (high - low)
            g = min(max(g, 0.0), 1.0)
            out.append(t * (g + (1 - g) / factor))
        return out
    if scaling == "index":
        def n(r):
            return rot * math.log(original_len / (2 * math.pi * r)) / (2 * math.log(base))
        i0, i1 = max(math.floor(n(high)), 0), min(math.ceil(n(low)), rot - 1)
        out = []
        for i, t in enumerate(th):
            g = 1 - min(max((i - i0) / max(i1 - i0, 0.001), 0.0), 1.0)
            out.append(t * (g + (1 - g) / factor))
        return out
    return th


def rope(x, positions, th, rot, start=0, pairing="half", magnitude=1.0, gradient=False):
    """x [..., tokens, heads, dim] float64, positions [..., tokens] integers. The angles are reduced
    in long double, so that positions up to 2^40 leave them exact to 1e-7."""
    turns = np.asarray(th, dtype=np.longdouble) / (2 * np.longdouble("3.14159265358979323846264338327950288"))
    a = np.asarray(positions, dtype=np.longdouble)[..., None] * turns
    a = ((a - np.rint(a)).astype(np.float64) * 2 * math.pi)[..., None, :]
    c, s = magnitude * np.cos(a), magnitude * np.sin(a)
    if gradient:
        s = -s
    y = x.copy()
    r = x[..., start:start + rot]
    if pairing == "half":
        a_, b_ = r[..., :rot // 2], r[..., rot // 2:]
        y[..., start:start + rot // 2] = a_ * c - b_ * s
        y[..., start + rot // 2:start + rot] = b_ * c + a_ * s
    else:
        a_, b_ = r[..., 0::2], r[..., 1::2]
        y[..., start:start + rot:2] = a_ * c - b_ * s
        y[..., start + 1:start + rot:2] = b_ * c + a_ * s
    return y


# ---- the cache ----

def code_values(storage):
    """The value of every code: e4m3 with its two NaN codes, or e2m1."""
    if storage == "mxfp4":
        half = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
        return np.array(half + [-v for v in half])
    out = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out.append((-v if c & 128 else v) if c & 127 != 127 else math.nan)
    return np.array(out)


def quantise(x, storage, dtype):
    """(codes, scale bytes) of rows [..., dim] of float64 values of the 16-bit type, by search: the
    least scale byte that fits, the nearest code, ties to the even one."""
    v = code_values(storage)
    n = 127 if storage == "mxfp8" else 8
    grid, top = v[:n], v[n - 1]
    most = float(torch.finfo(TORCH[dtype]).max)
    shape = x.shape
    blocks = x.reshape(-1, 32)
    codes = np.zeros(blocks.shape, dtype=np.uint8)
    scales = np.zeros(len(blocks), dtype=np.uint8)
    for i, b in enumerate(blocks):
        if not np.isfinite(b).all():
            scales[i] = 255
            continue
        s = 1
        while np.abs(b).max() > top * 2.0 ** (s - 127):
            s += 1
        scales[i] = s
        fits = grid * 2.0 ** (s - 127) <= most
        g = grid[fits]
        a = np.abs(b) / 2.0 ** (s - 127)
        up = np.searchsorted(g, a).clip(max=len(g) - 1)     # first code that is not below
        dn = np.maximum(up - 1, 0)
        du, dd = np.abs(g[up] - a), np.abs(a - g[dn])
        c = np.where(du < dd, up, np.where(dd < du, dn, np.where(up % 2 == 0, up, dn)))
        codes[i] = c | np.where(np.signbit(b), 128 if storage == "mxfp8" else 8, 0)
    codes = codes.reshape(shape)
    scales = scales.reshape(shape[:-1] + (-1,))
    if storage == "mxfp4":
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return codes, scales


def dequantise(codes, scales, storage):
    v = code_values(storage)
    if storage == "mxfp4":
        codes = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (-1,))
    x = v[codes].reshape(codes.shape[:-1] + (-1, 32))
    s = scales[..., :x.shape[-2]].astype(np.float64)
    s = np.where(s == 255, math.nan, 2.0 ** (s - 127))
    return (x * s[..., None]).reshape(codes.shape)


# ---- attention ----

def attention(q, k, v, scale, cap=0.0):
    """One sequence: q [q_heads, dim], k and v [tokens, kv_heads, dim] float64. Returns out, lse, and
    for the tolerances sum p |v| and the largest sum |q k| * scale over the tokens."""
    hq = q.shape[0]
    hk = k.shape[1]
    out, absum = np.zeros((hq, v.shape[2])), np.zeros((hq, v.shape[2]))
    lse, work = np.full(hq, -math.inf), np.zeros(hq)
    for h in range(hq):
        kk, vv = k[:, h // (hq // hk)], v[:, h // (hq // hk)]
        if len(kk) == 0:
            continue
        s = kk @ q[h] * scale
        work[h] = (np.abs(kk) @ np.abs(q[h])).max() * scale
        if cap:
            s = cap * np.tanh(s / cap)
        m = s.max()
        p = np.exp(s - m)
        lse[h] = m + math.log(p.sum())
        p = p / p.sum()
        out[h], absum[h] = p @ vv, p @ np.abs(vv)
    return out, lse, absum, work
