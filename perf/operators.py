"""The serving operators of an attention block, as cases to measure: rotary positions, the paged
key-value cache (quantised as it is written, and read back), the attention of one new token over it.

`run` computes a case either in the plain form (elementary torch operations in 32 bits, rounded
once at the end) or, where `own` is true, with all_gather_gemm_amd.attention. `exact` computes it
from the definitions in 64 bits.

Definitions. Rotary: pair i of a head's rotated part turns by position * theta_i. Cache: rows of
16-bit values, or of 8-bit (e4m3) or 4-bit (e2m1) codes with one power-of-two scale byte for each
32 values: the least 2^e, e >= -126, that brings the block's largest magnitude to at most 448 or 6;
codes round to nearest, ties to even. Attention: softmax over the scaled scores of a sequence's
tokens (the last `window` of them where a window is set; scores capped as cap*tanh(s/cap) where a
cap is set), times the values; also the natural logarithm of the softmax's sum. An empty sequence
gives zeros and minus infinity.
"""
import math
import random

import torch

own = False

_DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}
_TOP = {"mxfp8": 448.0, "mxfp4": 6.0}        # largest magnitude of a code
_FEW = {"mxfp8": 0.875, "mxfp4": 0.75}       # ... as a mantissa in [1/2, 1)
_EXP = {"mxfp8": 9, "mxfp4": 3}              # ... and its exponent


# ---------------------------------------------------------------- cases

def _rope(tokens, heads, dim, rot, pairing, scaling, dtype, grad=False, top=8192, order="run"):
    return {"op": "rope", "tokens": tokens, "heads": heads, "dim": dim, "rot": rot,
            "pairing": pairing, "scaling": scaling, "dtype": dtype, "grad": grad, "top": top,
            "order": order}


def _cache(tokens, heads, dim, page, storage, dtype):
    return {"op": "cache", "tokens": tokens, "heads": heads, "dim": dim, "page": page,
            "storage": storage, "dtype": dtype}


def _attn(op, batch, length, lens, q_heads, kv_heads, dim, page, storage, dtype, window=0, cap=0.0):
    return {"op": op, "batch": batch, "length": length, "lens": lens, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "storage": storage, "dtype": dtype,
            "window": window, "cap": cap}


def listed():
    return [
        # one new token of one sequence on one of 8 ranks (64 heads of 128 = 8192 columns, 8 key
        # heads): the least call there is, all latency
        dict(_rope(1, 9, 128, 128, "half", "none", "bf16", top=131072, order="random"),
             name="rope_one_token"),
        # a long prompt of 16384 tokens, all 64 q and 8 k heads, frequencies stretched for 131072
        dict(_rope(16384, 72, 128, 128, "half", "turns", "bf16", top=131072), name="rope_prompt"),
        # the gradient over a ragged batch of training tokens: heads of 80, the first half rotated
        # in interleaved pairs
        dict(_rope(4097, 28, 80, 40, "interleaved", "none", "f16", grad=True), name="rope_grad_part"),
        # the keys and values of 48 sequences' new tokens, stored in 8 bits and read back
        dict(_cache(48, 8, 128, 16, "mxfp8", "bf16"), name="cache_step_8bit"),
        # a prompt's keys and values into 8 bits and back, as when a prefix is moved
        dict(_cache(16384, 8, 128, 64, "mxfp8", "bf16"), name="cache_prompt_8bit"),
        # the same in 4 bits, an odd count of tokens, fp16, pages of 24
        dict(_cache(5001, 4, 64, 24, "mxfp4", "f16"), name="cache_prompt_4bit"),
        # the attention of one short sequence on one rank: latency
        dict(_attn("attn", 1, 300, "equal", 8, 1, 128, 16, "16bit", "bf16"), name="attn_one_short"),
        # one very long sequence on one rank: all the length has to be split
        dict(_attn("attn", 1, 131072, "equal", 8, 1, 128, 64, "mxfp8", "bf16"), name="attn_one_long_8bit"),
        # a batch of sequences of all lengths (one of them empty), 7 q heads a key head
        dict(_attn("attn", 61, 9000, "ragged", 28, 4, 128, 16, "16bit", "f16"), name="attn_ragged"),
        # a full batch of long sequences: the most bytes
        dict(_attn("attn", 64, 8192, "equal", 64, 8, 128, 64, "16bit", "bf16"), name="attn_batch_large"),
        # 4-bit cache, heads of 64, a window, capped scores, ragged
        dict(_attn("attn", 96, 6000, "ragged", 16, 8, 64, 32, "mxfp4", "bf16", 4096, 30.0),
             name="attn_window_4bit"),
        # the whole step between the projections: rotate q and k, write k and v, attend
        dict(_attn("step", 32, 4000, "ragged", 32, 8, 128, 16, "mxfp8", "bf16"), name="step_8bit"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: every size over its range, odd ones among them."""
    op = rng.choice(["rope", "cache", "attn", "attn", "step"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        heads = rng.choice([1, 5, 9, 16, 28, 40, 72])
        tokens = _log(rng, 1, min(16384, 16384 * 72 * 128 // (heads * dim)))
        return _rope(tokens, heads, dim, rng.choice([dim, dim // 2, 24, 20]),
                     rng.choice(["half", "interleaved"]),
                     rng.choice(["none", "linear", "base", "turns", "index"]), dtype,
                     rng.random() < 0.4, rng.choice([32768, 131072]), rng.choice(["run", "random"]))
    if op == "cache":
        storage = rng.choice(["16bit", "mxfp8", "mxfp4"])
        dim = rng.choice([64, 96, 128, 256])
        heads = rng.choice([1, 2, 4, 5, 8])
        return _cache(_log(rng, 1, 16384 * 8 * 128 // (heads * dim)), heads, dim,
                      rng.choice([1, 8, 16, 24, 64, 256]), storage, dtype)
    storage = rng.choice(["16bit", "mxfp8", "mxfp4"])
    dim = rng.choice([64, 96, 128, 256] + ([80] if storage == "16bit" else []))
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    q_heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 16])
    batch = _log(rng, 1, 256)
    most = 64 * 8192 * 8 * 128 // (batch * kv_heads * dim)
    length = _log(rng, 1, min(131072, most))
    return _attn(op, batch, length, rng.choice(["equal", "ragged"]), q_heads, kv_heads, dim,
                 rng.choice([8, 16, 24, 64, 256]), storage, dtype,
                 rng.choice([0, 0, 0, 1000, 4096]), rng.choice([0.0, 0.0, 0.0, 30.0]))


def _lengths(case):
    """The sequences' lengths: part of the case, the new token counted in."""
    batch, length = case["batch"], case["length"]
    if case["lens"] == "equal":
        return [length] * batch
    r = random.Random(7919 * batch + length)
    lens = [_log(r, 1, length) for _ in range(batch)]
    lens[r.randrange(batch)] = length
    if batch > 3:
        lens[lens.index(min(lens))] = 0
    return lens


def _attended(case):
    w = case["window"]
    return sum(min(n, w) if w else n for n in _lengths(case))


def _row_bytes(case):
    d = case["dim"]
    return {"16bit": 2 * d, "mxfp8": d + d // 32, "mxfp4": d // 2 + d // 32}[case["storage"]]


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 4 * n * case["dim"] + 8 * case["tokens"], "flops": 3 * n * case["rot"]}
    if case["op"] == "cache":   # written and read back, keys and values
        n = 2 * case["tokens"] * case["heads"]
        return {"bytes": n * (4 * case["dim"] + 2 * _row_bytes(case)) + 16 * case["tokens"],
                "flops": 4 * n * case["dim"]}
    rows = case["batch"] * case["q_heads"]
    seen = _attended(case)
    b = 2 * seen * case["kv_heads"] * _row_bytes(case) + rows * (4 * case["dim"] + 4)
    f = 4 * seen * case["q_heads"] * case["dim"]
    if case["op"] == "step":    # the new tokens' q read and written rotated, k and v read
        b += 4 * rows * case["dim"] + 4 * case["batch"] * case["kv_heads"] * case["dim"]
        f += 3 * (rows + case["batch"] * case["kv_heads"]) * case["dim"]
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------- inputs

def _scaling(case):
    """The frequencies' stretch: from 8192 positions to 131072 where the case has one."""
    kind = case.get("scaling", "none")
    return {"none": {}, "linear": {"factor": 4.0}, "base": {"factor": 4.0},
            "turns": {"factor": 16.0, "original_len": 8192.0, "low": 1.0, "high": 4.0},
            "index": {"factor": 16.0, "original_len": 8192.0, "low": 1.0, "high": 32.0,
                      "magnitude": 0.1 * math.log(16.0) + 1.0}}[kind]


def _thetas(case):
    """The rotation per position of each pair, in radians (64 bits), and the magnitude."""
    rot, kind, s = case.get("rot", case["dim"]), case.get("scaling", "none"), _scaling(case)
    base = 10000.0
    if kind == "base":
        base *= s["factor"] ** (rot / (rot - 2))
    i = torch.arange(rot // 2, dtype=torch.float64)
    th = base ** (-2.0 * i / rot)
    if kind == "linear":
        th = th / s["factor"]
    if kind == "turns":
        g = ((s["original_len"] * th / (2 * math.pi) - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        th = th * (g + (1 - g) / s["factor"])
    if kind == "index":
        at = lambda r: rot * math.log(s["original_len"] / (2 * math.pi * r)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(s["high"])), 0), min(math.ceil(at(s["low"])), rot - 1)
        g = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        th = th * (g + (1 - g) / s["factor"])
    return th, s.get("magnitude", 1.0)


def _plan_rope(case, top):
    """What a program keeps for the rotation: the framework's handle, or a table of cosines and
    sines."""
    rot, pairing = case.get("rot", case["dim"]), case.get("pairing", "half")
    if own:
        from all_gather_gemm_amd import attention
        return attention.Rope(case["dim"], rot_dim=rot, pairing=pairing, dtype=case["dtype"],
                              scaling=case.get("scaling", "none"), **_scaling(case))
    th, mag = _thetas(case)
    a = torch.arange(top, dtype=torch.float64, device="cuda")[:, None] * th.to("cuda")
    return (mag * a.cos()).float(), (mag * a.sin()).float()


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _pools(case, pages, g):
    """Keys and values of all pages, as a program that has run for a while holds them: random
    values in the cache's storage."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    if case["storage"] == "16bit":
        return {n: _normal(g, shape, _DTYPE[case["dtype"]]) for n in "kv"}
    got = {}
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for n in "kv":
        parts = [_quantise(_normal(g, (min(step, pages - p),) + shape[1:], _DTYPE[case["dtype"]]),
                           case["storage"]) for p in range(0, pages, step)]
        got[n], got[n + "_scale"] = (torch.cat(x) for x in zip(*parts))
    return got


def _plan_cache(case, pools):
    """The cache's handle: the framework's, or the tensors themselves."""
    if not own:
        return pools
    from all_gather_gemm_amd import attention
    return attention.PagedCache(pools["k"], pools["v"], pools.get("k_scale"), pools.get("v_scale"),
                                dtype=case["dtype"], storage=case["storage"])


def _plan_attn(case):
    if not own:
        return None
    from all_gather_gemm_amd import attention
    return attention.DecodeAttention(case["q_heads"], case["kv_heads"], case["dim"],
                                     dtype=case["dtype"], storage=case["storage"],
                                     window=case["window"], soft_cap=case["cap"])


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    g, d, td = _generator(seed), case["dim"], _DTYPE[case["dtype"]]
    if case["op"] == "rope":
        t, h = case["tokens"], case["heads"]
        # the rotated heads lie in front of two more in the projection's output
        x = _normal(g, (t, h + 2, d), td)[:, :h]
        if case["order"] == "run":
            first = int(torch.randint(0, case["top"] - t + 1, (1,), generator=g, device="cuda"))
            pos = torch.arange(first, first + t, device="cuda")
        else:
            pos = torch.randint(0, case["top"], (t,), generator=g, device="cuda")
        return {"x": x, "positions": pos}
    if case["op"] == "cache":
        t, h, page = case["tokens"], case["heads"], case["page"]
        qkv = _normal(g, (t, 2 * h, d), td)
        pages = 1 + -(-5 * t // (4 * page))
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:t].contiguous()
        return {"k": qkv[:, :h], "v": qkv[:, h:], "slots": slots, "pages": pages}
    b, h, page = case["batch"], case["kv_heads"], case["page"]
    lens = torch.tensor(_lengths(case), dtype=torch.int32)
    each = (lens + page - 1) // page
    pages = max(1, int(each.sum()))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    # sequence b's pages are the next `each[b]` of a random order; -1 beyond its length
    wide = torch.arange(max(1, int(each.max())), dtype=torch.int64)[None, :]
    begin = (each.cumsum(0) - each).to(torch.int64)[:, None]
    at = torch.where(wide < each[:, None], begin + wide, -1).to("cuda")
    table = torch.where(at >= 0, order[at.clamp(min=0)], -1).to(torch.int32)
    s = {"table": table, "lens": lens.to("cuda"), "pools": _pools(case, pages, g)}
    qkv = _normal(g, (b, case["q_heads"] + 2 * h, d), td)
    s["q"] = qkv[:, :case["q_heads"]]
    if case["op"] == "step":
        s["k"] = qkv[:, case["q_heads"]:case["q_heads"] + h]
        s["v"] = qkv[:, case["q_heads"] + h:]
        pos = s["lens"].to(torch.int64) - 1          # -1: an idle place in the batch
        last = pos.clamp(min=0)
        own_page = table.to(torch.int64).gather(1, (last // page)[:, None])[:, 0]
        s["positions"] = last
        s["slots"] = torch.where(pos >= 0, own_page * page + last % page, -1)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "rope":
        s["rope"] = _plan_rope(case, case["top"])
        return s
    if case["op"] == "cache":
        shape = (s["pages"], case["heads"], case["page"])
        if case["storage"] == "16bit":
            pools = {n: torch.zeros(shape + (case["dim"],), dtype=_DTYPE[case["dtype"]], device="cuda")
                     for n in "kv"}
        else:
            row = case["dim"] // (1 if case["storage"] == "mxfp8" else 2)
            pools = {n: torch.zeros(shape + (row,), dtype=torch.uint8, device="cuda") for n in "kv"}
            for n in "kv":
                pools[n + "_scale"] = torch.zeros(shape + (_scale_bytes(case["dim"]),),
                                                  dtype=torch.uint8, device="cuda")
        s["cache"] = _plan_cache(case, pools)
        return s
    s["cache"] = _plan_cache(case, s["pools"])
    s["attn"] = _plan_attn(case)
    if case["op"] == "step":
        s["rope"] = _plan_rope(case, case["length"])
    return s


# ---------------------------------------------------------------- the plain forms, 32 bits

def _scale_bytes(dim):
    return -(-(dim // 32) // 4) * 4


def _power(e):
    """2^e for whole e in [-126, 127]."""
    return ((e + 127) << 23).view(torch.float32)


def _quantise(x, storage):
    """(codes, scale bytes) of rows of 16-bit values."""
    top = torch.finfo(x.dtype).max
    f = x.float().unflatten(-1, (-1, 32))
    amax = f.abs().amax(-1, keepdim=True)
    odd = ~torch.isfinite(amax)
    m, e = torch.frexp(torch.where(odd, 1.0, amax))
    e = (e - _EXP[storage] + (m > _FEW[storage]).to(torch.int32)).to(torch.int32).clamp(min=-126)
    # the largest code whose value the 16-bit type holds
    over = _TOP[storage] * torch.ldexp(torch.ones_like(amax).double(), e) > top
    most = torch.where(over, 240.0 if storage == "mxfp8" else 3.0, _TOP[storage]).float()
    q = torch.where(odd, 0.0, f) * _power(-e)
    q = torch.maximum(torch.minimum(q, most), -most)
    scale = torch.where(odd, 255, e + 127).to(torch.uint8)[..., 0]
    pad = _scale_bytes(x.shape[-1]) - scale.shape[-1]
    scale = torch.nn.functional.pad(scale, (0, pad))
    q = q.flatten(-2)
    if storage == "mxfp8":
        return q.to(torch.float8_e4m3fn).view(torch.uint8), scale
    a = q.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
            + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8)
            + (a > 5.0).to(torch.uint8)) | (torch.signbit(q).to(torch.uint8) << 3)
    code = code.unflatten(-1, (-1, 2))
    return code[..., 0] | (code[..., 1] << 4), scale


def _values(codes, scale, dim, storage):
    """The values, in 32 bits, that codes and scale bytes stand for."""
    if storage == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
        low = (c & 1).float()
        e = ((c >> 1) & 3).to(torch.int32)
        v = torch.where(e == 0, 0.5 * low, (1 + 0.5 * low) * _power((e - 1).clamp(min=0)))
        v = torch.where((c & 8) != 0, -v, v)
    b = scale[..., :dim // 32].to(torch.int32)
    s = torch.where(b == 255, math.nan, _power(b.clamp(max=254) - 127))
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _turn(x, positions, table, rot, pairing, grad):
    cos, sin = table[0][positions][:, None], table[1][positions][:, None]
    if grad:
        sin = -sin
    f = x.float()
    r, rest = f[..., :rot], f[..., rot:]
    if pairing == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((r, rest), -1).to(x.dtype)


def _write(pools, k, v, slots, storage):
    """Scatter to the slots; a token whose slot is negative is left out (one with a slot is then
    written twice instead, so that the host need not wait for the count)."""
    page = pools["k"].shape[2]
    keep = slots >= 0
    pick = torch.where(keep, torch.arange(len(slots), device="cuda"), keep.to(torch.uint8).argmax())
    at = slots[pick]
    for n, x in (("k", k[pick]), ("v", v[pick])):
        if storage == "16bit":
            pools[n][at // page, :, at % page] = x
        else:
            pools[n][at // page, :, at % page], pools[n + "_scale"][at // page, :, at % page] = \
                _quantise(x, storage)


def _fetch(pools, slots, dim, storage, dtype):
    page = pools["k"].shape[2]
    a, b = slots // page, slots % page
    if storage == "16bit":
        return [pools[n][a, :, b] for n in "kv"]
    return [_values(pools[n][a, :, b], pools[n + "_scale"][a, :, b], dim, storage).to(dtype)
            for n in "kv"]


def _attend(s):
    case, q, lens = s["case"], s["q"], s["lens"]
    b, h, d = case["batch"], case["kv_heads"], case["dim"]
    table = s["table"].clamp(min=0)

    def gathered(n):
        x = s["pools"][n][table]
        if case["storage"] == "16bit":
            x = x.float()
        else:
            x = _values(x, s["pools"][n + "_scale"][table], d, case["storage"])
        return x.permute(0, 2, 1, 3, 4).reshape(b, h, -1, d)

    qt = q.float().reshape(b, h, -1, d).transpose(-1, -2).contiguous()
    score = torch.matmul(gathered("k"), qt) * (1.0 / math.sqrt(d))       # [b, h, tokens, group]
    if case["cap"]:
        score = case["cap"] * torch.tanh(score / case["cap"])
    t = torch.arange(score.shape[2], device="cuda")[None, :]
    seen = t < lens[:, None]
    if case["window"]:
        seen &= t >= lens[:, None] - case["window"]
    score = score.masked_fill(~seen[:, None, :, None], -math.inf)
    top = score.amax(2, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - top)
    total = p.sum(2)                                                     # [b, h, group]
    out = torch.matmul(p.transpose(-1, -2).contiguous(), gathered("v"))
    out = out / torch.where(total == 0, 1.0, total)[..., None]
    return {"out": out.reshape(b, -1, d).to(q.dtype),
            "lse": (top[:, :, 0] + total.log()).reshape(b, -1)}


# ---------------------------------------------------------------- one pass

def run(state):
    case, s = state["case"], state
    if case["op"] == "rope":
        if own:
            return (s["rope"].grad if case["grad"] else s["rope"].run)(s["x"], s["positions"])
        return _turn(s["x"], s["positions"], s["rope"], case["rot"], case["pairing"], case["grad"])
    if case["op"] == "cache":
        if own:
            s["cache"].append(s["k"], s["v"], s["slots"])
            k, v = s["cache"].read(s["slots"])
        else:
            _write(s["cache"], s["k"], s["v"], s["slots"], case["storage"])
            k, v = _fetch(s["cache"], s["slots"], case["dim"], case["storage"], s["k"].dtype)
        return {"k": k, "v": v}
    if own:
        q = s["q"]
        if case["op"] == "step":
            q = s["cache"].append_rope(s["rope"], q, s["k"], s["v"], s["positions"], s["slots"])
        out, lse = s["attn"].run(q, s["cache"], s["table"], s["lens"], return_lse=True)
        return {"out": out, "lse": lse}
    if case["op"] == "step":
        q = _turn(s["q"], s["positions"], s["rope"], case["dim"], "half", False)
        k = _turn(s["k"], s["positions"], s["rope"], case["dim"], "half", False)
        _write(s["pools"], k, s["v"], s["slots"], case["storage"])
        s = dict(s, q=q)
    return _attend(s)


# ---------------------------------------------------------------- 64 bits

def _binade(a):
    """floor(log2 a) of positive normal doubles, from their exponent bits."""
    return (a.view(torch.int64) >> 52) - 1023


def _two_to(e):
    return ((e + 1023) << 52).view(torch.float64)


def _grid64(x, storage, dtype):
    """What rows of 16-bit values read back as, from the definition: magnitudes rounded to the
    grid of the codes around each block's scale."""
    f = x.double().unflatten(-1, (-1, 32))
    amax, top = f.abs().amax(-1, keepdim=True), _TOP[storage]
    e = _binade(amax.clamp(min=2.0 ** -140)) - (8 if storage == "mxfp8" else 2)
    s = _two_to((e + (amax > top * _two_to(e)).long()).clamp(min=-126))
    a = f.abs() / s
    least, bits = (-6, 3) if storage == "mxfp8" else (0, 1)
    unit = _two_to(_binade(a.clamp(min=2.0 ** least)) - bits)
    r = torch.round(a / unit) * unit
    r = torch.where(r * s > torch.finfo(dtype).max, 240.0 if storage == "mxfp8" else 3.0, r)
    return (torch.copysign(r, f) * s).flatten(-2)


def _turn64(x, positions, case, grad=False):
    rot, half = case.get("rot", case["dim"]), case.get("pairing", "half") == "half"
    th, mag = _thetas(case)
    a = positions.double()[:, None] * th.to("cuda")
    z = torch.polar(torch.full_like(a, mag), -a if grad else a)[:, None]
    f = x.double()
    y = f.clone()
    first = slice(0, rot // 2) if half else slice(0, rot, 2)
    second = slice(rot // 2, rot) if half else slice(1, rot, 2)
    w = torch.complex(f[..., first], f[..., second]) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _codes64(codes, scale, dim, storage):
    c = codes.long()
    if storage == "mxfp4":
        c = torch.stack((c % 16, c // 16), -1).flatten(-2)
        grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        v = grid[c % 8] * (1 - 2 * (c // 8)).double()
    else:
        e, m = (c // 8) % 16, (c % 8).double()
        v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * _two_to(e - 7))
        v = v * (1 - 2 * (c // 128)).double()
    s = _two_to(scale[..., :dim // 32].long() - 127)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope":
        return _turn64(s["x"], s["positions"], case, case["grad"])
    if case["op"] == "cache":
        if case["storage"] == "16bit":
            return {n: s[n].double() for n in "kv"}
        return {n: _grid64(s[n], case["storage"], s[n].dtype) for n in "kv"}
    b, h, d, page = case["batch"], case["kv_heads"], case["dim"], case["page"]
    q = s["q"].double()
    new = {}
    if case["op"] == "step":
        # what is asked and what is stored are values of the 16-bit type, as for any caller
        q = _turn64(s["q"], s["positions"], case).to(s["q"].dtype).double()
        new["k"] = _turn64(s["k"], s["positions"], case).to(s["k"].dtype)
        new["v"] = s["v"]
        for n in "kv":
            new[n] = new[n].double() if case["storage"] == "16bit" else \
                _grid64(new[n], case["storage"], new[n].dtype)
    out = torch.zeros((b, case["q_heads"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((b, case["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(_lengths(case)):
        first = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        t = torch.arange(first, n, device="cuda")
        at, row = s["table"][i].long()[t // page], t % page
        kv = []
        for name in "kv":
            x = s["pools"][name][at, :, row]
            x = x.double() if case["storage"] == "16bit" else \
                _codes64(x, s["pools"][name + "_scale"][at, :, row], d, case["storage"])
            if new:
                x[-1] = new[name][i]
            kv.append(x)
        for j in range(h):
            group = slice(j * (case["q_heads"] // h), (j + 1) * (case["q_heads"] // h))
            z = (kv[0][:, j].contiguous() @ q[i, group].t().contiguous()) / math.sqrt(d)
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            lse[i, group] = torch.logsumexp(z, 0)
            p = torch.softmax(z, 0).t().contiguous()
            out[i, group] = p @ kv[1][:, j].contiguous()
    return {"out": out, "lse": lse}
