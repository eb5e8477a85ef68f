"""The operators for long contexts over the paged key-value cache, as cases to measure: attention of a
batch that shares prefixes, attention over the pages that an index's cheap score selects, and eviction
by accumulated attention weight.

`run` computes a case either in the plain form (elementary torch operations in 32 bits, rounded once
at the end) or, where `own` is true, with all_gather_gemm_amd. `exact` computes it from the
definitions in 64 bits.

Definitions. A sequence's new token attends, per q head, with the softmax of the scaled scores (capped
as cap*tanh(s/cap) where a cap is set). Prefix: its tokens are those of its group's prefix and then its
own. Index: for a page and kv head the largest and the least of each element over the page's keys, in
units of 2^e, rounded outwards to whole numbers, with e the least from -126 on for which all of them fit
[-127, 127]. Score of a page: q's elements as whole numbers c in units of the least 2^f for which those of
all the kv head's q heads fit; the sum over elements and heads of c times the largest where c > 0, times
the least where c < 0 (so what q . k is at most, in the codes); as a 32-bit float, times 2^e. Selected are
the first `sink` pages, the last `recent` and of the others those with the highest scores, the lower page
first where they are equal, `budget` in all. Mass: a token's is decayed and gets the sum of its softmax
weights over the kv head's q heads. Eviction keeps the first `sink` tokens, the last `recent` and of the
others those with the most mass, the earlier first where they are equal, `budget` in all, and moves their
rows, in order, to other pages.
"""
import math
import random

import torch

own = False

_DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def _prefix(batch, groups, prefix, length, q_heads, kv_heads, dim, page, storage, dtype, cap=0.0):
    return {"op": "prefix", "batch": batch, "groups": groups, "prefix": prefix, "length": length,
            "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "storage": storage,
            "dtype": dtype, "cap": cap}


def _index(batch, length, kv_heads, dim, page, storage, dtype):
    return {"op": "index", "batch": batch, "length": length, "kv_heads": kv_heads, "dim": dim,
            "page": page, "storage": storage, "dtype": dtype}


def _select(batch, length, lens, budget, q_heads, kv_heads, dim, page, storage, dtype):
    return {"op": "select", "batch": batch, "length": length, "lens": lens, "budget": budget,
            "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "storage": storage,
            "dtype": dtype}


def _mass(batch, length, lens, q_heads, kv_heads, dim, page, storage, dtype, window=0, cap=0.0):
    return {"op": "mass", "batch": batch, "length": length, "lens": lens, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "storage": storage, "dtype": dtype,
            "window": window, "cap": cap}


def _evict(batch, length, lens, budget, kv_heads, dim, page, storage, dtype):
    return {"op": "evict", "batch": batch, "length": length, "lens": lens, "budget": budget,
            "kv_heads": kv_heads, "dim": dim, "page": page, "storage": storage, "dtype": dtype}


def listed():
    return [
        # four conversations just begun behind one system prompt, on one of 8 ranks: latency
        dict(_prefix(4, 1, 2000, 100, 8, 1, 128, 16, "16bit", "bf16"), name="prefix_small"),
        # a batch of samples of one long prompt, a whole block's 64 q and 8 kv heads
        dict(_prefix(64, 1, 8192, 512, 64, 8, 128, 64, "16bit", "bf16"), name="prefix_batch"),
        # three system prompts of different lengths in one ragged batch, 8-bit cache, 7 q heads a kv head
        dict(_prefix(45, 3, 6000, 700, 28, 4, 128, 16, "mxfp8", "f16"), name="prefix_groups_8bit"),
        # many requests about one long document: the most products
        dict(_prefix(256, 1, 32768, 1024, 64, 8, 128, 64, "16bit", "bf16"), name="prefix_document"),
        # the index of a prompt's pages, made once it is in the cache
        dict(_index(1, 16384, 8, 128, 16, "16bit", "bf16"), name="index_prompt"),
        # three short chats, 4-bit cache, heads of 64: update, select and attend, latency
        dict(_select(3, 2000, "ragged", 16, 16, 4, 64, 16, "mxfp4", "f16"), name="select_small"),
        # one very long sequence on one rank, 8-bit cache, 4096 of 131072 tokens attended to
        dict(_select(1, 131072, "equal", 64, 8, 1, 128, 64, "mxfp8", "bf16"), name="select_one_long_8bit"),
        # a ragged batch to 32768 tokens, 2048 of them attended to
        dict(_select(32, 32768, "ragged", 128, 32, 8, 128, 16, "16bit", "bf16"), name="select_batch"),
        # the weights of one sequence's new token added up: latency
        dict(_mass(1, 4096, "equal", 8, 1, 128, 16, "16bit", "bf16"), name="mass_one"),
        # the same for a batch of long sequences
        dict(_mass(32, 16384, "equal", 64, 8, 128, 64, "16bit", "bf16"), name="mass_batch"),
        # three chats of up to 2000 tokens cut to 512, 4-bit cache, pages of 24
        dict(_evict(3, 2000, "ragged", 512, 4, 64, 24, "mxfp4", "f16"), name="evict_small_4bit"),
        # a batch of 16384 tokens each cut to a quarter
        dict(_evict(32, 16384, "equal", 4096, 8, 128, 64, "16bit", "bf16"), name="evict_batch"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    """One more case: every size over its range, odd ones among them."""
    op = rng.choice(["prefix", "prefix", "index", "select", "select", "mass", "evict"])
    dtype = rng.choice(["f16", "bf16"])
    storage = rng.choice(["16bit", "16bit", "mxfp8", "mxfp4"])
    dim = rng.choice([64, 96, 128, 256] + ([80] if storage == "16bit" else []))
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    q_heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 16])
    page = rng.choice([8, 16, 24, 64, 256])
    lens = rng.choice(["equal", "ragged"])
    if op == "prefix":
        batch = _log(rng, 1, 256)
        most = 256 * 64 * 32768 * 128 // (batch * q_heads * dim)
        prefix = _log(rng, 16, min(32768, most))
        length = _log(rng, 1, min(4096, 256 * 8 * 1024 * 128 // (batch * kv_heads * dim)))
        return _prefix(batch, rng.choice([g for g in (1, 1, 2, 3, 8) if g <= batch]), prefix, length,
                       q_heads, kv_heads, dim, page, storage, dtype, rng.choice([0.0, 0.0, 0.0, 30.0]))
    batch = _log(rng, 1, 128)
    room = 32 * 16384 * 8 * 128 // (batch * kv_heads * dim)
    if op == "index":
        return _index(batch, _log(rng, 1, min(131072, room)), kv_heads, dim, page, storage, dtype)
    if op == "select":
        page = rng.choice([8, 16, 24, 64])
        length = _log(rng, 1, min(131072, room))
        # the budget from a few pages to a quarter of the longest sequence's
        budget = _log(rng, 4, max(4, min(length // (4 * page), 8192 // page)))
        return _select(batch, length, lens, budget, q_heads, kv_heads, dim, page, storage, dtype)
    if op == "mass":
        return _mass(batch, _log(rng, 1, min(131072, room)), lens, q_heads, kv_heads, dim, page, storage,
                     dtype, rng.choice([0, 0, 1000, 4096]), rng.choice([0.0, 0.0, 0.0, 30.0]))
    length = _log(rng, 16, min(131072, room))
    return _evict(batch, length, lens, _log(rng, 8, max(8, length // 3)), kv_heads, dim, page, storage,
                  dtype)


_SINK, _RECENT = 1, 2        # pages that are always selected


def _kept_ends(case):
    """Tokens that eviction keeps at a sequence's two ends."""
    return min(4, case["budget"] // 4), case["budget"] // 4


def _lengths(case):
    """The sequences' lengths: part of the case, the new token counted in."""
    batch, length = case["batch"], case["length"]
    if case.get("lens") == "equal":
        return [length] * batch
    r = random.Random(7919 * batch + length)
    lens = [_log(r, 1, length) for _ in range(batch)]
    lens[r.randrange(batch)] = length
    if batch > 3:
        lens[lens.index(min(lens))] = 0
    return lens


def _groups(case):
    """(first sequence of each prefix and the end, the prefixes' lengths)."""
    r = random.Random(104729 * case["batch"] + case["prefix"])
    n = case["groups"]
    starts = [0] + sorted(r.sample(range(1, case["batch"]), n - 1)) + [case["batch"]]
    return starts, [case["prefix"]] + [_log(r, 1, case["prefix"]) for _ in range(n - 1)]


def _row_bytes(case):
    d = case["dim"]
    return {"16bit": 2 * d, "mxfp8": d + d // 32, "mxfp4": d // 2 + d // 32}[case["storage"]]


def work(case):
    h, d, row = case["kv_heads"], case["dim"], _row_bytes(case)
    lens = _lengths(case)
    rows = case["batch"] * case.get("q_heads", 0)
    ends = rows * (4 * d + 4)                                   # q, out and lse
    if case["op"] == "prefix":
        starts, sizes = _groups(case)
        seen = sum(lens) * case["q_heads"]
        seen += sum(n * (b - a) for n, a, b in zip(sizes, starts, starts[1:])) * case["q_heads"]
        return {"bytes": 2 * (sum(lens) + sum(sizes)) * h * row + ends, "flops": 4 * seen * d}
    if case["op"] == "index":
        pages = sum(-(-n // case["page"]) for n in lens)
        return {"bytes": sum(lens) * h * row + pages * h * (2 * d + 1), "flops": 2 * sum(lens) * h * d}
    if case["op"] == "select":
        pages = [-(-n // case["page"]) for n in lens]
        # the pages attended to: all of them full but the last
        seen = sum(min(n, case["budget"] * case["page"]) for n in lens)
        own_pages = sum((n - 1) % case["page"] + 1 for n in lens if n)
        return {"bytes": sum(pages) * h * (2 * d + 1) + own_pages * h * row + 2 * seen * h * row + ends
                + 4 * h * sum(min(n, case["budget"]) for n in pages),
                "flops": 4 * sum(pages) * h * d + 4 * seen * case["q_heads"] * d}
    if case["op"] == "mass":
        w = case["window"]
        seen = sum(min(n, w) if w else n for n in lens)
        return {"bytes": seen * h * row + 8 * sum(lens) * h + rows * (2 * d + 4),
                "flops": 2 * seen * case["q_heads"] * d}
    kept = sum(min(n, case["budget"]) for n in lens)
    # masses read, the kept ones and their rows read and written, the list of them written
    moved = {"16bit": 4 * d}.get(case["storage"], 2 * row + 2 * d)      # (quantised rows are read back)
    return {"bytes": 4 * sum(lens) * h + kept * h * (2 * moved + 12), "flops": sum(lens) * h}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _scale_bytes(dim):
    return -(-(dim // 32) // 4) * 4


def _pool(case, pages, g):
    """Rows of all pages, as a program that has run for a while holds them: random values of the
    cache's storage around an offset of each element, as keys have them."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    at = _normal(g, (shape[1], 1, shape[3]))
    kind = _DTYPE[case["dtype"]] if case["storage"] == "16bit" else torch.uint8
    wide = shape[3] // 2 if case["storage"] == "mxfp4" else shape[3]
    data = torch.empty(shape[:3] + (wide,), dtype=kind, device="cuda")
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for p in range(0, pages, step):
        x = _normal(g, (min(step, pages - p),) + shape[1:]) + at
        if case["storage"] == "mxfp8":
            x = (x * 64).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        elif case["storage"] == "mxfp4":
            edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
            x = torch.bucketize(x.abs() * 2, edges).to(torch.uint8) | (torch.signbit(x).to(torch.uint8) << 3)
            x = x[..., 0::2] | (x[..., 1::2] << 4)
        data[p:p + step] = x.to(kind)
    if case["storage"] == "16bit":
        return data, None
    scale = torch.randint(0, 2, shape[:3] + (_scale_bytes(shape[3]),), generator=g, device="cuda")
    return data, (scale + (121 if case["storage"] == "mxfp8" else 126)).to(torch.uint8)


def _pools(case, pages, g):
    s = {}
    for n in "kv":
        s[n], s[n + "_scale"] = _pool(case, pages, g)
    return s


def _tables(sizes, page, g):
    """Page tables of runs of sequences (lists of lengths) over one pool whose pages are in a random
    order, -1 behind each length; and the count of pages."""
    each = [torch.tensor([-(-n // page) for n in lens]) for lens in sizes]
    pages = max(1, sum(int(e.sum()) for e in each))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    out, at = [], 0
    for e in each:
        wide = torch.arange(max(1, int(e.max())))[None, :]
        begin = (e.cumsum(0) - e)[:, None] + at
        at += int(e.sum())
        where = torch.where(wide < e[:, None], begin + wide, -1).to("cuda")
        out.append(torch.where(where >= 0, order[where.clamp(min=0)], -1).to(torch.int32))
    return out, pages


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    g, d, h, page, b = _generator(seed), case["dim"], case["kv_heads"], case["page"], case["batch"]
    lens = _lengths(case)
    s = {"lens": _ints(lens)}
    if case["op"] == "prefix":
        starts, sizes = _groups(case)
        (s["prefix_table"], s["table"]), pages = _tables([sizes, lens], page, g)
        s["prefix_lens"], s["starts"] = _ints(sizes), _ints(starts)
    else:
        (s["table"],), pages = _tables([lens], page, g)
    s["pools"] = _pools(case, pages, g)
    if "q_heads" in case:
        # q lies in front of k and v in the projection's output
        s["q"] = _normal(g, (b, case["q_heads"] + 2 * h, d), _DTYPE[case["dtype"]])[:, :case["q_heads"]]
    wide = s["table"].shape[1] * page
    if case["op"] in ("index", "select"):
        s["from"] = s["lens"] - 1 if case["op"] == "select" else torch.zeros_like(s["lens"])
        s["codes"] = torch.zeros((pages, h, 2, d), dtype=torch.int8, device="cuda")
        s["scales"] = torch.zeros((pages, h), dtype=torch.uint8, device="cuda")
    if case["op"] in ("mass", "evict"):
        # a few tokens hold most of what has been added up, some were never looked at
        m = torch.exp(2 * _normal(g, (b, h, wide)))
        s["mass"] = m * (torch.rand((b, h, wide), generator=g, device="cuda") > 0.2)
    if case["op"] == "mass":
        s["lse"] = _softmax(*_scores(case, s, _seen(case, s)))[2]
    if case["op"] == "evict":
        (s["to_table"],), s["to_pages"] = _tables([[min(n, case["budget"]) for n in lens]], page, g)
        if case["storage"] != "16bit":      # where the kept rows are read back from; none: zeros
            t = torch.arange(case["budget"], device="cuda")[None, :]
            p = s["to_table"].long()[:, (t[0] // page).clamp(max=s["to_table"].shape[1] - 1)]
            s["slots"] = torch.where(t < s["lens"][:, None], p * page + t % page, -1).flatten()
    return s


def _cache(case, pools):
    from all_gather_gemm_amd import attention
    return attention.PagedCache(pools["k"], pools["v"], pools["k_scale"], pools["v_scale"],
                                dtype=case["dtype"], storage=case["storage"])


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "select":      # every page's entry but those that a step renews is there already
        step = max(1, (1 << 27) // (case["kv_heads"] * case["page"] * case["dim"]))
        for p in range(0, s["codes"].shape[0], step):
            x = _values(case, {n: v if v is None else v[p:p + step] for n, v in s["pools"].items()}, "k")
            s["codes"][p:p + step], s["scales"][p:p + step] = _bounds(x, x)
    if case["op"] == "evict":
        s["to"] = {n: None if v is None else v.new_zeros((s["to_pages"],) + v.shape[1:])
                   for n, v in s["pools"].items()}
    if own:
        from all_gather_gemm_amd import attention, long_context
        geometry = dict(dtype=case["dtype"], storage=case["storage"])
        s["cache"] = _cache(case, s["pools"])
        if case["op"] == "prefix":
            s["attend"] = long_context.PrefixAttention(case["q_heads"], case["kv_heads"], case["dim"],
                                                       soft_cap=case["cap"], **geometry)
        if case["op"] in ("index", "select"):
            s["index"] = long_context.PageIndex(s["cache"], s["codes"], s["scales"])
        if case["op"] == "select":
            s["attend"] = attention.DecodeAttention(case["q_heads"], case["kv_heads"], case["dim"],
                                                    **geometry)
        if case["op"] == "mass":
            s["adder"] = long_context.AttentionMass(case["q_heads"], case["kv_heads"], case["dim"],
                                                    window=case["window"], soft_cap=case["cap"], **geometry)
        if case["op"] == "evict":
            s["to_cache"] = _cache(case, s["to"])
            sink, recent = _kept_ends(case)
            s["evictor"] = long_context.Evictor(case["budget"], sink=sink, recent=recent)
    return s


# ---------------------------------------------------------------- the plain forms, 32 bits

def _power(e):
    """2^e for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _values(case, pools, n):
    """The values, in 32 bits, of a pool's rows."""
    x = pools[n]
    if case["storage"] == "16bit":
        return x.float()
    if case["storage"] == "mxfp8":
        v = x.view(torch.float8_e4m3fn).float()
    else:
        c = torch.stack((x & 15, x >> 4), -1).flatten(-2)
        low, e = (c & 1).float(), ((c >> 1) & 3).to(torch.int32)
        v = torch.where(e == 0, 0.5 * low, (1 + 0.5 * low) * _power((e - 1).clamp(min=0)))
        v = torch.where((c & 8) != 0, -v, v)
    s = _power(pools[n + "_scale"][..., :case["dim"] // 32].to(torch.int32) - 127)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _gathered(case, s, n, table):
    """[..., kv_heads, tokens, dim] of the pages in table [..., pages]."""
    at = table.clamp(min=0).long()
    x = _values(case, {k: v if v is None else v[at] for k, v in s["pools"].items() if k[0] == n}, n)
    x = x.movedim(-3, -4)
    return x.reshape(x.shape[:-3] + (-1, x.shape[-1]))


def _capped(case, score):
    cap = case.get("cap", 0.0)
    return cap * torch.tanh(score / cap) if cap else score


def _seen(case, s):
    t = torch.arange(s["table"].shape[1] * case["page"], device="cuda")[None, :]
    seen = t < s["lens"][:, None]
    if case.get("window"):
        seen &= t >= s["lens"][:, None] - case["window"]
    return seen


def _q_rows(case, q):
    """[batch, kv_heads, group, dim] of 32-bit q."""
    return q.float().reshape(q.shape[0], case["kv_heads"], -1, case["dim"])


def _scores(case, s, seen):
    """The scores [batch, kv_heads, group, tokens] of a sequence's own tokens, and no values."""
    k = _gathered(case, s, "k", s["table"])
    score = torch.matmul(_q_rows(case, s["q"]), k.transpose(-1, -2).contiguous())
    score = _capped(case, score * (1.0 / math.sqrt(case["dim"])))
    return score.masked_fill(~seen[:, None, None, :], -math.inf), None


def _softmax(score, v):
    """Weights (of the largest 1), their sum and its logarithm, the weighted sum of v."""
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - top)
    total = p.sum(-1)
    lse = (top[..., 0] + total.log()).flatten(1)
    out = None if v is None else \
        torch.matmul(p, v) / torch.where(total == 0, 1.0, total)[..., None]
    return p, total, lse, out


def _attend_prefix(s):
    case = s["case"]
    starts, sizes = _groups(case)
    own_scores, _ = _scores(case, s, _seen(case, s))
    own_v = _gathered(case, s, "v", s["table"])
    out, lse = [], []
    for i, (a, b) in enumerate(zip(starts, starts[1:])):
        table = s["prefix_table"][i, :-(-sizes[i] // case["page"])]
        k, v = (_gathered(case, s, n, table)[:, :sizes[i]] for n in "kv")
        q = _q_rows(case, s["q"][a:b]).transpose(0, 1)                    # [h, batch, group, d]
        score = torch.matmul(q.reshape(q.shape[0], -1, q.shape[-1]).contiguous(),
                             k.transpose(-1, -2).contiguous())
        score = _capped(case, score * (1.0 / math.sqrt(case["dim"])))     # [h, batch * group, tokens]
        mine = own_scores[a:b].transpose(0, 1).reshape(score.shape[0], score.shape[1], -1)
        top = torch.maximum(score.amax(-1), mine.amax(-1))[..., None]
        score, mine = torch.exp(score - top), torch.exp(mine - top)
        total = score.sum(-1) + mine.sum(-1)
        mine = mine.reshape(q.shape[:3] + (-1,)).transpose(0, 1).contiguous()
        o = torch.matmul(score, v).reshape(q.shape).transpose(0, 1) + torch.matmul(mine, own_v[a:b])
        at = lambda x: x.reshape(q.shape[:3]).transpose(0, 1)             # noqa: E731
        out.append((o / at(total)[..., None]).reshape(b - a, -1, case["dim"]))
        lse.append(at(top[..., 0] + total.log()).reshape(b - a, -1))
    return {"out": torch.cat(out).to(s["q"].dtype), "lse": torch.cat(lse)}


def _least_exponent(most):
    """The least e from -126 on with most <= 127 * 2^e."""
    m, e = torch.frexp(most)
    return (e - 7 + (m > 127 / 128).to(torch.int32)).clamp(min=-126)


def _bounds(top, low):
    """(codes [..., 2, dim], scale bytes) of rows [..., page, dim] of which `top` has the values to take
    the largest of and `low` those to take the least of."""
    hi, lo = top.amax(-2), low.amin(-2)
    e = _least_exponent(torch.maximum(hi.abs(), lo.abs()).amax(-1))
    unit = _power(-e)[..., None]
    codes = torch.stack((torch.ceil(hi * unit), torch.floor(lo * unit)), -2)
    return codes.to(torch.int8), (e + 127).to(torch.uint8)


def _update(s):
    """The entries of the pages that hold tokens from s["from"] on: all of a prompt's, or each
    sequence's last one."""
    case, page, lens = s["case"], s["case"]["page"], s["lens"][:, None]
    table = s["table"]
    j = torch.arange(table.shape[1], device="cuda")[None, :]
    if case["op"] == "select":
        j = (lens.long() - 1).clamp(min=0) // page
        table = table.gather(1, j)
    # a page that no token is in: written again as the first sequence's longest has it
    x = _gathered(case, s, "k", table.reshape(-1, 1))                     # [pages, h, page, d]
    there = (j[..., None] * page + torch.arange(page, device="cuda") < lens[..., None]).reshape(-1, 1, page, 1)
    codes, scales = _bounds(x.masked_fill(~there, -math.inf), x.masked_fill(~there, math.inf))
    keep = there.flatten(1).any(1)
    pick = torch.where(keep, torch.arange(len(keep), device="cuda"), keep.to(torch.uint8).argmax())
    at = table.reshape(-1).long()[pick]
    s["codes"][at], s["scales"][at] = codes[pick], scales[pick]


def _selected(s):
    """(page table [batch, kv_heads, budget], lengths) of the selected pages."""
    case, page, budget, lens = s["case"], s["case"]["page"], s["case"]["budget"], s["lens"]
    q = _q_rows(case, s["q"])
    f = _least_exponent(q.abs().amax((-1, -2)))
    c = torch.round(q * _power(-f)[..., None, None])
    w = torch.cat((c.clamp(min=0).sum(-2), c.clamp(max=0).sum(-2)), -1).to(torch.int32)   # [b, h, 2 d]
    at = s["table"].clamp(min=0).long()
    codes = s["codes"][at].flatten(-2).to(torch.int32)                    # [b, pages, h, 2 d]
    total = (codes * w[:, None]).sum(-1)
    score = (total.float() * _power(s["scales"][at].to(torch.int32) - 127)).transpose(1, 2)
    pages = ((lens + page - 1) // page)[:, None, None]
    j = torch.arange(score.shape[-1], device="cuda")
    ends = (j < _SINK) | (j >= pages - _RECENT)
    score = torch.where(ends, math.inf, score).masked_fill(j >= pages, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :budget]
    n = pages.clamp(max=budget)
    first = torch.arange(order.shape[-1], device="cuda") < n
    order = torch.where(first, order, score.shape[-1]).sort(-1).values
    table = s["table"][:, None].expand(-1, order.shape[1], -1).gather(
        2, order.clamp(max=score.shape[-1] - 1))
    table = torch.where(first, table, -1)
    table = torch.nn.functional.pad(table, (0, budget - table.shape[-1]), value=-1)
    pages, n = pages[:, 0, 0], n[:, 0, 0]
    return table, ((n - pages) * page + lens).to(torch.int32)


def _attend_selected(s):
    case = s["case"]
    _update(s)
    table, n = _selected(s)
    b, h = table.shape[:2]
    at = table.clamp(min=0).long()
    heads = torch.arange(h, device="cuda")[None, :, None]

    def rows(name):
        got = {k: v if v is None else v[at, heads] for k, v in s["pools"].items() if k[0] == name}
        return _values(case, got, name).reshape(b, h, -1, case["dim"])

    score = torch.matmul(_q_rows(case, s["q"]), rows("k").transpose(-1, -2).contiguous())
    seen = torch.arange(score.shape[-1], device="cuda") < n[:, None]
    score = (score * (1.0 / math.sqrt(case["dim"]))).masked_fill(~seen[:, None, None, :], -math.inf)
    _, _, lse, out = _softmax(score, rows("v"))
    return {"out": out.reshape(b, -1, case["dim"]).to(s["q"].dtype), "lse": lse, "table": table, "lens": n,
            "codes": s["codes"], "scales": s["scales"]}


def _add_mass(s):
    case = s["case"]
    score, _ = _scores(case, s, _seen(case, s))
    lse = s["lse"].reshape(score.shape[:3])[..., None]
    p = torch.exp(score - torch.where(lse == -math.inf, 0.0, lse)).sum(2)
    there = (torch.arange(p.shape[-1], device="cuda") < s["lens"][:, None])[:, None]
    return torch.where(there, _DECAY * s["mass"] + p, s["mass"])


_DECAY = 0.96875        # 31/32: what was looked at long ago counts for less


def _evicted(s):
    case, page, budget, lens = s["case"], s["case"]["page"], s["case"]["budget"], s["lens"]
    sink, recent = _kept_ends(case)
    mass = s["mass"]
    t = torch.arange(mass.shape[-1], device="cuda")
    n = lens[:, None, None]
    key = torch.where((t < sink) | (t >= n - recent), math.inf, mass).masked_fill(t >= n, -1.0)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    m = n.clamp(max=budget)
    first = torch.arange(order.shape[-1], device="cuda") < m
    kept = torch.where(first, order, mass.shape[-1]).sort(-1).values
    kept = torch.where(first, kept, -1)
    kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[-1]), value=-1)
    at = kept.clamp(min=0)
    b, h = kept.shape[:2]
    from_page = s["table"][:, None].expand(-1, h, -1).gather(2, at // page).long()
    j = torch.arange(budget, device="cuda")
    to = s["to_table"].long()[:, (j // page).clamp(max=s["to_table"].shape[1] - 1)]   # [b, budget]
    there = j < m[:, 0]
    # (a place behind a sequence's end takes the first token's place and row once more)
    some = int(torch.tensor(_lengths(case)).argmax())
    pick = lambda x, y: torch.where(there, x, y)          # noqa: E731
    to_page, to_row = pick(to, s["to_table"][some, 0].long()), pick(j % page, 0)
    src_b, src_j = pick(torch.arange(b, device="cuda")[:, None], some), pick(j, 0)
    heads = torch.arange(h, device="cuda")[None, :, None]
    from_page = from_page[src_b[:, None], heads, src_j[:, None]]
    row = (at % page)[src_b[:, None], heads, src_j[:, None]]
    for name, pool in s["to"].items():
        if pool is not None:
            pool[to_page[:, None], heads, to_row[:, None]] = s["pools"][name][from_page, heads, row]
    new = torch.where(j < m, mass.gather(2, at), 0.0)
    out = {"kept": kept.to(torch.int32), "lens": lens.clamp(max=budget), "mass": new}
    if case["storage"] == "16bit":
        return dict(out, k=s["to"]["k"], v=s["to"]["v"])
    slots = s["slots"]
    for name in "kv":
        at = slots.clamp(min=0)
        got = {x: s["to"][x][at // page, :, at % page] for x in (name, name + "_scale")}
        x = _values(case, got, name).to(_DTYPE[case["dtype"]])
        out[name] = torch.where((slots >= 0)[:, None, None], x, 0.0)
    return out


# ---------------------------------------------------------------- one pass

def run(state):
    case, s = state["case"], state
    if case["op"] == "prefix":
        if not own:
            return _attend_prefix(s)
        out, lse = s["attend"].run(s["q"], s["cache"], s["prefix_table"], s["prefix_lens"], s["table"],
                                   s["lens"], starts=s["starts"], return_lse=True)
        return {"out": out, "lse": lse}
    if case["op"] == "index":
        if own:
            s["index"].update(s["table"], s["lens"], s["from"])
        else:
            _update(s)
        return {"codes": s["codes"], "scales": s["scales"]}
    if case["op"] == "select":
        if not own:
            return _attend_selected(s)
        s["index"].update(s["table"], s["lens"], s["from"])
        table, n = s["index"].select(s["q"], s["table"], s["lens"], case["budget"], sink=_SINK,
                                     recent=_RECENT)
        out, lse = s["attend"].run(s["q"], s["cache"], table, n, return_lse=True)
        return {"out": out, "lse": lse, "table": table, "lens": n, "codes": s["codes"],
                "scales": s["scales"]}
    if case["op"] == "mass":
        if not own:
            return _add_mass(s)
        return s["adder"].add(s["mass"], s["q"], s["lse"], s["cache"], s["table"], s["lens"],
                              decay=_DECAY)
    if not own:
        return _evicted(s)
    n, kept, mass = s["evictor"].run(s["cache"], s["table"], s["lens"], s["mass"], s["to_table"],
                                     to=s["to_cache"])
    out = {"kept": kept, "lens": n, "mass": mass}
    if case["storage"] == "16bit":
        return dict(out, k=s["to"]["k"], v=s["to"]["v"])
    k, v = s["to_cache"].read(s["slots"])
    return dict(out, k=k, v=v)


# ---------------------------------------------------------------- 64 bits

def _two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _rows64(case, s, name, table, tokens, head):
    """Values [tokens, dim] in 64 bits of one kv head's rows at these places of a page table's row."""
    page, dim = case["page"], case["dim"]
    at, row = table.long()[tokens // page], tokens % page
    x = s["pools"][name][at, head, row]
    if case["storage"] == "16bit":
        return x.double()
    c = x.long()
    if case["storage"] == "mxfp4":
        c = torch.stack((c % 16, c // 16), -1).flatten(-2)
        grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        v = grid[c % 8] * (1 - 2 * (c // 8)).double()
    else:
        e, m = (c // 8) % 16, (c % 8).double()
        v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * _two_to(e - 7)) * (1 - 2 * (c // 128)).double()
    b = s["pools"][name + "_scale"][at, head, row].long()[..., :dim // 32]
    return (v.unflatten(-1, (-1, 32)) * _two_to(b - 127)[..., None]).flatten(-2)


def _attend64(case, q, k, v):
    """(out, lse) of rows of q over one head's keys and values."""
    z = (q @ k.t().contiguous()) / math.sqrt(case["dim"])
    if case.get("cap"):
        z = case["cap"] * torch.tanh(z / case["cap"])
    return torch.softmax(z, -1) @ v, torch.logsumexp(z, -1)


def _codes64(x, used):
    """(upper and lower codes [pages, 2, dim], scale exponents) of keys [pages, tokens, dim], of which the
    first used[i] count."""
    there = torch.arange(x.shape[1], device=x.device)[None, :, None] < used[:, None, None]
    hi = x.masked_fill(~there, -math.inf).amax(1)
    lo = x.masked_fill(~there, math.inf).amin(1)
    most = torch.maximum(hi.abs(), lo.abs()).amax(1)
    e = (torch.ceil(torch.log2(most / 127)).clamp(min=-127) - 1).long()     # the logarithm may be off by one
    for _ in range(2):
        e += (most > 127 * _two_to(e)).long()
    e = e.clamp(min=-126)
    unit = _two_to(e)[:, None]
    return torch.stack((torch.ceil(hi / unit), torch.floor(lo / unit)), 1).to(torch.int8), e


def _highest64(key, ends, budget):
    """Which of the places are kept, in order: `ends`, and the highest keys of the rest."""
    rest = [i for i in range(len(key)) if not ends[i]]
    rest.sort(key=lambda i: (-key[i], i))
    return sorted([i for i in range(len(key)) if ends[i]] + rest[:max(0, budget - sum(ends))])


def exact(case, seed):
    lens = _lengths(case)
    h, d, page, b = case["kv_heads"], case["dim"], case["page"], case["batch"]
    pages = [-(-n // page) for n in lens]
    if case["op"] == "evict" and sum(lens) * h > 8000000:    # sorted on the host
        return None
    s = _inputs(case, seed)
    if "q_heads" in case:
        q, group = s["q"].double(), case["q_heads"] // h
        out = torch.zeros((b, case["q_heads"], d), dtype=torch.float64, device="cuda")
        lse = torch.full((b, case["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
    if case["op"] == "prefix":
        starts, sizes = _groups(case)
        for i, (first, end) in enumerate(zip(starts, starts[1:])):
            for j in range(h):
                heads = slice(j * group, (j + 1) * group)
                t = torch.arange(sizes[i], device="cuda")
                k, v = (_rows64(case, s, n, s["prefix_table"][i], t, j) for n in "kv")
                po, pl = _attend64(case, q[first:end, heads].reshape(-1, d).contiguous(), k, v)
                po, pl = po.reshape(end - first, group, d), pl.reshape(end - first, group)
                for a in range(first, end):
                    t = torch.arange(lens[a], device="cuda")
                    k, v = (_rows64(case, s, n, s["table"][a], t, j) for n in "kv")
                    so, sl = _attend64(case, q[a, heads].contiguous(), k, v)
                    both = torch.logaddexp(pl[a - first], sl)
                    lse[a, heads] = both
                    out[a, heads] = po[a - first] * (pl[a - first] - both).exp()[:, None] + \
                        (so * (sl - both).exp()[:, None] if lens[a] else 0.0)
        return {"out": out, "lse": lse}
    if case["op"] == "mass":
        new = s["mass"].double()
        for a, n in enumerate(lens):
            first = max(0, n - case["window"]) if case["window"] else 0
            new[a, :, :n] *= _DECAY
            t = torch.arange(first, n, device="cuda")
            for j in range(h if n else 0):
                heads = slice(j * group, (j + 1) * group)
                z = (q[a, heads] @ _rows64(case, s, "k", s["table"][a], t, j).t().contiguous()) / math.sqrt(d)
                if case["cap"]:
                    z = case["cap"] * torch.tanh(z / case["cap"])
                new[a, j, first:n] += torch.exp(z - s["lse"][a, heads].double()[:, None]).sum(0)
        return new
    if case["op"] == "evict":
        budget = case["budget"]
        sink, recent = _kept_ends(case)
        kept = torch.full((b, h, budget), -1, dtype=torch.int64)
        mass = torch.zeros((b, h, budget), dtype=torch.float64, device="cuda")
        to = {n: torch.zeros((s["to_pages"], h, page, d), dtype=torch.float64, device="cuda") for n in "kv"}
        host = s["mass"].double().cpu().tolist()
        for a, n in enumerate(lens):
            ends = [t < sink or t >= n - recent for t in range(n)]
            for j in range(h if n else 0):
                which = _highest64(host[a][j][:n], ends, budget) if n > budget else list(range(n))
                kept[a, j, :len(which)] = torch.tensor(which)
                w = torch.tensor(which, device="cuda")
                mass[a, j, :len(which)] = s["mass"][a, j, w].double()
                at = torch.arange(len(which), device="cuda")
                for name in "kv":
                    to[name][s["to_table"][a].long()[at // page], j, at % page] = \
                        _rows64(case, s, name, s["table"][a], w, j)
        got = {"kept": kept.to(torch.int32).to("cuda"), "lens": s["lens"].clamp(max=budget), "mass": mass}
        if case["storage"] != "16bit":
            at, there = s["slots"].clamp(min=0), (s["slots"] >= 0)[:, None, None]
            to = {n: torch.where(there, x[at // page, :, at % page], 0.0) for n, x in to.items()}
        return dict(got, **to)
    codes, scales = torch.zeros_like(s["codes"]), torch.zeros_like(s["scales"])
    for a, n in enumerate(lens):
        at = s["table"][a, :pages[a]].long()
        used = torch.full((pages[a],), page, device="cuda")
        used[pages[a] - 1:] = n - (pages[a] - 1) * page
        for j in range(h if n else 0):
            x = _rows64(case, s, "k", s["table"][a], torch.arange(pages[a] * page, device="cuda"), j)
            codes[at, j], e = _codes64(x.view(pages[a], page, d), used)
            scales[at, j] = (e + 127).to(torch.uint8)
    if case["op"] == "index":
        return {"codes": codes, "scales": scales}
    budget = case["budget"]
    new = torch.full((b, h, budget), -1, dtype=torch.int32, device="cuda")
    count = torch.zeros(b, dtype=torch.int32)
    for a, n in enumerate(lens):
        at = s["table"][a, :pages[a]].long()
        ends = [i < _SINK or i >= pages[a] - _RECENT for i in range(pages[a])]
        for j in range(h if n else 0):
            mine = q[a, j * group:(j + 1) * group]
            _, f = _codes64(mine[None], torch.tensor([group], device="cuda"))
            c = torch.round(mine / _two_to(f))[:, None]
            hi, lo = codes[at, j].double().unbind(1)
            total = (hi * c.clamp(min=0) + lo * c.clamp(max=0)).sum((0, 2))
            score = (total.float().double() * _two_to(scales[at, j].long() - 127)).tolist()
            which = _highest64(score, ends, budget) if pages[a] > budget else list(range(pages[a]))
            count[a] = (len(which) - pages[a]) * page + n
            which = torch.tensor(which, device="cuda")
            new[a, j, :len(which)] = at[which].to(torch.int32)
            t = (torch.arange(page, device="cuda") + page * which[:, None]).flatten()[:int(count[a])]
            out[a, j * group:(j + 1) * group], lse[a, j * group:(j + 1) * group] = _attend64(
                case, mine.contiguous(), *(_rows64(case, s, x, s["table"][a], t, j) for x in "kv"))
    return {"out": out, "lse": lse, "table": new, "lens": count.to("cuda"), "codes": codes, "scales": scales}
