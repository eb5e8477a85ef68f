"""Single-token attention over a paged cache on the GPU against a 64-bit reference.

Tolerances, with w = sum |q k| * scale at its largest token, A = sum p |v|: scores are 32-bit sums of
exact products over dim elements (dim * 2^-24 * w off at most, and a few roundings of |s|), weights
carry that and the hardware's exponential (2^-22), and enter the product with 11 bits (f16) or 16
(bf16, in two parts), the sums over tokens 2^-20 of A. So out is within
    half an ulp of |out| + A * (2 * (dim + 8) * 2^-24 * w + 2^-11 [f16: weights] or 2^-15 + 2^-18)
and lse within (dim + 8) * 2^-24 * w + 2^-21 * (1 + |lse|)."""
import math

import numpy as np
import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def T():
    import all_gather_gemm_amd.attention
    return all_gather_gemm_amd.attention


class Problem:
    """Random sequences in a paged cache. What no token owns (rows past a length, unused pages, unused
    table entries) holds NaN bit patterns and page numbers far out of range."""

    def __init__(self, T, lens, q_heads, kv_heads, dim, page, storage, dtype, seed=1, holes=(),
                 spread=1.0, window=0, cap=0.0, scale=0.0, num_wgs=0, transposed=False):
        g = torch.Generator().manual_seed(seed)
        self.T, self.lens, self.dtype, self.storage = T, list(lens), dtype, storage
        self.page, self.window, self.cap = page, window, cap
        self.scale = scale or 1 / math.sqrt(dim)
        td = ref.TORCH[dtype]
        need = [-(-n // page) for n in lens]
        wide = max(need + [0]) + 1
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g).tolist()
        table = torch.full((len(lens), wide + 3), 0x7FFFFFFF, dtype=torch.int32)
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
        k = torch.randn((tokens, kv_heads, dim), generator=g).to(td)
        v = torch.randn((tokens, kv_heads, dim), generator=g).to(td)
        slots, self.absent, at = [], [], 0
        for b, n in enumerate(lens):
            mine = order[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = torch.tensor(mine, dtype=torch.int32)
            slots += [mine[i // page] * page + i % page for i in range(n)]
            gone = [j for j in holes if j < need[b]]
            table[b, gone] = torch.tensor([-1, pages, -(1 << 31)] * len(gone), dtype=torch.int32)[:len(gone)]
            self.absent.append(gone)
        slots = torch.tensor(slots, dtype=torch.int64, device=DEV)
        if tokens:
            self.cache.append(k.to(DEV), v.to(DEV), slots)
            k, v = self.cache.read(slots)       # what the cache stands for
        self.k, self.v = ref.f64(k), ref.f64(v)
        self.table = table.to(DEV)[:, :wide]    # rows further apart than they are long
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
        q = spread * torch.randn((len(lens), q_heads + 1, dim), generator=g)
        self.q = q.to(td).to(DEV)[:, 1:]        # strided
        self.attn = T.DecodeAttention(q_heads, kv_heads, dim, dtype=dtype, storage=storage, scale=scale,
                                      window=window, soft_cap=cap, num_wgs=num_wgs)

    def run(self, **kw):
        return self.attn.run(self.q, self.cache, self.table, self.lens_t, return_lse=True, **kw)

    def check(self, out, lse):
        q, out, lse = ref.f64(self.q), ref.f64(out), ref.f64(lse)
        dim, at = q.shape[-1], 0
        part = 2.0 ** -11 if self.dtype == "f16" else 2.0 ** -15
        for b, n in enumerate(self.lens):
            first = max(0, n - self.window) if self.window else 0
            seen = [t for t in range(first, n) if t // self.page not in self.absent[b]]
            k, v = self.k[at:at + n][seen], self.v[at:at + n][seen]
            at += n
            o, s, a, w = ref.attention(q[b], k, v, self.scale, self.cap)
            if not seen:
                assert (out[b] == 0).all() and np.isneginf(lse[b]).all()
                continue
            err = (dim + 8) * 2.0 ** -24 * w
            tol = ref.HALF_ULP[self.dtype] * np.abs(o) + \
                a * (2 * err + part + 2.0 ** -18)[:, None] + ref.TINY[self.dtype]
            assert (np.abs(out[b] - o) <= tol).all(), (b, n, np.abs(out[b] - o).max())
            assert (np.abs(lse[b] - s) <= err + 2.0 ** -21 * (1 + np.abs(s))).all(), (b, n)


EDGES = [0, 1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 300, 0, 1000]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("storage,dim", [
    ("16bit", 8), ("16bit", 64), ("16bit", 72), ("16bit", 128), ("16bit", 200), ("16bit", 256),
    ("mxfp8", 32), ("mxfp8", 64), ("mxfp8", 96), ("mxfp8", 128), ("mxfp8", 160), ("mxfp8", 256),
    ("mxfp4", 32), ("mxfp4", 64), ("mxfp4", 96), ("mxfp4", 128), ("mxfp4", 224), ("mxfp4", 256)])
def test_types_and_widths(T, dtype, storage, dim):
    p = Problem(T, EDGES, 6, 2, dim, 16, storage, dtype)
    p.check(*p.run())


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 100, 256])
@pytest.mark.parametrize("storage", ["16bit", "mxfp8", "mxfp4"])
def test_page_sizes(T, page, storage):
    p = Problem(T, [1, 40, 0, 257, 600], 8, 1, 128, page, storage, "bf16", seed=page, transposed=page == 24)
    p.check(*p.run())


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (5, 5), (7, 1), (16, 1), (17, 1), (66, 2), (48, 3), (71, 1)])
@pytest.mark.parametrize("dtype,storage", [("bf16", "16bit"), ("f16", "mxfp8")])
def test_head_groups(T, q_heads, kv_heads, dtype, storage):
    p = Problem(T, [130, 1, 0, 515], q_heads, kv_heads, 64, 16, storage, dtype, seed=q_heads)
    p.check(*p.run())


@pytest.mark.parametrize("window,cap,scale,spread", [
    (1, 0.0, 0.0, 1.0), (100, 0.0, 0.0, 1.0), (128, 5.0, 0.0, 4.0), (0, 30.0, 0.0, 1.0),
    (0, 0.0, 1.0, 3.0), (0, 0.5, 0.3, 1.0), (1 << 40, 0.0, 0.0, 1.0)])
def test_window_cap_scale(T, window, cap, scale, spread):
    for dtype, storage in (("f16", "16bit"), ("bf16", "mxfp4")):
        p = Problem(T, EDGES, 4, 2, 128, 16, storage, dtype, window=window, cap=cap, scale=scale, spread=spread)
        p.check(*p.run())


# one head's tokens over: one workgroup, few, more than are joined at once (16), and groups of
# groups with a short last one; and several sequences in one workgroup
@pytest.mark.parametrize("lens,kv_heads,num_wgs", [
    ([5000], 1, 1), ([5000], 1, 3), ([2200], 1, 17), ([8000, 3], 1, 40), ([33000], 1, 0),
    ([17000, 0, 5, 16000, 129], 2, 300), ([40] * 70, 3, 7), ([1] * 130, 1, 0), ([0, 0, 0], 2, 0),
    ([300, 0, 20] * 50, 2, 64), ([4100] * 5, 4, 33)])
def test_split_and_join(T, lens, kv_heads, num_wgs):
    p = Problem(T, lens, 4 * kv_heads, kv_heads, 64, 16, "16bit", "f16", num_wgs=num_wgs, spread=2.0)
    out, lse = p.run()
    p.check(out, lse)
    for _ in range(3):      # counters are left cleared, and the order of the joining is fixed
        again, lse2 = p.run()
        assert torch.equal(out, again) and torch.equal(lse, lse2)


# heads of a few tiles: each in one workgroup, each in one wave, several to a wave, cut or not
@pytest.mark.parametrize("storage,dim", [("16bit", 64), ("16bit", 128), ("mxfp8", 64), ("mxfp4", 128)])
@pytest.mark.parametrize("lens,kv_heads,num_wgs", [
    ([200], 1, 0), ([300], 1, 0), ([130, 256, 0, 200], 2, 0), ([300, 257, 0, 384], 2, 0),
    ([300, 257, 200, 384], 2, 0), ([300, 260] * 15, 3, 7), ([40] * 100, 3, 0), ([200, 129] * 50, 3, 0),
    ([300, 200, 100] * 40, 3, 0), ([300, 200, 1] * 20, 3, 0), ([100, 2000] + [60] * 130, 3, 100)])
def test_short_heads(T, storage, dim, lens, kv_heads, num_wgs):
    p = Problem(T, lens, 2 * kv_heads, kv_heads, dim, 16, storage, "f16", num_wgs=num_wgs, spread=2.0)
    out, lse = p.run()
    p.check(out, lse)
    again, lse2 = p.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("storage", ["16bit", "mxfp8", "mxfp4"])
def test_absent_pages(T, storage):
    p = Problem(T, [16, 33, 200, 0, 700], 8, 2, 128, 16, storage, "bf16", holes=(0, 2, 7, 8, 9))
    p.check(*p.run())       # the first sequence has no page at all


def test_lengths_past_the_table_and_below_zero(T):
    p = Problem(T, [40, 64, 10], 2, 1, 64, 16, "16bit", "f16")
    want, lse = p.run()
    table = p.table[:, :4].contiguous()
    lens = torch.tensor([40, 2000000000, -7], dtype=torch.int32, device=DEV)
    out, l2 = p.attn.run(p.q, p.cache, table, lens, return_lse=True)
    assert torch.equal(out[:2], want[:2]) and torch.equal(l2[:2], lse[:2])
    assert (out[2] == 0).all() and torch.isneginf(l2[2]).all()
    out, l2 = p.attn.run(p.q, p.cache, table[:, :0], lens, return_lse=True)
    assert (out == 0).all() and torch.isneginf(l2).all()


def test_sharp_and_flat_softmax(T):
    """One token far above the rest, first or last; scores that climb so that the maximum is raised
    many times; all keys equal; scores at the ends of the 16-bit type."""
    n, dim = 700, 64
    for case in ("first", "last", "climb", "flat", "large"):
        p = Problem(T, [n], 4, 1, dim, 16, "16bit", "f16", scale=1.0 if case != "large" else 1e-4)
        k = p.k.copy()
        q = torch.zeros_like(p.q)
        q[..., 0] = 1.0
        if case == "large":
            q[..., 0] = 60000.0
        k[:, 0, 0] = {"first": np.eye(1, n, 0)[0] * 60, "last": np.eye(1, n, n - 1)[0] * 60,
                      "climb": np.linspace(-80, 80, n), "flat": np.full(n, 3.0),
                      "large": np.linspace(-60000, 60000, n)}[case]
        kt = torch.from_numpy(k).half().to(DEV)
        slots = torch.cat([p.table[0, i // 16].long()[None] * 16 + i % 16 for i in range(n)])
        p.cache.append(kt, torch.from_numpy(p.v).half().to(DEV), slots)
        p.k, p.q = ref.f64(kt), q
        p.check(*p.run())


def test_infinities_and_nan_in_what_is_attended(T):
    """As the formula has them: -inf scores get no weight, a NaN key makes the row NaN, infinities in
    values stay where they are. In tokens that are not attended to nothing of it shows."""
    n, dim = 200, 64
    p = Problem(T, [n], 2, 1, dim, 16, "16bit", "bf16", window=100)
    q = torch.zeros_like(p.q)
    q[..., 0] = 1.0
    p.q = q
    slots = torch.cat([p.table[0, i // 16].long()[None] * 16 + i % 16 for i in range(n)])
    base_k, base_v = (torch.from_numpy(x).bfloat16().to(DEV) for x in (p.k, p.v))
    base_k[:, 0, 1:] = 0.5
    k, v = base_k.clone(), base_v.clone()
    k[:100] = float("nan")
    v[:100] = float("inf")
    k[150:, 0, 0] = float("-inf")
    p.cache.append(k, v, slots)
    out, lse = p.run()
    o, s, _, _ = ref.attention(ref.f64(q)[0][:, :1], ref.f64(k)[100:150, :, :1], ref.f64(v)[100:150], p.scale)
    assert np.abs(ref.f64(out)[0] - o).max() < 2.0 ** -7 and np.abs(ref.f64(lse)[0] - s).max() < 1e-4
    k2, v2 = base_k.clone(), base_v.clone()
    v2[120, 0, 3] = float("inf")
    p.cache.append(k2, v2, slots)
    out, _ = p.run()
    assert torch.isposinf(out[0, :, 3]).all() and torch.isfinite(out[0, :, :3]).all() and \
        torch.isfinite(out[0, :, 4:]).all()
    k2[130, 0, 9] = float("nan")
    p.cache.append(k2, base_v, slots)
    out, lse = p.run()
    assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_far_offsets(T):
    """Pages whose bytes lie past 2^32 from the pool's start."""
    page, dim = 64, 128
    pages = (1 << 32) // (page * dim * 2) + 40
    k = torch.empty((pages, 1, page, dim), dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    cache = T.PagedCache(k, v)
    n = 10 * page - 5
    ids = torch.arange(pages - 10, pages, device=DEV)
    g = torch.Generator().manual_seed(3)
    kt, vt = (torch.randn((n, 1, dim), generator=g).bfloat16().to(DEV) for _ in "kv")
    t = torch.arange(n, device=DEV)
    cache.append(kt, vt, ids[t // page] * page + t % page)
    q = torch.randn((1, 8, dim), generator=g).bfloat16().to(DEV)
    attn = T.DecodeAttention(8, 1, dim)
    out, lse = attn.run(q, cache, ids.int()[None], torch.tensor([n], dtype=torch.int32, device=DEV), return_lse=True)
    o, s, a, _ = ref.attention(ref.f64(q)[0], ref.f64(kt), ref.f64(vt), 1 / math.sqrt(dim))
    assert (np.abs(ref.f64(out)[0] - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -12 * a).all()
    back = cache.read(ids[t // page] * page + t % page)
    assert torch.equal(back[0], kt) and torch.equal(back[1], vt)


def test_streams_outputs_and_workspace(T):
    """Another stream than the tensors' own; an output that is a view, around which nothing is
    written; a workspace of the caller's."""
    import ctypes
    p = Problem(T, [500, 9], 8, 2, 128, 16, "mxfp8", "f16")
    want, lse = p.run()
    big = torch.full((2, 10, 131), 5.0, dtype=torch.float16, device=DEV)
    out = big[:, 1:9, 1:129]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, l2 = p.run(out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(l2, lse)
    rest = big.clone()
    rest[:, 1:9, 1:129] = 5.0
    assert (rest == 5.0).all()
    d, h = p.attn.desc, ctypes.c_void_p()
    need = T.lib.ag_attn_workspace_bytes(ctypes.byref(d))
    ws = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device=DEV)
    at = (ws.data_ptr() + 255) // 256 * 256
    assert T.lib.ag_attn_create(ctypes.byref(d), at, need - 1, ctypes.byref(h)) == -1
    assert T.lib.ag_attn_create(ctypes.byref(d), at + 16, need, ctypes.byref(h)) == -1
    assert T.lib.ag_attn_create(ctypes.byref(d), at, need, ctypes.byref(h)) == 0
    mine, p.attn.handle = p.attn.handle, h.value
    got, l2 = p.run()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(l2, lse)
    assert T.lib.ag_attn_destroy(h.value) == 0
    p.attn.handle = mine


def test_graph_replays(T):
    """The step (rotate, write, attend) captured once and replayed as the sequences grow, with eager
    work between: every replay is the eager result."""
    dim, page, heads, q_heads, batch = 128, 16, 2, 8, 5
    cache, twin = (T.PagedCache.empty(64, page, heads, dim, storage="mxfp8") for _ in "ab")
    rope, attn = T.Rope(dim), T.DecodeAttention(q_heads, heads, dim, storage="mxfp8")
    eager = T.DecodeAttention(q_heads, heads, dim, storage="mxfp8")
    table = torch.randperm(60, generator=torch.Generator().manual_seed(1))[:60].int().view(5, 12).to(DEV)
    qkv = torch.empty((batch, q_heads + 2 * heads, dim), dtype=torch.bfloat16, device=DEV)
    lens = torch.zeros(batch, dtype=torch.int32, device=DEV)
    slots, pos = torch.zeros(batch, dtype=torch.int64, device=DEV), torch.zeros(batch, dtype=torch.int64, device=DEV)
    out = torch.empty((batch, q_heads, dim), dtype=torch.bfloat16, device=DEV)
    q_out = torch.empty_like(out)

    def step(c, a, q_to, to):
        c.append_rope(rope, qkv[:, :q_heads], qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:],
                      pos, slots, q_out=q_to)
        a.run(q_to, c, table, lens, out=to)

    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        step(cache, attn, q_out, out)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.Generator().manual_seed(2)
    grown = torch.tensor([0, 1, 30, 100, 3], dtype=torch.int32, device=DEV)
    for i in range(20):
        grown += torch.tensor([1, 1, 0, 2, i % 3], dtype=torch.int32, device=DEV)
        lens.copy_(grown)
        pos.copy_((grown - 1).clamp(min=0).long())
        slots.copy_(table.long().gather(1, (pos // page)[:, None])[:, 0] * page + pos % page)
        qkv.copy_(torch.randn(qkv.shape, generator=g).bfloat16())
        graph.replay()
        q2, o2 = torch.empty_like(out), torch.empty_like(out)
        step(twin, eager, q2, o2)
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(q_out, q2), i


def test_refusals(T):
    p = Problem(T, [20, 3], 4, 2, 64, 16, "16bit", "bf16")
    for bad in (p.q.half(), p.q[:, :2], p.q[..., :32], p.q.cpu()):
        with pytest.raises(ValueError):
            p.attn.run(bad, p.cache, p.table, p.lens_t)
    for table in (p.table.long(), p.table[:1], p.table.t().contiguous().t()):
        with pytest.raises(ValueError):
            p.attn.run(p.q, p.cache, table, p.lens_t)
    for lens in (p.lens_t.long(), p.lens_t[:1], p.lens_t.cpu()):
        with pytest.raises(ValueError):
            p.attn.run(p.q, p.cache, p.table, lens)
    other = T.PagedCache.empty(2, 16, 2, 64, storage="mxfp8")
    with pytest.raises(T.AgmmError):
        p.attn.run(p.q, other, p.table, p.lens_t)
    with pytest.raises(T.AgmmError):
        T.DecodeAttention(3, 2, 64)
    assert p.attn.run(p.q[:0], p.cache, p.table[:0], p.lens_t[:0]).shape == (0, 4, 64)
