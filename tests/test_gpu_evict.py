"""Accumulated attention weights, the tokens that they keep, and moving their rows, on the GPU against the
definitions in include/agmm_long.h. Kept tokens, their masses and moved rows have to be equal.

Tolerance of an added mass, with w = sum |q k| * scale at the sequence's largest token: a score is off by (dim + 8) *
2^-24 * w, the log-sum-exp's product with log2 e and the difference by 2^-23 (|s| + |lse|), the hardware's
exponential by 2^-22, the sum of G weights by G * 2^-24 of it, and the decayed mass by one rounding; a weight p so by
p * (2 * (dim + 8) * 2^-24 * w + 2^-22 * (|s| + |lse|) + 2^-20)."""
import math

import numpy as np
import pytest
import torch

import attention_reference as ref
import long_reference as lr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    import all_gather_gemm_amd.attention
    return all_gather_gemm_amd.attention


@pytest.fixture(scope="module")
def L():
    import all_gather_gemm_amd.long_context
    return all_gather_gemm_amd.long_context


# ---- masses ----

class Masses:
    def __init__(self, T, L, lens, q_heads, kv_heads, dim, page, storage, dtype, seed=1, spread=1.0, window=0, cap=0.0,
                 scale=0.0, decay=0.75, room=7, **kw):
        self.pool = lr.Pool(T, lens, kv_heads, dim, page, storage, dtype, seed=seed, **kw)
        self.runs, self.decay, self.window, self.cap = range(len(lens)), decay, window, cap
        self.scale = scale or 1 / math.sqrt(dim)
        self.q = self.pool.q(len(lens), q_heads, seed=seed + 50, spread=spread)
        self.table, self.lens = self.pool.table(self.runs), self.pool.lengths(self.runs)
        shape = (len(lens), kv_heads + 1, max(lens + [0]) + room)
        wide = torch.rand(shape, generator=torch.Generator().manual_seed(seed)).to(lr.DEV)
        self.mass = wide[:, 1:]
        geometry = dict(dtype=dtype, storage=storage, scale=scale, window=window, soft_cap=cap)
        attn = T.DecodeAttention(q_heads, kv_heads, dim, **geometry)
        _, self.lse = attn.run(self.q, self.pool.cache, self.table, self.lens, return_lse=True)
        self.adder = L.AttentionMass(q_heads, kv_heads, dim, **geometry)

    def add(self, **kw):
        return self.adder.add(self.mass, self.q, self.lse, self.pool.cache, self.table, self.lens,
                              decay=self.decay, **kw)

    def check(self, got, mass=None):
        mass = self.mass if mass is None else mass
        q, lse, old, got = ref.f64(self.q), ref.f64(self.lse), ref.f64(mass), ref.f64(got)
        hk = self.pool.kv_heads
        group = q.shape[1] // hk
        for b in self.runs:
            n = self.pool.lens[b]
            first = max(0, n - self.window) if self.window else 0
            seen = self.pool.there(b) & (np.arange(n) >= first)
            assert (got[b, :, n:] == old[b, :, n:]).all()
            for h in range(hk):
                qh = q[b, h * group:(h + 1) * group]
                k = self.pool.k[b][:, h]
                s = k @ qh.T * self.scale
                w = (np.abs(k) @ np.abs(qh).T).max(initial=0.0) * self.scale
                if self.cap:
                    s = self.cap * np.tanh(s / self.cap)
                x = lse[b, h * group:(h + 1) * group]
                with np.errstate(invalid="ignore", over="ignore"):
                    p = np.where(seen[:, None], np.exp(s - x), 0.0)
                want = self.decay * old[b, h, :n] + p.sum(1)
                with np.errstate(invalid="ignore"):
                    err = np.where(seen[:, None], p * (2 * (q.shape[2] + 8) * 2.0 ** -24 * w +
                                                       2.0 ** -22 * (np.abs(s) + np.abs(x)) + 2.0 ** -20), 0.0).sum(1)
                tol = err + (group + 2) * 2.0 ** -24 * np.abs(want)
                assert (np.abs(got[b, h, :n] - want) <= tol).all(), (b, h)


EDGES = [0, 1, 2, 15, 16, 17, 63, 64, 65, 300, 0, 1000]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("storage,dim", [
    ("16bit", 8), ("16bit", 64), ("16bit", 72), ("16bit", 128), ("16bit", 200), ("16bit", 256),
    ("mxfp8", 32), ("mxfp8", 64), ("mxfp8", 96), ("mxfp8", 128), ("mxfp8", 160), ("mxfp8", 256),
    ("mxfp4", 32), ("mxfp4", 64), ("mxfp4", 96), ("mxfp4", 128), ("mxfp4", 224), ("mxfp4", 256)])
def test_mass_types_and_widths(T, L, dtype, storage, dim):
    m = Masses(T, L, EDGES, 6, 2, dim, 16, storage, dtype)
    m.check(m.add())


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (5, 5), (16, 1), (17, 1), (33, 1), (80, 2)])
@pytest.mark.parametrize("storage", ["16bit", "mxfp4"])
def test_mass_heads(T, L, q_heads, kv_heads, storage):
    m = Masses(T, L, [700, 33, 0], q_heads, kv_heads, 64, 24, storage, "bf16")
    m.check(m.add())


@pytest.mark.parametrize("kw", [dict(window=1), dict(window=100), dict(cap=0.5, spread=8.0), dict(cap=30.0, window=64),
                                dict(spread=30.0), dict(scale=0.5), dict(holes=(0, 2, 5)), dict(decay=0.0),
                                dict(decay=1.0, transposed=True)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_mass_options(T, L, kw, dim):
    m = Masses(T, L, [700, 33, 0, 1, 129], 8, 2, dim, 16, "16bit", "bf16", **kw)
    m.check(m.add())


def test_mass_in_place(T, L):
    m = Masses(T, L, [700, 33, 0], 8, 2, 128, 16, "16bit", "bf16")
    old, want = m.mass.clone(), m.add()
    assert m.add(out=m.mass) is m.mass
    assert torch.equal(m.mass, want)
    m.check(m.mass, old)


def test_mass_shorter_than_the_sequences(T, L):
    """Tokens past the masses, and masses past the table."""
    m = Masses(T, L, [700, 33, 300], 8, 2, 128, 16, "16bit", "bf16")
    want = m.add()
    full, m.mass = m.mass, m.mass[:, :, :290]
    assert torch.equal(m.add(), want[:, :, :290])
    m.mass, m.table = full, m.table[:, :10]
    got = m.add()
    assert torch.equal(got[:, :, :160], want[:, :, :160])
    assert torch.equal(got[0, :, 160:700], full[0, :, 160:700] * m.decay)


def test_mass_adds_up_to_the_heads(T, L):
    """All weights of a q head add up to 1: the masses of a kv head to its number of heads."""
    m = Masses(T, L, [5000], 16, 2, 128, 64, "mxfp8", "bf16", decay=0.0)
    total = m.add()[:, :, :5000].double().sum(-1)
    assert (total - 8).abs().max() < 8 * 2.0 ** -16


def test_mass_without_weights(T, L):
    """A log-sum-exp of minus infinity adds nothing."""
    m = Masses(T, L, [40], 4, 1, 64, 16, "16bit", "bf16")
    m.lse[:, 1] = -math.inf
    m.lse[:, 3] = -math.inf
    m.q = m.q.clone()
    got = m.add()
    keep = m.lse.clone()
    m.lse = torch.where(m.lse == -math.inf, 300.0, m.lse)   # exp(s - 300) rounds to 0
    assert torch.equal(got, m.add())
    m.lse = keep.fill_(-math.inf)
    assert torch.equal(m.add()[:, :, :40], m.mass[:, :, :40] * m.decay)


# ---- keeping ----

def check_kept(pool, mass, got, budget, sink, recent, limit=1 << 30):
    n, kept, new = (x.cpu() for x in got)
    host = mass.cpu().double().numpy()
    for b in range(len(pool.lens)):
        m = min(pool.lens[b], mass.shape[2], limit)
        there = pool.there(b)[:m]
        for h in range(pool.kv_heads):
            want = lr.highest(list(host[b, h, :m]), there, sink, recent, budget)
            assert n[b] == len(want), b
            assert kept[b, h].tolist() == want + [-1] * (budget - len(want)), (b, h)
            x = mass[b, h, want].cpu()
            assert torch.equal(new[b, h, :len(want)].nan_to_num(7.0), x.nan_to_num(7.0))
            assert (new[b, h, len(want):] == 0).all()


def some_mass(pool, seed=5, room=3):
    g = torch.Generator().manual_seed(seed)
    m = torch.exp(3 * torch.randn((len(pool.lens), pool.kv_heads + 1, max(pool.lens) + room), generator=g))
    m *= torch.rand(m.shape, generator=g) > 0.3
    return m.to(lr.DEV)[:, 1:]


@pytest.mark.parametrize("lens", [[0, 1, 15, 64, 65, 300, 1000], [2047, 2048, 2049, 5], [16384, 16385, 16383],
                                  [40000, 7]])
@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (64, 4, 16), (65, 0, 65), (700, 0, 0), (64, 64, 0)])
def test_kept(T, L, lens, budget, sink, recent):
    pool = lr.Pool(T, lens, 2, 8, 16, "16bit", "bf16")
    mass = some_mass(pool)
    e = L.Evictor(budget, sink=sink, recent=recent)
    got = e.choose(pool.cache, pool.table(range(len(lens))), pool.lengths(range(len(lens))), mass)
    check_kept(pool, mass, got, budget, sink, recent)


@pytest.mark.parametrize("kind", ["equal", "zero", "few", "negative", "odd", "close"])
def test_kept_values(T, L, kind):
    """Equal masses are kept from the front; NaN is the most; values one step apart are told apart."""
    lens = [500, 3000]
    pool = lr.Pool(T, lens, 1, 8, 16, "16bit", "bf16")
    mass = some_mass(pool).clone()
    if kind == "equal":
        mass.fill_(0.37)
    if kind == "zero":
        mass.zero_()
        mass[:, :, ::2] = -0.0
    if kind == "few":
        mass = (mass > 10).float()
    if kind == "negative":
        mass = -mass
    if kind == "odd":
        mass[:, :, 7] = math.nan
        mass[:, :, 300] = -math.nan
        mass[:, :, 9] = math.inf
        mass[:, :, 10] = -math.inf
    if kind == "close":
        steps = torch.randperm(mass.shape[2], generator=torch.Generator().manual_seed(1)) // 3
        mass[:] = (0x3F800000 + steps).to(torch.int32).view(torch.float32).to(lr.DEV)
    for budget, sink, recent in ((100, 2, 10), (499, 0, 0), (7, 0, 0)):
        e = L.Evictor(budget, sink=sink, recent=recent)
        got = e.choose(pool.cache, pool.table(range(2)), pool.lengths(range(2)), mass)
        check_kept(pool, mass, got, budget, sink, recent)


def test_kept_of_absent_pages(T, L):
    lens = [500, 40, 0, 9]
    pool = lr.Pool(T, lens, 2, 8, 8, "16bit", "bf16", holes=(0, 1, 3, 62))
    mass = some_mass(pool)
    for budget, sink, recent in ((100, 9, 10), (600, 0, 0), (4, 2, 2)):
        e = L.Evictor(budget, sink=sink, recent=recent)
        got = e.choose(pool.cache, pool.table(range(4)), pool.lengths(range(4)), mass)
        check_kept(pool, mass, got, budget, sink, recent)


def test_kept_odd_lengths(T, L):
    """Tokens past the masses or the table are not kept; negative lengths count as 0."""
    pool = lr.Pool(T, [64, 64], 1, 8, 16, "16bit", "bf16")
    mass = some_mass(pool)
    e = L.Evictor(20, sink=1, recent=3)
    full = pool.table(range(2), extra=0)
    lens = torch.tensor([1 << 30, -7], dtype=torch.int32, device=lr.DEV)
    n, kept, _ = e.choose(pool.cache, full, lens, mass)
    assert n.tolist() == [20, 0] and kept[0, 0, -1] == 63 and (kept[1] == -1).all()
    n, kept, _ = e.choose(pool.cache, full, lens, mass[:, :, :50])
    assert n.tolist() == [20, 0] and kept[0, 0, -3:].tolist() == [47, 48, 49]


# ---- moving ----

@pytest.mark.parametrize("storage,dim,dtype", [("16bit", 8, "f16"), ("16bit", 72, "bf16"), ("16bit", 128, "bf16"),
                                               ("16bit", 256, "f16"), ("mxfp8", 32, "bf16"), ("mxfp8", 160, "f16"),
                                               ("mxfp4", 32, "f16"), ("mxfp4", 96, "bf16"), ("mxfp4", 256, "bf16")])
@pytest.mark.parametrize("page,to_page", [(16, 16), (24, 7)])
def test_moved_rows(T, L, storage, dim, dtype, page, to_page):
    lens = [0, 5, 100, 333, 64]
    pool = lr.Pool(T, lens, 2, dim, page, storage, dtype, holes=(1,), transposed=page == 24)
    mass = some_mass(pool)
    budget = 50
    e = L.Evictor(budget, sink=2, recent=8)
    each = -(-budget // to_page)
    to = T.PagedCache.empty(5 * each + 2, to_page, 2, dim, dtype=dtype, storage=storage)
    held = [x for x in (to.k, to.v, to.k_scale, to.v_scale) if x is not None]
    for x in held:
        x.view(torch.uint8).fill_(0xA5)
    before = [x.clone() for x in held]
    order = torch.randperm(5 * each, generator=torch.Generator().manual_seed(9)).view(5, each)
    to_table = order.int().to(lr.DEV)
    table, n_all = pool.table(range(5)), pool.lengths(range(5))
    n, kept, new = e.run(pool.cache, table, n_all, mass, to_table, to=to)
    check_kept(pool, mass, (n, kept, new), budget, 2, 8)
    slots = torch.full((5, budget), -1, dtype=torch.int64)
    for b in range(5):
        for j in range(int(n[b])):
            slots[b, j] = order[b, j // to_page] * to_page + j % to_page
    k, v = to.read(slots.flatten().to(lr.DEV))
    k, v = (ref.f64(x).reshape(5, budget, 2, dim) for x in (k, v))
    for b in range(5):
        for h in range(2):
            w = [t for t in kept[b, h].tolist() if t >= 0]
            assert (k[b, :len(w), h] == pool.k[b][w, h]).all() and (v[b, :len(w), h] == pool.v[b][w, h]).all()
    # rows that nothing was moved to are as they were
    mine = {int(s) for s in slots.flatten() if s >= 0}
    rest = [s for s in range(to.k.shape[0] * to_page) if s not in mine]
    pages, rows = torch.tensor(rest) // to_page, torch.tensor(rest) % to_page
    bits = lambda x: x.view(torch.uint8)[pages.to(lr.DEV), :, rows.to(lr.DEV)]  # noqa: E731
    for x, y in zip(held, before):
        assert torch.equal(bits(x), bits(y))


def test_moved_within_one_cache(T, L):
    """Into pages of the cache that nothing holds, and the attention over what is kept."""
    lens = [300, 40, 500]
    budget, page, dim = 64, 16, 64
    pool = lr.Pool(T, lens, 2, dim, page, "16bit", "bf16", spare=20)
    mass = some_mass(pool)
    e = L.Evictor(budget, sink=4, recent=16)
    to_table = torch.tensor(pool.free[:12], dtype=torch.int32, device=lr.DEV).view(3, 4)
    n, kept, _ = e.run(pool.cache, pool.table(range(3)), pool.lengths(range(3)), mass, to_table)
    q = pool.q(3, 8)
    out, lse = T.DecodeAttention(8, 2, dim).run(q, pool.cache, to_table, n, return_lse=True)
    for h in range(2):
        w = [[t for t in kept[b, h].tolist() if t >= 0] for b in range(3)]
        lr.check_attention("bf16", q[:, 4 * h:4 * h + 4], out[:, 4 * h:4 * h + 4], lse[:, 4 * h:4 * h + 4],
                           [pool.k[b][w[b], h:h + 1] for b in range(3)],
                           [pool.v[b][w[b], h:h + 1] for b in range(3)], 1 / math.sqrt(dim))


def test_moved_nowhere(T, L):
    """Absent pages of the destination, tokens and rows past the tables, lengths past the budget."""
    pool = lr.Pool(T, [64], 1, 64, 16, "16bit", "bf16")
    e = L.Evictor(32, sink=0, recent=0)
    to = T.PagedCache.empty(2, 16, 1, 64)
    kept = torch.arange(32, dtype=torch.int32, device=lr.DEV).view(1, 1, 32)
    one = torch.tensor([[1, -1]], dtype=torch.int32, device=lr.DEV)
    many = torch.tensor([1 << 30], dtype=torch.int32, device=lr.DEV)
    e.move(pool.cache, pool.table([0]), kept, many, one, to=to)
    assert (to.k[0] == 0).all()
    assert (ref.f64(to.k[1, 0]) == pool.k[0][:16, 0]).all()
    to.k.zero_()
    e.move(pool.cache, pool.table([0]), kept, many, one[:, :1], to=to)
    assert (to.k[0] == 0).all() and (ref.f64(to.k[1, 0]) == pool.k[0][:16, 0]).all()
    to.k.zero_()
    kept[0, 0, 3], kept[0, 0, 4] = 1 << 30, -9
    e.move(pool.cache, pool.table([0]), kept, many, one, to=to)
    assert (to.k[1, 0, 3:5] == 0).all() and (ref.f64(to.k[1, 0, 5]) == pool.k[0][5, 0]).all()
    to.k.zero_()
    e.move(pool.cache, pool.table([0]), kept, many.fill_(-1), one, to=to)
    assert (to.k == 0).all()


def test_captured(T, L):
    """Adding, choosing and moving in one graph, replayed as the lengths change."""
    m = Masses(T, L, [300, 40, 500], 8, 2, 64, 16, "16bit", "bf16", spare=30)
    e = L.Evictor(64, sink=4, recent=16)
    to_table = torch.tensor(m.pool.free[:12], dtype=torch.int32, device=lr.DEV).view(3, 4)

    def step():
        mass = m.add()
        return (mass,) + e.run(m.pool.cache, m.table, m.lens, mass, to_table)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    full = m.lens.clone()
    for lens in (full, full // 3, full - 20, full):
        m.lens.copy_(lens)
        g.replay()
        torch.cuda.synchronize()
        moved = m.pool.cache.k.clone()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert torch.equal(moved.view(torch.int16), m.pool.cache.k.view(torch.int16))


def test_another_stream(T, L):
    m = Masses(T, L, [300, 40, 500], 8, 2, 64, 16, "16bit", "bf16", spare=30)
    e = L.Evictor(64, sink=4, recent=16)
    to_table = torch.tensor(m.pool.free[:12], dtype=torch.int32, device=lr.DEV).view(3, 4)
    want = (m.add(),) + e.run(m.pool.cache, m.table, m.lens, m.mass, to_table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = (m.add(stream=s),) + e.run(m.pool.cache, m.table, m.lens, m.mass, to_table, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_nothing(T, L):
    m = Masses(T, L, [30, 4], 8, 2, 64, 16, "16bit", "bf16")
    a = (m.pool.cache, m.table[:0], m.lens[:0])
    assert m.adder.add(m.mass[:0], m.q[:0], m.lse[:0], *a).shape == (0, 2, 37)
    assert m.adder.add(m.mass[:, :, :0], m.q, m.lse, m.pool.cache, m.table, m.lens).shape == (2, 2, 0)
    n, kept, new = L.Evictor(8, 1, 2).run(*a, m.mass[:0], m.table[:0].clone())
    assert n.shape == (0,) and kept.shape == (0, 2, 8)
    n, kept, new = L.Evictor(8, 1, 2).choose(m.pool.cache, m.table, m.lens, m.mass[:, :, :0])
    assert n.tolist() == [0, 0] and (kept == -1).all() and (new == 0).all()
