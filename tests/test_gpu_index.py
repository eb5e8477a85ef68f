"""The page index, the pages that its score selects, and the attention over them, on the GPU against the
definitions in include/agmm_long.h. Entries, scores' order and selected pages are whole numbers: they have to be
equal. The attention's tolerances: long_reference.check_attention."""
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


def pages_of(n, page):
    return -(-n // page)


def check_entries(pool, index, run, starts=0):
    """The entries of the pages of a run from token `starts` on."""
    codes, scales = index.codes.cpu().numpy(), index.scales.cpu().numpy()
    n, page = pool.lens[run], pool.page
    for j in range(starts // page, pages_of(n, page)):
        at = pool.pages[run][j]
        if j in pool.gone[run]:
            continue
        want, s = lr.entry(pool.k[run][j * page:(j + 1) * page])
        assert (scales[at] == s).all(), (run, j)
        for h, w in enumerate(want):
            if w is not None:
                assert (codes[at, h] == w).all(), (run, j, h)


def want_selected(pool, index, run, q, budget, sink, recent):
    """(table [kv_heads, budget], tokens) from the index's entries."""
    n, page, hk = pool.lens[run], pool.page, pool.kv_heads
    m = pages_of(n, page)
    at = np.array(pool.pages[run][:m], dtype=np.int64)
    there = [j not in pool.gone[run] for j in range(m)]
    codes = index.codes.cpu().numpy().astype(np.int64)
    scales = index.scales.cpu().numpy()
    table = np.full((hk, budget), -1)
    tokens = 0
    for h in range(hk):
        group = q.shape[0] // hk
        s = lr.scores(q[h * group:(h + 1) * group], codes[at, h], scales[at, h]) if m else []
        which = lr.highest(list(s), there, sink, recent, budget)
        table[h, :len(which)] = at[which]
        tokens = sum(min(page, n - j * page) for j in which)
    return table, tokens


EDGES = [0, 1, 15, 16, 17, 100, 333, 0, 1000]


class Problem:
    def __init__(self, T, L, lens, q_heads, kv_heads, dim, page, storage, dtype, seed=1, spread=1.0, **kw):
        self.pool = lr.Pool(T, lens, kv_heads, dim, page, storage, dtype, seed=seed, **kw)
        self.runs = range(len(lens))
        self.q = self.pool.q(len(lens), q_heads, seed=seed + 50, spread=spread)
        self.table, self.lens = self.pool.table(self.runs), self.pool.lengths(self.runs)
        self.index = L.PageIndex(self.pool.cache)
        self.index.codes.fill_(77)
        self.index.scales.fill_(77)
        self.index.update(self.table, self.lens)

    def select(self, budget, sink=1, recent=2, **kw):
        return self.index.select(self.q, self.table, self.lens, budget, sink=sink, recent=recent, **kw)

    def check(self, got, budget, sink=1, recent=2):
        table, tokens = got[0].cpu().numpy(), got[1].cpu().numpy()
        q = ref.f64(self.q)
        for b in self.runs:
            want, n = want_selected(self.pool, self.index, b, q[b], budget, sink, recent)
            assert (table[b] == want).all(), (b, table[b], want)
            assert tokens[b] == n, b


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("storage,dim", [
    ("16bit", 8), ("16bit", 64), ("16bit", 72), ("16bit", 128), ("16bit", 200), ("16bit", 256),
    ("mxfp8", 32), ("mxfp8", 64), ("mxfp8", 96), ("mxfp8", 128), ("mxfp8", 256),
    ("mxfp4", 32), ("mxfp4", 64), ("mxfp4", 96), ("mxfp4", 128), ("mxfp4", 256)])
def test_types_and_widths(T, L, dtype, storage, dim):
    p = Problem(T, L, EDGES, 6, 2, dim, 16, storage, dtype)
    for b in p.runs:
        check_entries(p.pool, p.index, b)
    got = p.select(9)
    p.check(got, 9)
    # tables past 256 pages take another way to the same
    wide = p.index.select(p.q, p.pool.table(p.runs, extra=300), p.lens, 9)
    assert all(torch.equal(x, y) for x, y in zip(wide, got))
    # what belongs to no sequence is left as it was
    free = p.pool.free
    assert (p.index.codes[free] == 77).all() and (p.index.scales[free] == 77).all()


@pytest.mark.parametrize("page", [1, 3, 8, 24, 64, 100, 256])
def test_page_sizes(T, L, page):
    p = Problem(T, L, [0, 1, page, page + 1, 900, 2500], 8, 2, 64, page, "16bit", "bf16", seed=page,
                transposed=page == 24)
    for b in p.runs:
        check_entries(p.pool, p.index, b)
    p.check(p.select(7), 7)


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (5, 5), (16, 1), (128, 1), (40, 2)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_heads(T, L, q_heads, kv_heads, dim):
    p = Problem(T, L, [700, 33, 1200], q_heads, kv_heads, dim, 16, "16bit", "f16", seed=dim, spread=3.0)
    p.check(p.select(12), 12)


@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 1), (3, 2, 1), (8, 8 - 1, 1), (8, 0, 8), (40, 4, 4), (63, 1, 2),
                                                (200, 1, 1)])
def test_budgets(T, L, budget, sink, recent):
    p = Problem(T, L, [1000, 40, 16 * 63, 16 * 64, 0, 7], 8, 2, 128, 16, "16bit", "bf16")
    p.check(p.select(budget, sink, recent), budget, sink, recent)


@pytest.mark.parametrize("n", [2047, 2048, 2049, 2050, 16384, 16385, 40000])
def test_many_pages(T, L, n):
    """Pages of one token, at and past what a workgroup's threads hold at once."""
    p = Problem(T, L, [n, n // 3], 2, 1, 8, 1, "16bit", "bf16", seed=n)
    p.check(p.select(n // 5, 3, 9), n // 5, 3, 9)


def test_equal_scores(T, L):
    """Pages with one score are taken from the front: all alike, and a few above many."""
    n = 40 * 16
    k = torch.ones((n, 1, 64))
    k[16 * 30:16 * 33] = 2.0
    p = Problem(T, L, [n], 4, 1, 64, 16, "16bit", "bf16", k=k)
    p.q.copy_(p.q.abs() + 0.5)
    p.check(p.select(10, 1, 2), 10, 1, 2)
    table, _ = p.select(10, 1, 2)
    want = [0, 1, 2, 3, 4, 30, 31, 32, 38, 39]
    assert table[0, 0].tolist() == [p.pool.pages[0][j] for j in want]
    p.q.zero_()         # all scores are 0
    p.check(p.select(10, 0, 1), 10, 0, 1)


@pytest.mark.parametrize("power", [-130, -126, -120, -60, 0, 60, 110, 121])
def test_ends_of_the_range(T, L, power):
    """Keys and q at the ends of bf16's range, subnormal ones too; codes of tiny values next to large ones."""
    g = torch.Generator().manual_seed(3)
    k = torch.randn((160, 2, 64), generator=g).double()
    k = k.clamp(-1, 1) * 2.0 ** power
    k[40] = 2.0 ** min(power + 6, 126)
    k[41] = -k[40]
    p = Problem(T, L, [160], 4, 2, 64, 16, "16bit", "bf16", k=k)
    check_entries(p.pool, p.index, 0)
    for q in (1.0, 2.0 ** 100, 2.0 ** -130):
        p.q.copy_((torch.randn(p.q.shape, generator=g).double() * q).to(torch.bfloat16))
        p.check(p.select(5), 5)


def test_not_finite(T, L):
    """A page with a NaN or an infinity comes first; q's elements that are not finite count as 0."""
    k = torch.randn((320, 2, 64), generator=torch.Generator().manual_seed(4))
    k[100, 0, 5] = math.nan
    k[201, 1, 63] = -math.inf
    k[319, 0, 0] = math.inf
    p = Problem(T, L, [320], 4, 2, 64, 16, "16bit", "f16", k=k)
    check_entries(p.pool, p.index, 0)
    p.q[0, 1, 7] = math.nan
    p.q[0, 3, 0] = math.inf
    p.check(p.select(4, 1, 1), 4, 1, 1)


def test_absent_pages(T, L):
    p = Problem(T, L, [700, 40, 3, 0, 16 * 9], 8, 2, 64, 16, "16bit", "bf16", holes=(0, 2, 3, 8, 43))
    for b in p.runs:
        check_entries(p.pool, p.index, b)
    for budget, sink, recent in ((8, 2, 3), (100, 1, 1), (3, 1, 2)):
        p.check(p.select(budget, sink, recent), budget, sink, recent)


@pytest.mark.parametrize("new", [1, 5, 40])
def test_update_from(T, L, new):
    """Only the pages from the first new token on are made again."""
    lens = [0, 1, 16, 17, 100, 333]
    p = Problem(T, L, lens, 2, 1, 64, 16, "mxfp8", "bf16")
    p.index.codes.fill_(77)
    p.index.scales.fill_(77)
    starts = p.lens - new
    p.index.update(p.table, p.lens, starts)
    made = set()
    for b, n in enumerate(lens):
        check_entries(p.pool, p.index, b, max(0, n - new))
        made |= set(p.pool.pages[b][max(0, n - new) // 16:pages_of(n, 16)])
    rest = [i for i in range(p.index.scales.shape[0]) if i not in made]
    assert (p.index.scales[rest] == 77).all() and (p.index.codes[rest] == 77).all()
    # nothing new, and starts past the end
    before = p.index.codes.clone()
    p.index.update(p.table, p.lens, p.lens)
    p.index.update(p.table, p.lens, p.lens + 100)
    assert torch.equal(before, p.index.codes)
    p.index.update(p.table, p.lens, torch.full_like(p.lens, -9))
    for b in p.runs:
        check_entries(p.pool, p.index, b)


def test_odd_lengths(T, L):
    p = Problem(T, L, [64, 48, 32], 4, 1, 64, 16, "16bit", "bf16")
    full = p.pool.table(p.runs, extra=0)
    lens = torch.tensor([1 << 30, -4, -(1 << 31)], dtype=torch.int32, device=lr.DEV)
    table, tokens = p.index.select(p.q, full, lens, 6)
    assert tokens.tolist() == [64, 0, 0]
    assert table[0, 0].tolist() == p.pool.pages[0] + [-1, -1] and (table[1:] == -1).all()
    p.index.update(full, lens)
    check_entries(p.pool, p.index, 0)


@pytest.mark.parametrize("storage,dim,dtype", [("16bit", 128, "bf16"), ("16bit", 80, "f16"), ("mxfp8", 128, "f16"),
                                               ("mxfp4", 64, "bf16"), ("16bit", 256, "bf16"), ("mxfp8", 256, "f16")])
@pytest.mark.parametrize("page", [16, 24])
def test_attention_over_selected(T, L, storage, dim, dtype, page):
    lens = [0, 1, page, 333, 1000, 3 * page + 1]
    p = Problem(T, L, lens, 8, 2, dim, page, storage, dtype, holes=(2,))
    budget = 9
    table, tokens = p.select(budget)
    p.check((table, tokens), budget)
    attn = T.DecodeAttention(8, 2, dim, dtype=dtype, storage=storage)
    out, lse = attn.run(p.q, p.pool.cache, table, tokens, return_lse=True)
    # head by head: a kv head has pages of its own
    for h in range(2):
        keys, values = [], []
        for b, n in enumerate(lens):
            at = {x: j for j, x in enumerate(p.pool.pages[b])}
            which = [at[x] for x in table[b, h].tolist() if x >= 0]
            t = np.array([i for j in which for i in range(j * page, min(n, (j + 1) * page))], dtype=np.int64)
            keys.append(p.pool.k[b][t][:, h:h + 1])
            values.append(p.pool.v[b][t][:, h:h + 1])
        own = slice(4 * h, 4 * h + 4)
        lr.check_attention(dtype, p.q[:, own], out[:, own], lse[:, own], keys, values, 1 / math.sqrt(dim))


def test_tables_of_heads_that_agree(T, L):
    """A table for each kv head that holds the same pages gives what one table for all gives, bit for bit."""
    p = Problem(T, L, [0, 5, 700, 3000], 16, 4, 128, 16, "16bit", "bf16", holes=(3,))
    for kw in ({}, {"window": 100}, {"soft_cap": 5.0}):
        attn = T.DecodeAttention(16, 4, 128, **kw)
        a = attn.run(p.q, p.pool.cache, p.table, p.lens, return_lse=True)
        for t in (p.table[:, None].expand(-1, 4, -1), p.table[:, None].repeat(1, 4, 1)):
            b = attn.run(p.q, p.pool.cache, t, p.lens, return_lse=True)
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured(T, L):
    """update, select and attend in one graph, replayed as the sequences grow."""
    p = Problem(T, L, [900, 500, 64, 1], 8, 2, 64, 16, "16bit", "bf16")
    attn = T.DecodeAttention(8, 2, 64)

    def step():
        p.index.update(p.table, p.lens, p.lens - 1)
        table, tokens = p.select(8)
        return (table, tokens) + attn.run(p.q, p.pool.cache, table, tokens, return_lse=True)

    full = p.lens.clone()
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for lens in (full, full // 2, full - 17, full):
        p.lens.copy_(lens)
        g.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_another_stream(T, L):
    p = Problem(T, L, [900, 500, 64, 1], 8, 2, 64, 16, "16bit", "bf16")
    want = p.select(8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.index.update(p.table, p.lens, stream=s)
    got = p.select(8, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_nothing(T, L):
    p = Problem(T, L, [64, 48], 4, 1, 64, 16, "16bit", "bf16")
    table, tokens = p.index.select(p.q[:0], p.table[:0], p.lens[:0], 4)
    assert table.shape == (0, 1, 4) and tokens.shape == (0,)
    p.index.update(p.table[:0], p.lens[:0])
    table, tokens = p.index.select(p.q, p.table[:, :0], p.lens, 4)
    assert (table == -1).all() and (tokens == 0).all()
    p.index.update(p.table[:, :0], p.lens)
