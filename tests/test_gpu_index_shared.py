"""Entries of pages that stand in several places of one update's tables, with as many or as few of their tokens: each
has to be, whole, the one of the place with the most (numbers: equal)."""
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


class Shared:
    """One run of tokens in a pool, and sequences whose tables are made of its pages: places[b] lists indexes into
    the run's pages."""

    def __init__(self, T, L, tokens, kv_heads, dim, page, storage, dtype, places, lens, starts=None, seed=1):
        self.pool = lr.Pool(T, [tokens], kv_heads, dim, page, storage, dtype, seed=seed)
        self.page, self.places, self.n = page, places, lens
        wide = max(len(p) for p in places)
        t = torch.full((len(places), wide), 0x7FFFFFFF, dtype=torch.int32)
        for b, p in enumerate(places):
            t[b, :len(p)] = torch.tensor([self.pool.pages[0][i] for i in p], dtype=torch.int32)
        self.table = t.to(lr.DEV)
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device=lr.DEV)  # noqa: E731
        self.lens, self.starts = ints(lens), None if starts is None else ints(starts)
        self.first = [0] * len(lens) if starts is None else [max(0, s) for s in starts]
        self.index = L.PageIndex(self.pool.cache)

    def most(self):
        """{index into the run's pages: its most tokens of any place that is renewed}"""
        out = {}
        for p, n, s in zip(self.places, self.n, self.first):
            for j in range(s // self.page, -(-n // self.page) if s < n else 0):
                out[p[j]] = max(out.get(p[j], 0), min(self.page, n - j * self.page))
        return out

    def update(self):
        self.index.codes.fill_(77)
        self.index.scales.fill_(77)
        self.index.update(self.table, self.lens, self.starts)
        return self.index.codes.cpu().numpy(), self.index.scales.cpu().numpy()

    def check(self):
        codes, scales = self.update()
        most, k = self.most(), self.pool.k[0]
        for i, at in enumerate(self.pool.pages[0]):
            if i not in most:
                assert (codes[at] == 77).all() and (scales[at] == 77).all(), i
                continue
            want, s = lr.entry(k[i * self.page:i * self.page + most[i]])
            assert (scales[at] == s).all(), (i, most[i], scales[at], s)
            assert (codes[at] == np.stack(want)).all(), (i, most[i])
        for _ in range(3):
            again = self.update()
            assert (again[0] == codes).all() and (again[1] == scales).all()


@pytest.mark.parametrize("lens", [[48, 35, 41, 17], [17, 41, 35, 48], [35, 41, 17, 33], [1, 0, 2, 15], [47, 47, 46, 47]])
@pytest.mark.parametrize("storage,dim", [("16bit", 64), ("16bit", 128), ("16bit", 200), ("mxfp8", 96), ("mxfp4", 128)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_forks(T, L, dtype, storage, dim, lens):
    """Sequences that go on from one prompt and count different numbers of its tokens."""
    Shared(T, L, 48, 2, dim, 16, storage, dtype, [[0, 1, 2]] * 4, lens).check()


@pytest.mark.parametrize("page", [2, 24, 256])
def test_one_page_twice_in_a_table(T, L, page):
    """A sequence's last page, of which it has a part there and all of it further in front, and two such sequences."""
    Shared(T, L, 3 * page, 2, 128, page, "16bit", "bf16", [[0, 1, 2, 1]], [3 * page + 1]).check()
    Shared(T, L, 3 * page, 2, 128, page, "16bit", "bf16", [[0, 1, 2, 1], [2, 0]],
           [3 * page + page // 2, page + 1]).check()
    Shared(T, L, 3 * page, 2, 128, page, "16bit", "bf16", [[1], [2, 1]], [page // 2, page + 1]).check()


def test_a_step(T, L):
    """One new token each: only the places from `starts` on count, so a page can have fewer tokens than elsewhere."""
    s = Shared(T, L, 64, 2, 64, 16, "16bit", "bf16", [[0, 1, 2, 3]] * 5, [64, 35, 34, 33, 17], [63, 34, 33, 32, 16])
    assert s.most() == {3: 16, 2: 3, 1: 1}
    s.check()
    s = Shared(T, L, 64, 2, 64, 16, "16bit", "bf16", [[0, 1, 2, 3]] * 4, [64, 35, 35, 9], [20, 35, 40, -3])
    assert s.most() == {1: 16, 2: 16, 3: 16, 0: 9}
    s.check()


@pytest.mark.parametrize("batch", [255, 256, 257, 700])
def test_many_sequences(T, L, batch):
    """More sequences than a workgroup has threads; every page is the last of many."""
    r = np.random.RandomState(batch)
    places = [r.randint(0, 9, 3).tolist() for _ in range(batch)]
    lens = r.randint(0, 49, batch).tolist()
    Shared(T, L, 9 * 16, 1, 64, 16, "16bit", "f16", places, lens).check()
    Shared(T, L, 9 * 16, 1, 64, 16, "mxfp8", "bf16", places, lens, [n - 1 for n in lens]).check()


@pytest.mark.parametrize("at", [0, 255, 256, 2047, 2048, 2049, 4999])
def test_long_tables(T, L, at):
    """A sequence ends in a page that another has, full, far in front of its end; alone it has the page for itself."""
    whole = list(range(5001))
    for other in ([whole], [[5000], whole], [whole, [5000]] + [[5000]] * 70):
        places = other + [[5000, at]]
        lens = [len(p) * 2 for p in other] + [3]
        Shared(T, L, 5001 * 2, 1, 32, 2, "mxfp4", "bf16", places, lens, seed=at).check()
    Shared(T, L, 5001 * 2, 1, 32, 2, "16bit", "bf16", [whole[:at] + whole[at + 1:], [5000, at]], [10000, 3],
           seed=at).check()


def test_selection_of_forks(T, L):
    """What is selected for sequences that share pages is what the whole entries give."""
    s = Shared(T, L, 12 * 16, 2, 64, 16, "16bit", "bf16", [list(range(12))] * 3, [192, 183, 150], seed=5)
    s.check()
    q = s.pool.q(3, 8)
    table, tokens = s.index.select(q, s.table, s.lens, 5)
    most, x = s.most(), ref.f64(q)
    for b, n in enumerate(s.n):
        m = -(-n // 16)
        made = [lr.entry(s.pool.k[0][16 * i:16 * i + most[i]]) for i in range(m)]
        for h in range(2):
            got = lr.scores(x[b, 4 * h:4 * h + 4], np.stack([c[h] for c, _ in made]),
                            np.array([e[h] for _, e in made]))
            which = lr.highest(list(got), [True] * m, 1, 2, 5)
            assert table[b, h].tolist() == [s.pool.pages[0][i] for i in which], (b, h)
        assert tokens[b] == 4 * 16 + n - 16 * (m - 1)
