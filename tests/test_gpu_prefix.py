"""Attention over shared prefixes on the GPU against a 64-bit reference over each sequence's tokens, prefix
and own ones (tolerances: long_reference.check_attention)."""
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


class Problem:
    """groups: (prefix length, own lengths of its sequences); `before` sequences in front of the first group
    and `behind` after the last have no prefix."""

    def __init__(self, T, L, groups, q_heads, kv_heads, dim, page, storage, dtype, before=(), behind=(), cap=0.0,
                 scale=0.0, num_wgs=0, seed=1, spread=1.0, starts=True, **kw):
        self.before = len(before)
        own = list(before) + [n for _, g in groups for n in g] + list(behind)
        self.pool = lr.Pool(T, [p for p, _ in groups] + own, kv_heads, dim, page, storage, dtype, seed=seed, **kw)
        self.n, self.batch = len(groups), len(own)
        bounds = np.cumsum([len(before)] + [len(g) for _, g in groups]).tolist()
        self.of = [next((g for g in range(self.n) if bounds[g] <= b < bounds[g + 1]), None)
                   for b in range(self.batch)]
        self.starts = torch.tensor(bounds, dtype=torch.int32, device=lr.DEV) if starts else None
        self.runs = range(self.n, self.n + self.batch)
        self.q = self.pool.q(self.batch, q_heads, seed=seed + 100, spread=spread)
        self.dtype, self.cap, self.scale = dtype, cap, scale or 1 / math.sqrt(dim)
        self.attn = L.PrefixAttention(q_heads, kv_heads, dim, dtype=dtype, storage=storage, soft_cap=cap,
                                      scale=scale, num_wgs=num_wgs)
        self.args = (self.q, self.pool.cache, self.pool.table(range(self.n)), self.pool.lengths(range(self.n)),
                     self.pool.table(self.runs), self.pool.lengths(self.runs))

    def run(self, **kw):
        return self.attn.run(*self.args, starts=self.starts, return_lse=True, **kw)

    def tokens(self, b):
        p = self.pool
        runs = ([] if self.of[b] is None else [self.of[b]]) + [self.n + b]
        return tuple(np.concatenate([x[r][p.there(r)] for r in runs]) for x in (p.k, p.v))

    def check(self, out, lse):
        kv = [self.tokens(b) for b in range(self.batch)]
        lr.check_attention(self.dtype, self.q, out, lse, [x for x, _ in kv], [x for _, x in kv], self.scale,
                           self.cap)


GROUPS = [(129, [3, 0, 17]), (0, [5, 0]), (1000, [1, 2, 130, 0, 33]), (1, [0]), (64, [70])]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("storage,dim", [
    ("16bit", 8), ("16bit", 64), ("16bit", 72), ("16bit", 128), ("16bit", 200), ("16bit", 256),
    ("mxfp8", 32), ("mxfp8", 64), ("mxfp8", 96), ("mxfp8", 128), ("mxfp8", 160), ("mxfp8", 256),
    ("mxfp4", 32), ("mxfp4", 64), ("mxfp4", 96), ("mxfp4", 128), ("mxfp4", 224), ("mxfp4", 256)])
def test_types_and_widths(T, L, dtype, storage, dim):
    p = Problem(T, L, GROUPS, 6, 2, dim, 16, storage, dtype, before=[9], behind=[0, 20])
    p.check(*p.run())


@pytest.mark.parametrize("page", [1, 3, 16, 24, 100, 256])
@pytest.mark.parametrize("storage", ["16bit", "mxfp8", "mxfp4"])
def test_page_sizes(T, L, page, storage):
    p = Problem(T, L, [(300, [1, 40]), (77, [5])], 8, 1, 128, page, storage, "bf16", seed=page,
                transposed=page == 24)
    p.check(*p.run())


@pytest.mark.parametrize("q_heads,kv_heads,batch", [(1, 1, 1), (2, 1, 40), (7, 1, 37), (20, 2, 14), (64, 2, 9),
                                                    (40, 1, 16)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_heads_and_rows(T, L, q_heads, kv_heads, batch, dim):
    """Rows of a group under, at and over multiples of a wave's 32 and a strip's 128."""
    p = Problem(T, L, [(513, [b % 5 for b in range(batch)]), (200, [1, 2])], q_heads, kv_heads, dim, 16, "16bit",
                "bf16", seed=batch)
    p.check(*p.run())


@pytest.mark.parametrize("num_wgs", [1, 2, 7, 64, 1000])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_ways_to_share_the_work(T, L, num_wgs, dim):
    """Runs that hold many strips, and strips in many pieces."""
    p = Problem(T, L, [(2500, [3] * 20), (300, [1] * 3), (1, [2]), (1111, [0, 0, 9])], 16, 2, dim, 16, "16bit", "f16",
                num_wgs=num_wgs)
    p.check(*p.run())


def test_many_groups(T, L):
    """More groups than a wave has lanes, some of them empty."""
    groups = [((37 * i) % 150, [i % 3] * (i % 4)) for i in range(150)]
    p = Problem(T, L, groups, 4, 2, 64, 16, "16bit", "bf16", before=[4, 4], behind=[8])
    p.check(*p.run())


@pytest.mark.parametrize("storage", ["16bit", "mxfp4"])
def test_absent_pages(T, L, storage):
    p = Problem(T, L, [(700, [100, 3]), (40, [8, 0, 600])], 8, 2, 64, 8, storage, "bf16", holes=(0, 3, 4, 40))
    p.check(*p.run())
    p = Problem(T, L, [(30, [5, 0])], 8, 2, 64, 8, storage, "bf16", holes=(0, 1, 2, 3))
    p.check(*p.run())


@pytest.mark.parametrize("cap", [0.5, 30.0])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_capped_scores(T, L, cap, dim, dtype):
    p = Problem(T, L, [(700, [40, 3, 0])], 8, 2, dim, 16, "16bit", dtype, cap=cap, spread=8.0)
    p.check(*p.run())


@pytest.mark.parametrize("spread", [0.0, 30.0])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_flat_and_sharp(T, L, spread, dtype):
    p = Problem(T, L, [(1500, [700, 3]), (90, [1500, 0])], 8, 1, 128, 64, "16bit", dtype, spread=spread)
    p.check(*p.run())


def test_without_starts(T, L):
    p = Problem(T, L, [(400, [6, 0, 90])], 8, 2, 128, 16, "16bit", "bf16", starts=False)
    p.check(*p.run())


def test_odd_starts(T, L):
    """Numbers of `starts` outside the batch count as its ends, one below an earlier one as that."""
    p = Problem(T, L, [(100, [6, 0, 90]), (33, []), (64, [4, 4])], 8, 2, 64, 16, "16bit", "bf16", before=[3])
    p.starts = torch.tensor([1, 4, 2, 99], dtype=torch.int32, device=lr.DEV)
    p.check(*p.run())
    p.starts = torch.tensor([-5, -1, -7, 0], dtype=torch.int32, device=lr.DEV)
    p.of = [None] * p.batch
    p.check(*p.run())


def test_odd_lengths(T, L):
    """Negative lengths count as 0; tokens past the tables are left out."""
    p = Problem(T, L, [(96, [32, 16]), (64, [48])], 4, 1, 64, 16, "16bit", "bf16")
    want = p.run()
    a = list(p.args)
    pt, ot = p.pool.table(range(2), extra=0), p.pool.table(p.runs, extra=0)
    a[2], a[4] = pt, ot
    a[3] = torch.tensor([1 << 30, 64], dtype=torch.int32, device=lr.DEV)
    got = p.attn.run(*a, starts=p.starts, return_lse=True)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    a[3] = torch.tensor([-3, -(1 << 31)], dtype=torch.int32, device=lr.DEV)
    got = p.attn.run(*a, starts=p.starts, return_lse=True)
    plain = T.DecodeAttention(4, 1, 64).run(a[0], a[1], a[4], a[5], return_lse=True)
    for x, y in zip(got, plain):   # joined with nothing: another rounding of the same sums
        assert torch.allclose(x.float(), y.float(), rtol=2.0 ** -7, atol=1e-6)


def test_not_finite(T, L):
    """A NaN or an infinity in a prefix's values reaches the sequences that share it, and no other; in pages that
    are absent, none."""
    p = Problem(T, L, [(100, [6, 7]), (100, [5])], 4, 1, 64, 16, "16bit", "bf16")
    page, row = p.pool.pages[0][2], 5
    p.pool.cache.v[page, 0, row, 3] = math.nan
    out, lse = p.run()
    assert torch.isnan(out[:2, :, 3]).all() and torch.isfinite(lse).all()
    assert torch.isfinite(out[2]).all() and torch.isfinite(out[:, :, 4:]).all()
    p.args[2][0, 2] = -1
    out, lse = p.run()
    assert torch.isfinite(out).all()


def test_large_values_stay_finite(T, L):
    """Averages of finite values are finite, up to the type's largest."""
    top = torch.finfo(torch.bfloat16).max
    lens = [600, 300, 40]
    v = torch.full((sum(lens), 1, 64), top)
    p = Problem(T, L, [(600, [300, 40])], 4, 1, 64, 16, "16bit", "bf16", v=v)
    out, _ = p.run()
    assert (out.float() <= top).all() and (out.float() >= top * (1 - 2.0 ** -7)).all()


@pytest.mark.parametrize("power", [10, 20, 22, 23, 24])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_large_scores(T, L, power, dtype):
    """Scores of 2^power and a little, growing from tile to tile, so that the maximum is raised again and again.

    Products are exact: one large element that all keys share and one small one, whose product is a multiple of half
    `step` and so of 2^(power - 23), the last bit of a 32-bit float at 2^power. So scores differ by what the small
    elements say, off by 2^-24 of it for the scale's rounding, and the exponent's own rounding is 2^-19 at 2^5 and less:
    a weight is within 2^-17 of itself. out: half an ulp, and A * (2^-16 + 2^-11 [f16: parts] or 2^-15)."""
    n, dim, step = 640, 64, 2.0 ** max(0, power - 22)
    k = torch.zeros((n + 40, 1, dim))
    k[..., 0] = 2.0 ** (power - 10)
    k[:, 0, 1] = step * (torch.arange(n + 40) // 20 + 2.0 * (torch.arange(n + 40) % 3))
    p = Problem(T, L, [(n, [30, 10])], 4, 1, dim, 16, "16bit", dtype, k=k, scale=1.0)
    p.q.zero_()
    p.q[..., 0] = 2.0 ** 10
    p.q[..., 1] = 0.5
    out, lse = p.run()
    q, out, lse = (x.double().cpu().numpy() for x in (p.q, out, lse))
    part = 2.0 ** -11 if dtype == "f16" else 2.0 ** -15
    for b in range(2):
        kk, vv = p.tokens(b)
        o, s, a, _ = ref.attention(q[b], kk, vv, 1.0)
        assert (np.abs(out[b] - o) <= ref.HALF_ULP[dtype] * np.abs(o) + a * (2.0 ** -16 + part)).all(), b
        # lse: 2^-24 for each of three roundings at its magnitude, and the scale's
        assert (np.abs(lse[b] - s) <= 2.0 ** -21 * (1 + np.abs(s))).all()


def test_repeats_are_equal(T, L):
    p = Problem(T, L, [(3000, [100] * 9), (500, [9, 8])], 16, 2, 128, 16, "mxfp8", "bf16")
    a = p.run()
    for _ in range(5):
        b = p.run()
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured(T, L):
    """A captured run serves lengths that grow."""
    p = Problem(T, L, [(900, [100, 50, 0])], 8, 2, 128, 16, "16bit", "bf16")
    full = p.args[5].clone()
    p.args[5].copy_(full // 2)
    p.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = p.run()
    for lens in (full // 2, full, full // 3):
        p.args[5].copy_(lens)
        g.replay()
        torch.cuda.synchronize()
        want = p.run()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    p.args[5].copy_(full)
    g.replay()
    p.check(out, lse)


def test_another_stream(T, L):
    p = Problem(T, L, [(900, [100, 50, 0])], 8, 2, 128, 16, "16bit", "bf16")
    want = p.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = p.run(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_strided_out(T, L):
    p = Problem(T, L, [(300, [10, 20])], 6, 2, 72, 16, "16bit", "f16")
    wide = torch.full((2, 8, 72), 7.0, dtype=torch.float16, device=lr.DEV)
    out, lse = p.run(out=wide[:, 1:7])
    p.check(out, lse)
    assert (wide[:, 0] == 7).all() and (wide[:, 7] == 7).all()


def test_scales_past_the_range(T, L):
    """Scores would leave the range of 32-bit floats: refused, unless they are capped."""
    for cap in (0.0, 5.0):
        p = Problem(T, L, [(40, [4, 0])], 4, 1, 64, 16, "16bit", "bf16", scale=2.0 ** 64, cap=cap)
        if cap:
            p.run()
        else:
            with pytest.raises(T.AgmmError) as e:
                p.run()
            assert e.value.code == -2


def test_infinite_scores(T, L):
    """A score past the range of floats, as an infinite one, gives NaN for its sequences and no others."""
    p = Problem(T, L, [(100, [6, 7]), (100, [5])], 4, 1, 64, 16, "16bit", "bf16")
    page, row = p.pool.pages[0][2], 5
    for k in (math.inf, 3.0e38):
        p.pool.cache.k[page, 0, row] = k
        p.q.fill_(3.0e38 if k < math.inf else 1.0)
        out, lse = p.run()
        assert torch.isnan(out[:2]).all()
        if k == math.inf:
            assert torch.isfinite(out[2]).all() and torch.isfinite(lse[2]).all()


def test_nothing(T, L):
    p = Problem(T, L, [(30, [4])], 4, 1, 64, 16, "16bit", "bf16")
    q, cache, pt, pl, t, n = p.args
    empty = p.attn.run(q[:0], cache, pt, pl, t[:0], n[:0], starts=p.starts)
    assert empty.shape == (0, 4, 64)
    out, lse = p.attn.run(q, cache, pt[:0], pl[:0], t, n, starts=p.starts[:1], return_lse=True)
    want = T.DecodeAttention(4, 1, 64).run(q, cache, t, n, return_lse=True)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
