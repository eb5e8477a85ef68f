"""Accumulated attention weights where keys hold infinities, and q heads that add nothing, on the GPU.

Tolerance: test_gpu_evict's, with w over the finite keys (an infinite one's score is -infinity, or its cap, with no
error)."""
import math

import numpy as np
import pytest
import torch

import attention_reference as ref
import long_reference as lr
from test_gpu_evict import Masses

pytestmark = pytest.mark.gpu

AT = 5          # the element that is infinite in some keys, and above 0 in every q


@pytest.fixture(scope="module")
def T():
    import all_gather_gemm_amd.attention
    return all_gather_gemm_amd.attention


@pytest.fixture(scope="module")
def L():
    import all_gather_gemm_amd.long_context
    return all_gather_gemm_amd.long_context


class Infinite(Masses):
    """Every seventh key is -infinity in one element; with a cap every eleventh +infinity."""

    def __init__(self, T, L, lens, q_heads, kv_heads, dim, dtype, cap=0.0, **kw):
        g = torch.Generator().manual_seed(9)
        k = torch.randn((sum(lens), kv_heads, dim), generator=g)
        k[3::7, :, AT] = -math.inf
        if cap:
            k[1::11, :, AT] = math.inf
        super().__init__(T, L, lens, q_heads, kv_heads, dim, 16, "16bit", dtype, cap=cap, k=k, **kw)
        self.q[..., AT] = self.q[..., AT].abs() + 0.5
        attn = T.DecodeAttention(q_heads, kv_heads, dim, dtype=dtype, soft_cap=cap, window=self.window)
        _, self.lse = attn.run(self.q, self.pool.cache, self.table, self.lens, return_lse=True)

    def check(self, got):
        q, lse, old, got = ref.f64(self.q), ref.f64(self.lse), ref.f64(self.mass), ref.f64(got)
        hk, dim = self.pool.kv_heads, self.pool.dim
        group = q.shape[1] // hk
        assert np.isfinite(lse).all()
        for b in self.runs:
            n = self.pool.lens[b]
            seen = np.arange(n) >= (max(0, n - self.window) if self.window else 0)
            for h in range(hk):
                qh, x = q[b, h * group:(h + 1) * group], lse[b, h * group:(h + 1) * group]
                k = self.pool.k[b][:, h]
                fine = np.isfinite(k).all(1)
                s = np.where(np.isfinite(k), k, 0.0) @ qh.T * self.scale
                w = (np.abs(k[fine]) @ np.abs(qh).T).max(initial=0.0) * self.scale
                s[~fine] = np.sign(k[~fine, AT])[:, None] * math.inf
                if self.cap:
                    s = self.cap * np.tanh(s / self.cap)
                p = np.where(seen[:, None], np.exp(s - x), 0.0)
                want = self.decay * old[b, h, :n] + p.sum(1)
                size = np.where(np.isfinite(s), np.abs(s), 0.0) + np.abs(x)
                err = (p * (2 * (dim + 8) * 2.0 ** -24 * w + 2.0 ** -22 * size + 2.0 ** -20)).sum(1)
                tol = err + (group + 2) * 2.0 ** -24 * np.abs(want)
                assert (np.abs(got[b, h, :n] - want) <= tol).all(), (b, h)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (14, 2), (16, 1), (17, 1), (33, 1)])
@pytest.mark.parametrize("kw", [dict(), dict(cap=5.0), dict(window=50)])
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
def test_infinite_keys(T, L, dtype, q_heads, kv_heads, kw, dim):
    m = Infinite(T, L, [100, 1, 37, 300], q_heads, kv_heads, dim, dtype, **kw)
    m.check(m.add())


@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("group", [2, 7, 16, 19])
def test_heads_that_add_nothing(T, L, group, bad, cap):
    """A log-sum-exp of -infinity adds nothing, whatever its head's q gives."""
    m = Masses(T, L, [40, 3], group, 1, 64, 16, "16bit", "bf16", cap=cap)
    off = [1] if group < 17 else [1, 17]
    m.lse[:, off] = -math.inf
    want = m.add()
    m.q[:, off] = bad
    assert torch.equal(m.add(), want)
    assert torch.isfinite(want).all()


@pytest.mark.parametrize("group", [1, 7, 17])
def test_only_infinite_keys(T, L, group):
    """All scores -infinity: no weights, so nothing is added."""
    k = torch.full((20, 1, 64), 1.0)
    k[:, :, AT] = -math.inf
    m = Masses(T, L, [20], group, 1, 64, 16, "16bit", "f16", k=k)
    m.q[..., AT] = m.q[..., AT].abs() + 0.5
    m.lse = T.DecodeAttention(group, 1, 64, dtype="f16").run(m.q, m.pool.cache, m.table, m.lens, return_lse=True)[1]
    assert (m.lse == -math.inf).all()
    assert torch.equal(m.add()[:, :, :20], m.mass[:, :, :20] * m.decay)


def test_kept_tokens(T, L):
    """What got no weight is not kept for a mass that is not a number."""
    m = Infinite(T, L, [64], 7, 1, 64, "bf16", decay=0.0)
    mass = m.add()
    _, kept, new = L.Evictor(16, sink=0, recent=0).choose(m.pool.cache, m.table, m.lens, mass)
    assert torch.isfinite(new).all()
    assert set(kept[0, 0].tolist()) == set(torch.topk(mass[0, 0, :64], 16).indices.tolist())
    assert not set(kept[0, 0].tolist()) & set(range(3, 64, 7))
