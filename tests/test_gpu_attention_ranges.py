"""Single-token attention on the GPU at the ends of its arguments' and values' ranges, against the
64-bit reference. Tolerances are those of test_gpu_attention.py's check, which has no term for
the cap or for the values' magnitude, unless a test says otherwise."""
import math

import numpy as np
import pytest
import torch

import attention_reference as ref
from test_gpu_attention import DEV, EDGES, Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    import all_gather_gemm_amd.attention
    return all_gather_gemm_amd.attention


def refill(p, k=None, v=None):
    """Other keys or values [tokens, kv_heads, dim] (float64) for the sequences of a problem."""
    td = ref.TORCH[p.dtype]
    slots, table = [], p.table.cpu()
    for b, n in enumerate(p.lens):
        slots += [int(table[b, i // p.page]) * p.page + i % p.page for i in range(n)]
    slots = torch.tensor(slots, dtype=torch.int64, device=DEV)
    k, v = (torch.from_numpy(x).to(td).to(DEV) for x in
            (p.k if k is None else k, p.v if v is None else v))
    p.cache.append(k, v, slots)
    k, v = p.cache.read(slots)
    p.k, p.v = ref.f64(k), ref.f64(v)


# A score's cap * tanh is a handful of 32-bit roundings of the score itself, which the 32-bit sum's
# bound (dim + 8 of them) covers, whatever the cap; from 1e5 on it is the score.
@pytest.mark.parametrize("cap", [1e-30, 0.01, 2.0, 30.0, 50.0, 1e3, 1e5, 1e8, 2.4e38, 3.4e38])
@pytest.mark.parametrize("dtype,storage,dim", [("f16", "16bit", 8), ("bf16", "16bit", 128), ("bf16", "mxfp4", 64)])
def test_caps(T, cap, dtype, storage, dim):
    cap = float(np.float32(cap))
    p = Problem(T, EDGES, 4, 2, dim, 16, storage, dtype, cap=cap, spread=2.0)
    p.check(*p.run())


def test_caps_of_infinite_and_nan_scores(T):
    """An infinite score is the cap, with its sign; a NaN one makes the row NaN."""
    n, dim, cap = 200, 64, 5.0
    p = Problem(T, [n], 2, 1, dim, 16, "16bit", "bf16", cap=cap, scale=1.0)
    p.q = torch.zeros_like(p.q)
    p.q[..., 0] = 1.0
    k = p.k.copy()
    k[:70, 0, 0], k[150:, 0, 0] = math.inf, -math.inf
    refill(p, k=k)
    out, lse = p.run()
    finite = k.copy()
    finite[:70, 0, 0], finite[150:, 0, 0] = 100 * cap, -100 * cap     # tanh is 1 there
    p.k = finite
    p.check(out, lse)
    k[100, 0, 7] = math.nan
    refill(p, k=k)
    out, lse = p.run()
    assert torch.isnan(out).all() and torch.isnan(lse).all()
