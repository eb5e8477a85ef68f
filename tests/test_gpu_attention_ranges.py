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


@pytest.mark.parametrize("scale", [1e-44, 1e-30, 1e38, 3.4e38])
def test_scales(T, scale):
    """Scales at the ends of 32 bits: the softmax of zeros, and of zeros and one key that is far above
    the others at the large scales and like them at the small ones."""
    p = Problem(T, [1, 40, 300], 2, 1, 64, 16, "16bit", "bf16", scale=scale)
    k = np.zeros_like(p.k)
    p.q = torch.zeros_like(p.q)
    p.q[..., 0] = 1.0
    refill(p, k=k)
    p.check(*p.run())
    ends = np.cumsum(p.lens)
    k[ends - 1, 0, 0] = 0.5
    refill(p, k=k)
    out = ref.f64(p.run()[0])
    for b, (n, end) in enumerate(zip(p.lens, ends)):
        want = p.v[end - 1, 0] if scale > 1 else p.v[end - n:end, 0].mean(0)
        # half an ulp, and of an average of normal values the 16 bits of a weight
        assert (np.abs(out[b] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -14).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_large_scores(T, dtype):
    """Scores of 2^20 to 2^32, where 32 bits hold them to no more than a whole number: the tokens with the
    largest key share the weight, whatever the order, and the others get none."""
    n, heads = 700, 24
    p = Problem(T, [n], heads, 1, 64, 16, "16bit", dtype, scale=1.0)
    p.q = torch.zeros_like(p.q)
    p.q[0, :, 0] = torch.exp2(torch.arange(heads) / 2 + 4).to(p.q.dtype)     # 2^4 to 2^15.5
    # (a step between keys is 256: 2^12 in a score)
    k = np.zeros_like(p.k)
    k[:, 0, 0] = 256.0 * np.random.default_rng(1).integers(-200, 200, n)
    for top in ([5], [650], [3, 70, 699]):
        k[top, 0, 0] = 256.0 * 220
        refill(p, k=k)
        out, lse = p.run()
        want, s = p.v[top, 0].mean(0), ref.f64(p.q)[0, :, 0] * 256 * 220 + math.log(len(top))
        assert (np.abs(ref.f64(out)[0] - want) <= ref.HALF_ULP[dtype] * np.abs(want) + 2.0 ** -10).all()
        assert (np.abs(ref.f64(lse)[0] - s) <= 2.0 ** -21 * (1 + np.abs(s))).all()
        k[top, 0, 0] = 0.0


LENS = [1, 2, 0, 300, 9000]


@pytest.mark.parametrize("storage", ["16bit", "mxfp8"])
@pytest.mark.parametrize("spread", [1.0, 6.0])
@pytest.mark.parametrize("size", [2.0 ** -100, 1e30, 2.0 ** 126.9])
def test_bf16_values_of_every_size(T, storage, spread, size):
    """Averages of finite values are finite: no sum on the way exceeds 32 bits. (Of values of one sign,
    so that the average is as large as they are.)"""
    p = Problem(T, LENS, 4, 2, 64, 16, storage, "bf16", spread=spread)
    v = size * (1.0 + np.random.default_rng(2).random(p.v.shape))
    refill(p, v=v)
    out, lse = p.run()
    assert torch.isfinite(out).all()
    p.check(out, lse)


def test_bf16_largest_values(T):
    """The largest value in every token comes out as it went in."""
    p = Problem(T, LENS, 4, 2, 64, 16, "16bit", "bf16")
    most = float(torch.finfo(torch.bfloat16).max)
    refill(p, v=np.full_like(p.v, -most))
    out, _ = p.run()
    assert all((out[b] == (-most if n else 0.0)).all() for b, n in enumerate(p.lens))


def test_no_weight_is_none(T):
    """Tokens whose score is minus infinity get no weight at all, however large their values are."""
    for dtype in ("bf16", "f16"):
        n = 200
        p = Problem(T, [n], 2, 1, 64, 16, "16bit", dtype)
        p.q = torch.zeros_like(p.q)
        p.q[..., 0] = 1.0
        most = float(torch.finfo(ref.TORCH[dtype]).max)
        k, v = p.k.copy(), p.v * 1e-3
        k[50:, 0, 0] = -math.inf
        v[50:] = most
        refill(p, k=k, v=v)
        out, lse = p.run()
        p.lens, p.k, p.v = [50], p.k[:50], p.v[:50]
        p.check(out, lse)


@pytest.mark.parametrize("storage,dim", [("16bit", 8), ("16bit", 256), ("mxfp8", 32), ("mxfp4", 64)])
@pytest.mark.parametrize("lens", [[2], [64, 1000]])
def test_f16_weights_in_two_parts(T, storage, dim, lens):
    """Values of one magnitude and alternating signs, weights almost alike: the result is a small part of
    A = sum p |v| and shows what the weights lose in the product. 22 bits of a weight leave 2^-22 of A and
    the sums 2^-18 as elsewhere; 11 bits would leave up to 2^-12."""
    p = Problem(T, lens, 4, 1, dim, 16, storage, "f16", scale=2.0 ** -10)
    v = np.ones_like(p.v)
    v[1::2] = -1.0
    refill(p, v=v)
    q, out = ref.f64(p.q), ref.f64(p.run()[0])
    at = 0
    for b, n in enumerate(lens):
        o, _, a, w = ref.attention(q[b], p.k[at:at + n], p.v[at:at + n], p.scale)
        at += n
        err = (dim + 8) * 2.0 ** -24 * w[:, None]
        tol = ref.HALF_ULP["f16"] * np.abs(o) + a * (2 * err + 2.0 ** -22 + 2.0 ** -18) + ref.TINY["f16"]
        assert (np.abs(out[b] - o) <= tol).all(), (np.abs(out[b] - o) / tol).max()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("keys", ["alike", "random"])
def test_infinite_values_of_any_weight(T, dtype, keys):
    """An infinite value makes its element infinite and no other, also where its weight is a power of 2
    and the second part has nothing of it."""
    n, dim = 300, 64
    p = Problem(T, [n], 2, 1, dim, 16, "16bit", dtype)
    k, v = (np.zeros_like(p.k) if keys == "alike" else p.k), p.v.copy()
    v[7, 0, 3], v[250, 0, 9] = math.inf, -math.inf
    refill(p, k=k, v=v)
    out, _ = p.run()
    assert torch.isposinf(out[0, :, 3]).all() and torch.isneginf(out[0, :, 9]).all()
    rest = [e for e in range(dim) if e not in (3, 9)]
    assert torch.isfinite(out[0][:, rest]).all()
