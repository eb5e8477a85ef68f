"""Rotary positions and the paged cache on the GPU against 64-bit references.

Tolerances. Rotary: a result is rounded once, half a unit of the 16-bit type (2^-8 or 2^-11 of its
magnitude, at most), after 32-bit work: the angle is exact to 2^-26 turns (1e-7), the hardware's sine
and cosine to 2^-20 (1e-6) or better, the products to 2^-23: 4e-6 of |x1| + |x2| in all. Cache: codes,
scale bytes and what reads back are exact."""
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


def normal(seed, shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(ref.TORCH[dtype]).to(DEV)


def check_rope(got, x, want, dtype, rot, start, pairing, magnitude=1.0):
    swap = np.abs(x).copy()
    r = swap[..., start:start + rot]
    other = np.roll(r, rot // 2, -1) if pairing == "half" else \
        r.reshape(r.shape[:-1] + (-1, 2))[..., ::-1].reshape(r.shape)
    swap[..., start:start + rot] += other
    tol = ref.HALF_ULP[dtype] * np.abs(want) + 4e-6 * abs(magnitude) * swap + ref.TINY[dtype]
    assert (np.abs(ref.f64(got) - want) <= tol).all()


CASES = [  # tokens, heads, dim, rot, start, pairing
    (1, 1, 128, 128, 0, "half"), (1, 9, 64, 64, 0, "interleaved"), (3, 5, 80, 40, 0, "interleaved"),
    (7, 3, 96, 32, 64, "half"), (5, 2, 64, 20, 0, "half"), (5, 2, 64, 20, 6, "interleaved"),
    (2, 4, 2, 2, 0, "half"), (2, 3, 33, 6, 5, "interleaved"), (4, 1, 256, 256, 0, "half"),
    (2, 2, 576, 64, 512, "interleaved"), (2, 2, 1024, 512, 3, "half"), (300, 70, 128, 128, 0, "half"),
    (1100, 33, 128, 64, 0, "interleaved"), (1, 1, 18, 14, 1, "half"),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,heads,dim,rot,start,pairing", CASES)
def test_rope(T, dtype, tokens, heads, dim, rot, start, pairing):
    x = normal(1, (tokens, heads, dim), dtype)
    pos = torch.randint(0, 1 << 17, (tokens,), generator=torch.Generator().manual_seed(2)).to(DEV)
    r = T.Rope(dim, rot_dim=rot, rot_start=start, pairing=pairing, dtype=dtype)
    th = ref.thetas(rot)
    for gradient in (False, True):
        got = (r.grad if gradient else r.run)(x, pos)
        want = ref.rope(ref.f64(x), pos.cpu().numpy(), th, rot, start, pairing, gradient=gradient)
        check_rope(got, ref.f64(x), want, dtype, rot, start, pairing)
        y = x.clone()   # in place: the same bits
        assert (r.grad if gradient else r.run)(y, pos, out=y) is y
        assert torch.equal(y.view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("kw", [
    dict(scaling="linear", factor=4.0), dict(scaling="base", factor=4.0),
    dict(scaling="turns", factor=8.0, original_len=8192.0),
    dict(scaling="index", factor=16.0, original_len=4096.0, high=32.0),
    dict(base=500000.0)])
def test_rope_scaled(T, kw):
    x = normal(3, (50, 2, 128), "f16")
    pos = torch.arange(50, device=DEV) * 2617
    r = T.Rope(128, dtype="f16", magnitude=1.25, **kw)
    th = ref.thetas(128, **kw)
    assert r.thetas() == pytest.approx(th, rel=1e-13)
    want = ref.rope(ref.f64(x), pos.cpu().numpy(), th, 128, magnitude=1.25)
    check_rope(r.run(x, pos), ref.f64(x), want, "f16", 128, 0, "half", 1.25)


def test_rope_far_and_negative_positions(T):
    """Angles stay exact where a 32-bit product would lose them: positions to 2^40 and below 0."""
    pos = torch.tensor([0, 1, -1, (1 << 24) + 1, (1 << 31) + 7, -(1 << 33) - 5, (1 << 40) + 3], device=DEV)
    x = normal(4, (len(pos), 2, 64), "f16")
    th = [0.5 ** i for i in range(32)]     # exact doubles, so the reference has the same angles
    r = T.Rope(64, dtype="f16", thetas=th)
    want = ref.rope(ref.f64(x), pos.cpu().numpy(), th, 64)
    check_rope(r.run(x, pos), ref.f64(x), want, "f16", 64, 0, "half")


def test_rope_views_and_batches(T):
    """Strided heads of a fused projection, odd addresses, an expanded input, batches with shared and
    own positions, another stream; nothing around the output is written."""
    r = T.Rope(64, dtype="bf16")
    th = ref.thetas(64)
    qkv = normal(5, (6, 9, 64), "bf16")
    x, pos = qkv[:, 2:7], torch.arange(100, 106, device=DEV)
    want = ref.rope(ref.f64(x), pos.cpu().numpy(), th, 64)
    big = torch.full((6, 9, 67), 7.0, dtype=torch.bfloat16, device=DEV)
    out = big[:, 1:6, 3:]
    r.run(x, pos, out=out)
    check_rope(out, ref.f64(x), want, "bf16", 64, 0, "half")
    rest = big.clone()
    rest[:, 1:6, 3:] = 7.0
    assert (rest == 7.0).all()
    one = normal(6, (1, 1, 64), "bf16").expand(6, 5, 64)
    want = ref.rope(ref.f64(one), pos.cpu().numpy(), th, 64)
    check_rope(r.run(one, pos), ref.f64(one), want, "bf16", 64, 0, "half")
    xb = normal(7, (3, 5, 6, 64), "bf16").transpose(1, 2)      # [batch, tokens, heads, dim] view
    for p in (pos, torch.arange(18, device=DEV).view(3, 6) * 11):
        want = ref.rope(ref.f64(xb), np.broadcast_to(p.cpu().numpy(), (3, 6)), th, 64)
        check_rope(r.run(xb, p), ref.f64(xb), want, "bf16", 64, 0, "half")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = r.run(xb, p, stream=s)
    s.synchronize()
    check_rope(got, ref.f64(xb), want, "bf16", 64, 0, "half")


def test_rope_gradient_against_differences(T):
    """R is linear: column j of it is R(x + e_j) - R(x), which the gradient's matrix transposes. With
    x = 0 the differences are the rounded columns themselves."""
    r = T.Rope(16, rot_dim=10, rot_start=4, pairing="interleaved", dtype="f16", magnitude=1.5)
    pos = torch.full((16,), 12345, device=DEV)
    eye = torch.eye(16, dtype=torch.float16, device=DEV)[:, None]
    m, mt = ref.f64(r.run(eye, pos))[:, 0], ref.f64(r.grad(eye, pos))[:, 0]
    assert np.abs(m.T - mt).max() <= 2 * 2.0 ** -11 * 1.5 + 8e-6
    dy = normal(8, (16, 1, 16), "f16")
    want = ref.f64(dy)[:, 0] @ m.T      # dx = R^T dy, rows
    assert np.abs(ref.f64(r.grad(dy, pos))[:, 0] - want).max() <= \
        16 * 2.0 ** -11 * 1.5 * np.abs(ref.f64(dy)).max()


def test_rope_refusals(T):
    r = T.Rope(64, dtype="bf16")
    x, pos = normal(9, (2, 3, 64), "bf16"), torch.arange(2, device=DEV)
    for bad in (x.half(), x.cpu(), x[..., :32], x[0], x.transpose(1, 2)):
        with pytest.raises(ValueError):
            r.run(bad, pos)
    for bad in (pos.int(), pos[:1], pos.cpu()):
        with pytest.raises(ValueError):
            r.run(x, bad)
    assert r.run(x[:0], pos[:0]).shape == (0, 3, 64) and r.run(x[:, :0], pos).shape == (2, 0, 64)
    with pytest.raises(ValueError):
        T.Rope(64, pairing="quarter")
    with pytest.raises(T.AgmmError):
        T.Rope(64, rot_dim=63)


# ---- the cache ----

def bits(t):
    return t.contiguous().view(torch.int16).cpu()


def hard_rows(dtype, heads, dim, seed):
    """Rows of 16-bit values of every scale, with what is hard to quantise among them."""
    td = ref.TORCH[dtype]
    x = torch.randn((24, heads, dim), generator=torch.Generator().manual_seed(seed))
    x = x * torch.exp2(torch.arange(24).float()[:, None, None] * (1.4 if dtype == "f16" else 10) -
                       (18.0 if dtype == "f16" else 120.0))
    x = x.to(td)
    f = torch.finfo(td)
    x[0] = 0
    x[1] = -0.0
    x[2, :, 5] = f.max
    x[3, :, 5:9] = -f.max
    x[4, :, 7] = float("nan")
    x[5, :, min(31, dim - 1)] = float("inf")
    x[6, :, 0] = float("-inf")
    x[7] = f.smallest_normal / 4
    x[8, 0] = torch.arange(dim).to(td) / 16            # ties on both grids
    x[9, 0] = torch.arange(dim).to(td) / 4 - 7
    x[10, :, 3], x[10, :, 4] = 448.0, 449.0
    x[11, 0, :32] = torch.linspace(-6, 6, 32).to(td)[:dim]
    x[12, 0, :32] = torch.tensor([448.0] + [2.0 ** -9 * i / 2 for i in range(31)]).to(td)[:dim]
    x[13] = 0
    x[13, :, 1] = f.smallest_normal * f.eps            # the least subnormal
    return x


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("storage,dim,page,heads", [
    ("16bit", 8, 1, 1), ("16bit", 72, 7, 3), ("16bit", 128, 16, 2), ("mxfp8", 32, 16, 1),
    ("mxfp8", 128, 5, 2), ("mxfp8", 160, 16, 3), ("mxfp4", 32, 8, 1), ("mxfp4", 96, 16, 2),
    ("mxfp4", 256, 64, 2)])
def test_cache_codes_and_read(T, dtype, storage, dim, page, heads):
    k, v = hard_rows(dtype, heads, dim, 1), hard_rows(dtype, heads, dim, 2).flip(0).contiguous()
    tokens = len(k)
    pages = 3 * tokens // page + 2
    cache = T.PagedCache.empty(pages, page, heads, dim, dtype=dtype, storage=storage)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:
            t.view(torch.uint8).fill_(0xA5)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:tokens]
    slots[14], slots[15] = -1, pages * page
    kept = [i for i in range(tokens) if i not in (14, 15)]
    cache.append(k.to(DEV), v.to(DEV), slots.to(DEV))
    ko, vo = cache.read(slots.to(DEV))
    for pool, scale, x, back in ((cache.k, cache.k_scale, k, ko), (cache.v, cache.v_scale, v, vo)):
        rows = pool.transpose(1, 2).reshape(pages * page, heads, -1).cpu()
        at = slots[kept]
        if storage == "16bit":
            assert torch.equal(bits(rows[at]), bits(x[kept]))
            want = x.clone()
        else:
            codes, scales = ref.quantise(ref.f64(x), storage, dtype)
            n = dim // 32
            srows = scale.transpose(1, 2).reshape(pages * page, heads, -1).cpu().numpy()
            assert np.array_equal(srows[at][..., :n], scales[kept])
            fine = np.repeat(scales[kept] != 255, codes.shape[-1] // n, -1)
            assert np.array_equal(rows[at].numpy()[fine], codes[kept][fine])
            want = torch.from_numpy(ref.dequantise(codes, scales, storage)).to(ref.TORCH[dtype])
        want[[14, 15]] = 0
        back = back.cpu()
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(back), nan)
        assert torch.equal(bits(back)[~nan], bits(want)[~nan])
        # rows that no token had stay as they were
        others = np.setdiff1d(np.arange(pages * page), at.numpy())
        raw = pool.view(torch.uint8).transpose(1, 2).reshape(pages * page, heads, -1).cpu()
        assert (raw[others] == 0xA5).all()


@pytest.mark.parametrize("storage", ["16bit", "mxfp8", "mxfp4"])
def test_cache_strided(T, storage):
    """A pool laid out [pages, page, heads, row], inputs that are views of one projection at an odd
    address, and outputs that are views: the same values as dense ones."""
    dim, heads, page, pages, tokens = 64, 3, 8, 6, 29
    flat = normal(11, (tokens * (2 * heads) * dim + 1,), "bf16")[1:]
    kv = flat.view(tokens, 2 * heads, dim)
    k, v = kv[:, :heads], kv[:, heads:]
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(4))[:tokens].to(DEV)
    a = T.PagedCache.empty(pages, page, heads, dim, storage=storage)
    a.append(k.contiguous(), v.contiguous(), slots)
    parts = [torch.zeros((pages, page, heads, t.shape[-1]), dtype=t.dtype, device=DEV).transpose(1, 2)
             for t in (a.k, a.v, a.k_scale, a.v_scale) if t is not None]
    b = T.PagedCache(*parts, storage=storage)
    b.append(k, v, slots)
    for x, y in ((a.k, b.k), (a.v, b.v)):
        assert torch.equal(x, y)
    ka, va = a.read(slots)
    out = torch.empty((tokens, 2 * heads, dim), dtype=torch.bfloat16, device=DEV)
    kb, vb = b.read(slots, k_out=out[:, heads:], v_out=out[:, :heads])
    assert torch.equal(ka, kb) and torch.equal(va, vb) and torch.equal(out[:, heads:], ka)


@pytest.mark.parametrize("storage,dim,kw", [
    ("16bit", 128, {}), ("16bit", 72, dict(rot_dim=20, rot_start=3)), ("mxfp8", 128, {}),
    ("mxfp8", 96, dict(rot_dim=48, pairing="interleaved")), ("mxfp4", 64, dict(rot_dim=32)),
    ("mxfp4", 256, dict(rot_dim=70, rot_start=9)), ("16bit", 64, dict(rot_dim=6, pairing="interleaved", rot_start=1))])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tokens", [1, 37])
def test_append_rope_is_rope_then_append(T, storage, dim, kw, dtype, tokens):
    heads, q_heads, page = 2, 6, 16
    qkv = normal(13, (tokens, q_heads + 2 * heads, dim), dtype)
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:]
    pos = torch.arange(tokens, device=DEV) * 977 + 5
    slots = torch.randperm(64, generator=torch.Generator().manual_seed(5))[:tokens].to(DEV)
    if tokens > 1:
        slots[3] = -1
    r = T.Rope(dim, dtype=dtype, **kw)
    a, b = (T.PagedCache.empty(4, page, heads, dim, dtype=dtype, storage=storage) for _ in "ab")
    qa = r.run(q, pos)
    a.append(r.run(k, pos), v, slots)
    qb = b.append_rope(r, q, k, v, pos, slots)
    assert torch.equal(bits(qa), bits(qb))
    for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
        assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    b.append_rope(r, q, k, v, pos, slots, q_out=q)      # in place
    assert torch.equal(bits(qa), bits(q))


def test_cache_refusals(T):
    c = T.PagedCache.empty(2, 16, 2, 64, storage="mxfp8")
    k, slots = normal(14, (3, 2, 64), "bf16"), torch.arange(3, device=DEV)
    for bad in (k.half(), k[:, :1], k[:2], k[..., :32], k.cpu()):
        with pytest.raises(ValueError):
            c.append(bad, k, slots)
        with pytest.raises(ValueError):
            c.append(k, bad, slots)
    with pytest.raises(ValueError):
        c.append(k, k, slots.int())
    c.append(k[:0], k[:0], slots[:0])
    assert c.read(slots[:0])[0].shape == (0, 2, 64)
    with pytest.raises(ValueError):
        T.PagedCache(c.k, c.v, dtype="bf16", storage="16bit")
    with pytest.raises(ValueError):
        T.PagedCache(c.k, c.v, c.k_scale, c.v_scale[..., :2], storage="mxfp8")
    with pytest.raises(ValueError):
        T.PagedCache(c.k, c.v.transpose(0, 2).contiguous().transpose(0, 2), c.k_scale, c.v_scale,
                     storage="mxfp8")
    r = T.Rope(128)
    with pytest.raises(T.AgmmError):
        c.append_rope(r, k, k, k, slots, slots)
