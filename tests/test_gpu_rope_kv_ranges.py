"""Rotary positions and the paged cache on the GPU at the ends of what their arguments allow."""
import numpy as np
import pytest
import torch

import attention_reference as ref
from test_gpu_rope_kv import DEV, bits, check_rope, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    import all_gather_gemm_amd.attention
    return all_gather_gemm_amd.attention


@pytest.mark.parametrize("storage", ["16bit", "mxfp8", "mxfp4"])
def test_slots_that_tokens_share(T, storage):
    """What two tokens write to one slot is undefined within that row, every element one of theirs in 16
    bits; all other rows hold what they should."""
    tokens, heads, dim, page, pages = 400, 3, 128, 16, 30
    k, v = normal(21, (tokens, heads, dim), "bf16"), normal(22, (tokens, heads, dim), "bf16")
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(6))[:tokens].to(DEV)
    shared = [(3, 4), (10, 390), (0, 399)]
    for a, b in shared:
        slots[b] = slots[a]
    alone = [t for t in range(tokens) if not any(t in p for p in shared)]
    cache, once = (T.PagedCache.empty(pages, page, heads, dim, storage=storage) for _ in "ab")
    cache.append(k, v, slots)
    once.append(k[alone], v[alone], slots[alone])
    rest = torch.ones(pages * page, dtype=torch.bool, device=DEV)
    rest[[int(slots[a]) for a, _ in shared]] = False
    every = torch.arange(pages * page, device=DEV)[rest]
    for x, y in zip(cache.read(every), once.read(every)):
        assert torch.equal(x, y)
    if storage == "16bit":
        for x, y in zip(cache.read(slots), (k, v)):
            for a, b in shared:
                assert ((x[a] == y[a]) | (x[a] == y[b])).all()


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
def test_rope_in_autograd(T, pairing):
    """A result of an input that requires a gradient has one: R^T of what comes back, and R of R^T's."""
    r = T.Rope(80, rot_dim=40, rot_start=8, pairing=pairing, dtype="f16")
    x, dy = normal(23, (30, 3, 80), "f16"), normal(24, (30, 3, 80), "f16")
    pos = torch.arange(30, device=DEV) * 31
    for there, back in ((r.run, r.grad), (r.grad, r.run)):
        want, dx = there(x, pos), back(dy, pos)
        leaf = x.clone().requires_grad_()
        y = there(leaf, pos)
        assert y.requires_grad and torch.equal(y, want)
        y.backward(dy)
        assert torch.equal(leaf.grad, dx)
        leaf.grad = None                    # a sum's gradient is one expanded element; through views
        there(leaf * 1, pos)[:, 1:].sum().backward()
        ones = torch.ones_like(x)
        ones[:, 0] = 0
        assert torch.equal(leaf.grad, back(ones, pos))
        # on another stream, backward there too
        s = torch.cuda.Stream()
        leaf.grad = None
        s.wait_stream(torch.cuda.current_stream())
        y = there(leaf, pos, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        y.backward(dy)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(leaf.grad, dx)
        # the gradient's own gradient
        dleaf = dy.clone().requires_grad_()
        g, = torch.autograd.grad(there(leaf, pos), leaf, dleaf, create_graph=True)
        g.backward(x)
        assert torch.equal(dleaf.grad, want)
        with pytest.raises(ValueError):
            there(leaf, pos, out=torch.empty_like(x))
        with torch.no_grad():
            assert not there(leaf, pos).requires_grad
            assert torch.equal(there(leaf, pos, out=torch.empty_like(x)), want)
    # a batch that shares its positions
    leaf = normal(25, (2, 30, 3, 80), "f16").requires_grad_()
    r.run(leaf, pos).backward(dy.expand(2, 30, 3, 80))
    assert torch.equal(leaf.grad[0], r.grad(dy, pos)) and torch.equal(leaf.grad[1], leaf.grad[0])


def test_rope_gradient_by_differences(T):
    """(L(x + h e) - L(x - h e)) / 2h of L(x) = sum(w R x): exact but for the roundings of the results, which
    are half an ulp of magnitudes up to 3 each, 16 of them over 2h = 2."""
    r = T.Rope(16, rot_dim=12, rot_start=2, dtype="f16")
    x = (torch.arange(32, device=DEV).view(1, 2, 16) / 16 - 1).half().requires_grad_()
    w = torch.linspace(-1, 1, 32, device=DEV).view(1, 2, 16).half()
    pos = torch.tensor([777], device=DEV)
    (r.run(x, pos).double() * w.double()).sum().backward()
    for i in range(32):
        h = torch.zeros(32, device=DEV, dtype=torch.float16)
        h[i] = 1.0
        with torch.no_grad():
            d = [(r.run(x + s * h.view(1, 2, 16), pos).double() * w.double()).sum() for s in (1, -1)]
        assert abs(float(d[0] - d[1]) / 2 - float(x.grad.view(-1)[i])) <= 2 * 16 * 3 * 2.0 ** -11 / 2


@pytest.mark.parametrize("pairing,rot", [("half", 40), ("half", 20), ("interleaved", 20)])
def test_rope_in_place_through_other_strides(T, pairing, rot):
    """A size of 1 has any stride: an output that is the input's memory is in place whatever it says, and
    pairs that two threads would share otherwise are read before they are written."""
    heads, dim = 70, 96
    r = T.Rope(dim, rot_dim=rot, pairing=pairing, dtype="bf16")
    pos = torch.tensor([4321], device=DEV)
    x = normal(26, (1, heads, dim), "bf16")
    want = r.run(x, pos)
    y = x.clone()
    r.run(y, pos, out=y.as_strided((1, heads, dim), (1, dim, 1)))
    assert torch.equal(y, want)
    one = x[:, :1].clone()      # one head, in a batch of one
    r.run(one, pos, out=one.as_strided((1, 1, dim), (7, 7, 1)))
    assert torch.equal(one, want[:, :1])
    y = x.clone()
    r.run(y[None], pos, out=y.as_strided((1, 1, heads, dim), (3, 5, dim, 1)))
    assert torch.equal(y, want)
    # and in the step in front of the attention
    cache = T.PagedCache.empty(2, 16, 2, dim)
    k, slots = normal(27, (1, 2, dim), "bf16"), torch.tensor([3], device=DEV)
    y = x.clone()
    cache.append_rope(r, y, k, k, pos, slots, q_out=y.as_strided((1, heads, dim), (1, dim, 1)))
    assert torch.equal(y, want)


# More threads than one launch takes (2^30), more batch entries than one grid has: the call is cut into
# launches, the later of which start in the middle of every argument.
PER_LAUNCH = 1 << 30


def test_rope_in_two_launches(T):
    n = PER_LAUNCH + 9
    r = T.Rope(2, dtype="bf16")
    x = torch.empty((n, 1, 2), dtype=torch.bfloat16, device=DEV).normal_(
        generator=torch.Generator(device=DEV).manual_seed(1))
    pos = torch.arange(n, device=DEV)
    y = r.run(x, pos)
    for part in (slice(0, n // 2 + 5), slice(n // 2 + 5, n)):
        assert torch.equal(y[part], r.run(x[part], pos[part]))


def test_rope_of_many_batch_entries(T):
    batch, tokens, heads, dim = 65535 + 70, 3, 2, 16
    r = T.Rope(dim, dtype="f16", rot_dim=12, rot_start=2)
    x = normal(31, (batch, tokens, heads, dim), "f16")
    pos = torch.arange(batch * tokens, device=DEV).view(batch, tokens)
    flat = x.view(-1, heads, dim)
    assert torch.equal(r.run(x, pos).view_as(flat), r.run(flat, pos.view(-1)))
    shared = pos[0].expand(batch, tokens).reshape(-1)
    assert torch.equal(r.grad(x, pos[0]).view_as(flat), r.grad(flat, shared))


def overlapping(n, seed):
    """n rows of 8 elements in n + 7: row t begins at element t."""
    flat = torch.empty(n + 7, dtype=torch.bfloat16, device=DEV).normal_(
        generator=torch.Generator(device=DEV).manual_seed(seed))
    return flat.as_strided((n, 1, 8), (1, 8, 1))


def test_cache_in_two_launches(T):
    n, page, pages = PER_LAUNCH + 40, 16, 20
    k, v = overlapping(n, 2), overlapping(n, 3)
    cache = T.PagedCache.empty(pages, page, 1, 8)
    kept = torch.cat((torch.arange(50), torch.arange(PER_LAUNCH - 50, n))).to(DEV)
    slots = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    slots[kept] = torch.randperm(pages * page, device=DEV)[:len(kept)]
    cache.append(k, v, slots)
    want = cache.read(slots[kept])
    assert torch.equal(want[0], k[kept]) and torch.equal(want[1], v[kept])
    out = cache.read(slots)
    for x, y in zip(out, want):
        assert torch.equal(x[kept], y)
        x[kept] = 0
        assert not any(bool(part.any()) for part in x.split(1 << 27))


def test_append_rope_in_two_launches(T):
    n = PER_LAUNCH // 2 + 40        # two threads a token: a unit of pairs, and one that passes through
    r = T.Rope(8, rot_dim=2, rot_start=6, dtype="bf16")
    q, k, v = (overlapping(n, s) for s in (4, 5, 6))
    pos = torch.arange(n, device=DEV)
    page, pages = 16, 20
    a, b = (T.PagedCache.empty(pages, page, 1, 8) for _ in "ab")
    kept = torch.cat((torch.arange(50), torch.arange(n - 90, n))).to(DEV)
    slots = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    slots[kept] = torch.randperm(pages * page, device=DEV)[:len(kept)]
    q_out = a.append_rope(r, q, k, v, pos, slots, q_out=torch.empty((n, 1, 8), dtype=q.dtype, device=DEV))
    for part in (slice(0, n // 2 + 5), slice(n // 2 + 5, n)):
        assert torch.equal(q_out[part], r.run(q[part].contiguous(), pos[part]))
    b.append(r.run(k[kept], pos[kept]), v[kept], slots[kept])
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


@pytest.mark.parametrize("storage,dim", [("mxfp8", 256), ("mxfp4", 64)])
def test_scales_past_32_bits(T, storage, dim):
    """Scale bytes of pages whose distance from the pool's start does not fit 32 bits."""
    pages, heads, page, apart, tokens = 40, 2, 16, 1 << 28, 500
    near = T.PagedCache.empty(pages, page, heads, dim, storage=storage)
    row = T.PagedCache.scale_bytes(dim)
    pools = [torch.empty(pages * apart, dtype=torch.uint8, device=DEV) for _ in "kv"]
    far = [p.as_strided((pages, heads, page, row), (apart, page * row, row, 1)) for p in pools]
    for t in far:
        t.fill_(255)
    cache = T.PagedCache(torch.zeros_like(near.k), torch.zeros_like(near.v), *far, storage=storage)
    k, v = normal(32, (tokens, heads, dim), "bf16"), normal(33, (tokens, heads, dim), "bf16")
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(7))[:tokens].to(DEV)
    for c in (near, cache):
        c.append(k, v, slots)
    for x, y in zip(near.read(slots), cache.read(slots)):
        assert torch.equal(x, y)
    attn = T.DecodeAttention(4, heads, dim, storage=storage)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None].contiguous()
    lens = torch.tensor([pages * page], dtype=torch.int32, device=DEV)
    q = normal(34, (1, 4, dim), "bf16")
    every = torch.arange(pages * page, device=DEV)
    empty = every[~torch.isin(every, slots)]
    for c in (near, cache):     # rows that nothing wrote: zeros in both
        c.append(torch.zeros((len(empty), heads, dim), dtype=k.dtype, device=DEV),
                 torch.zeros((len(empty), heads, dim), dtype=k.dtype, device=DEV), empty)
    assert torch.equal(attn.run(q, near, table, lens), attn.run(q, cache, table, lens))
