"""Results that a run allocates while it is launched on another stream than the current one: they take no
memory that the current stream still uses, and give none back that it still reads. The current stream is
kept busy meanwhile, for some milliseconds at a time."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
CLOCKS = 20_000_000


@pytest.fixture(scope="module")
def T():
    import all_gather_gemm_amd.attention
    return all_gather_gemm_amd.attention


def serving_calls(T):
    g = torch.Generator().manual_seed(1)
    tokens, heads, q_heads, dim, page = 40, 2, 8, 64, 16
    qkv = torch.randn((tokens, q_heads + 2 * heads, dim), generator=g).bfloat16().to(DEV)
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:]
    pos, slots = torch.arange(tokens, device=DEV), torch.arange(tokens, device=DEV)
    rope, cache = T.Rope(dim), T.PagedCache.empty(tokens, page, heads, dim)
    attn = T.DecodeAttention(q_heads, heads, dim)
    table = torch.arange(tokens, dtype=torch.int32, device=DEV)[:, None].contiguous()
    lens = torch.full((tokens,), page, dtype=torch.int32, device=DEV)
    cache.append(k, v, slots)
    return {
        "rope": lambda s: [rope.run(q, pos, stream=s)],
        "grad": lambda s: [rope.grad(q, pos, stream=s)],
        "append_rope": lambda s: [cache.append_rope(rope, q, k, v, pos, slots, stream=s)],
        "read": lambda s: list(cache.read(slots, stream=s)),
        "attention": lambda s: list(attn.run(q, cache, table, lens, return_lse=True, stream=s)),
    }


def check(call):
    want = [t.clone() for t in call(None)]
    call(None)                      # (the cache holds what it will)
    torch.cuda.synchronize()
    s, now = torch.cuda.Stream(), torch.cuda.current_stream()
    # memory that was freed here while the current stream is still to write it
    junk = [torch.empty_like(t) for t in want for _ in range(3)]
    torch.cuda._sleep(CLOCKS)
    for t in junk:
        t.zero_().sub_(7)
    mine = {t.data_ptr() for t in junk}
    del junk, t
    got = call(s)
    assert not mine & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # memory of results that the current stream is still to read
    now.wait_stream(s)
    torch.cuda._sleep(CLOCKS)
    kept = [t.clone() for t in got]
    mine = {t.data_ptr() for t in got}
    del got
    with torch.cuda.stream(s):
        other = [torch.zeros_like(t) for t in want for _ in range(3)]
    assert not mine & {t.data_ptr() for t in other}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))


@pytest.mark.parametrize("name", ["rope", "grad", "append_rope", "read", "attention"])
def test_serving_results(T, name):
    check(serving_calls(T)[name])


@pytest.mark.parametrize("name", ["gather", "finalize", "flags"])
def test_product_results(name):
    import all_gather_gemm_amd as A
    g = torch.Generator().manual_seed(2)
    draw = lambda *n: torch.randn(n, generator=g).half().to(DEV)     # noqa: E731
    D, M, N, K = 2, 256, 256, 256
    if name == "gather":
        op = A.AgMatmul(D, M, N, K, gather_a=True)
        shards, B = [draw(M // D, K) for _ in range(D)], draw(K, N)
        check(lambda s: list(op.run(shards, B, stream=s)))
    elif name == "finalize":
        op = A.GemmAllReduce(D, 0, M, N, K)
        C = torch.randn((M, N), generator=g).to(DEV)
        check(lambda s: [op.finalize(C, stream=s)])
    else:
        op = A.GemmAllReduceFlags(D, M, N, K)
        a, b = [draw(M, K) for _ in range(D)], [draw(K, N) for _ in range(D)]
        check(lambda s: [op.run(a, b, stream=s)])
