"""Single-token attention in each of its ways to share out the work: batches of many short heads, where each
wave works by itself, with long heads among them that many waves share, in every type, storage and
width; joins just below and above what is done at once; many empty sequences in front. Tolerances:
test_gpu_attention.py's."""
import pytest
import torch

from test_gpu_attention import Problem

pytestmark = pytest.mark.gpu
TILE, SINGLE, GROUP = 128, 32, 16


@pytest.fixture(scope="module")
def T():
    import all_gather_gemm_amd.attention
    return all_gather_gemm_amd.attention


def shares(p, kv_heads):
    """How a run of this problem divides its work, by the kernel's rules from the lengths: (whether each wave
    works by itself, pieces of the longest head)."""
    dim, storage, attn = p.q.shape[-1], p.storage, p.attn.desc
    heads = kv_heads * -(-(attn.q_heads // attn.kv_heads) // 16)
    tiles = []
    for n in p.lens:
        first = max(0, n - p.window) if p.window else 0
        tiles.append(-(-(n - (first & ~15)) // TILE) if n else 0)
    some = sum(t > 0 for t in tiles)
    few = sum(t in (1, 2) for t in tiles)
    total = sum(tiles) * heads
    per_cu = 1 if storage == "16bit" and dim > 128 else 2
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    capacity = p.table.shape[1] * p.page
    seen = min(p.window or capacity, capacity)
    wgs = min(attn.num_wgs or per_cu * min(cus, 256),
              max(1, -(-(seen + 15) // TILE) * heads * len(p.lens)))
    twos = few == some and sum(tiles) == 2 * some
    whole = 3 if all(t in (0, 3) for t in tiles) else 2 if twos else 1
    alone = total > 256 * whole and 3 * few * heads >= wgs
    if alone:
        quota = max(-(-total // (4 * wgs)), 1, min(1 if sum(tiles) == some else 2, -(-total // 1024)))
    else:
        quota = max(-(-total // wgs), whole, min(4 if sum(tiles) > 16 * some else 1, -(-total // 256)))
    longest, start = 1, 0
    for t in tiles:
        for _ in range(heads if t else 0):
            longest = max(longest, (start + t - 1) // quota - start // quota + 1)
            start += t
    return alone, longest


def run_twice(p):
    out, lse = p.run()
    p.check(out, lse)
    for _ in range(2):      # counters are left cleared, and the order of the joining is fixed
        again, lse2 = p.run()
        assert torch.equal(out, again) and torch.equal(lse, lse2)


STORAGES = [("16bit", 64), ("16bit", 128), ("16bit", 256), ("mxfp8", 64), ("mxfp8", 128), ("mxfp8", 256),
            ("mxfp4", 64), ("mxfp4", 128), ("mxfp4", 256)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("storage,dim", STORAGES)
def test_waves_by_themselves(T, storage, dim, dtype):
    """Short heads, ends of a window under a cap, and absent pages, in every type, storage and width."""
    lens = [100, 3, 0, 129, 250] * 40
    p = Problem(T, lens, 4, 2, dim, 16, storage, dtype, holes=(0, 5), window=140, cap=20.0, spread=2.0)
    assert shares(p, 2)[0]
    run_twice(p)


@pytest.mark.parametrize("dtype,storage,dim", [
    ("bf16", "16bit", 128), ("f16", "16bit", 256), ("bf16", "mxfp8", 128), ("f16", "mxfp4", 64)])
@pytest.mark.parametrize("long,least,most", [(3900, GROUP + 1, SINGLE), (7000, SINGLE + 1, 4 * GROUP),
                                             (70000, 16 * GROUP + 1, 1 << 20)])
def test_waves_by_themselves_share_long_heads(T, dtype, storage, dim, long, least, most):
    """One long head among many short ones: its pieces are joined at once, in groups, and in more groups
    than a group has pieces."""
    p = Problem(T, [100] * 75 + [long] + [90] * 75, 4, 2, dim, 16, storage, dtype, spread=2.0)
    alone, pieces = shares(p, 2)
    assert alone and least <= pieces <= most
    run_twice(p)


@pytest.mark.parametrize("tiles,pieces", [(n, n) for n in (
    SINGLE - 1, SINGLE, SINGLE + 1, SINGLE + GROUP - 1, SINGLE + GROUP, SINGLE + GROUP + 1, 16 * GROUP)] +
    [(1100, 275)])
@pytest.mark.parametrize("dtype,storage", [("f16", "16bit"), ("bf16", "mxfp8")])
def test_joins_around_their_limits(T, tiles, pieces, dtype, storage):
    """One head: as many pieces as tiles up to one for each compute unit, then a piece for 4 tiles."""
    p = Problem(T, [TILE * tiles - 7], 5, 1, 64, 16, storage, dtype, num_wgs=1024, spread=2.0)
    assert shares(p, 1) == (False, pieces)
    run_twice(p)


@pytest.mark.parametrize("front", [63, 64, 65, 200])
def test_empty_sequences_in_front(T, front):
    """More empty sequences in front of, between and behind those with tokens than a wave looks at at once."""
    for lens in ([0] * front + [300, 5], [7] + [0] * front + [2000] + [0] * front):
        run_twice(Problem(T, lens, 4, 2, 64, 16, "16bit", "bf16", seed=front))
