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
