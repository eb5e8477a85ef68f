"""Refusals of include/agmm_long.h that need a handle, and so a GPU: the documented codes, and nothing written."""
import ctypes

import pytest
import torch

import long_reference as lr

pytestmark = pytest.mark.gpu
INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def T():
    import all_gather_gemm_amd.attention
    return all_gather_gemm_amd.attention


@pytest.fixture(scope="module")
def L():
    import all_gather_gemm_amd.long_context
    return all_gather_gemm_amd.long_context


def prefix_run(L, attn, pool, q, out, groups=1, pages=None):
    """ag_prefix_run of run 0 as the prefix of the sequences 1 and 2."""
    table, n, own, lens = pool.table([0]), pool.lengths([0]), pool.table([1, 2]), pool.lengths([1, 2])
    size = L.lib.ag_prefix_scratch_bytes(ctypes.byref(attn.desc), 2, 1)
    scratch = torch.empty(size, dtype=torch.uint8, device=lr.DEV)
    return L.lib.ag_prefix_run(
        attn.handle, pool.cache._ref, q.data_ptr(), q.stride(0), q.stride(1), table.data_ptr(), table.stride(0),
        table.shape[1] if pages is None else pages, n.data_ptr(), None, groups, own.data_ptr(), own.stride(0),
        own.shape[1], lens.data_ptr(), 2, out.data_ptr(), out.stride(0), out.stride(1), None, scratch.data_ptr(), size,
        torch.cuda.current_stream().cuda_stream)


def test_prefix(T, L):
    pool = lr.Pool(T, [40, 3, 20], 1, 64, 16, "16bit", "bf16")
    q = pool.q(2, 4)
    out = torch.full((2, 4, 64), 7.0, dtype=torch.bfloat16, device=lr.DEV)
    plain = T.DecodeAttention(4, 1, 64)
    assert prefix_run(L, T.DecodeAttention(4, 1, 64, window=5), pool, q, out) == UNSUPPORTED
    assert prefix_run(L, T.DecodeAttention(4, 1, 64, scale=2.0 ** 64), pool, q, out) == UNSUPPORTED
    assert prefix_run(L, plain, pool, q, out, groups=-1) == INVALID
    assert prefix_run(L, plain, pool, q, out, groups=2) == INVALID      # and no starts
    assert prefix_run(L, plain, pool, q, out, pages=-1) == INVALID
    assert (out == 7.0).all()
    assert prefix_run(L, plain, pool, q, out) == 0
    assert torch.equal(out, L.PrefixAttention(4, 1, 64).run(q, pool.cache, pool.table([0]), pool.lengths([0]),
                                                            pool.table([1, 2]), pool.lengths([1, 2])))
