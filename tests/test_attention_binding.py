"""CPU-only checks of what the Python binding of include/agmm_attn.h refuses before it calls the library,
with stand-ins for tensors on a GPU."""
import pytest
import torch


@pytest.fixture(scope="module")
def T():
    import all_gather_gemm_amd.attention
    return all_gather_gemm_amd.attention


class Fake:
    """A dense tensor of a shape and type on a device, without memory."""
    is_cuda = True
    requires_grad = False

    def __init__(self, shape, dtype=torch.bfloat16, device="cuda:1"):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)

    def stride(self, dim=None):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s) if dim is None else s[dim]

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 4096

    def element_size(self):
        return self.dtype.itemsize


class Calls:
    """A library whose functions are counted and do nothing."""

    def __init__(self):
        self.names = []

    def __getattr__(self, name):
        def call(*a):
            self.names.append(name)
            return 0
        return call


def calls_of_all_runs(T):
    """(name, call) of every call that launches, with tensors on cuda:1."""
    row = lambda *s: Fake(s)                                     # noqa: E731
    i64 = lambda *s: Fake(s, torch.int64)                        # noqa: E731
    i32 = lambda *s: Fake(s, torch.int32)                        # noqa: E731
    cache = T.PagedCache(row(4, 2, 16, 64), row(4, 2, 16, 64))
    rope = T.Rope.__new__(T.Rope)
    rope.handle, rope.torch_dtype, rope.head_dim = 1, torch.bfloat16, 64
    attn = T.DecodeAttention.__new__(T.DecodeAttention)
    attn.handle, attn.torch_dtype, attn.q_heads, attn.head_dim = 1, torch.bfloat16, 4, 64
    rope.close = attn.close = lambda: None
    k, q = row(3, 2, 64), row(3, 4, 64)
    return [
        ("ag_rope_run", lambda **kw: rope.run(q, i64(3), out=row(3, 4, 64), **kw)),
        ("ag_rope_run", lambda **kw: rope.grad(q, i64(3), out=row(3, 4, 64), **kw)),
        ("ag_kv_append", lambda **kw: cache.append(k, k, i64(3), **kw)),
        ("ag_kv_append_rope", lambda **kw: cache.append_rope(rope, q, k, k, i64(3), i64(3),
                                                             q_out=row(3, 4, 64), **kw)),
        ("ag_kv_read", lambda **kw: cache.read(i64(3), k_out=k, v_out=k, **kw)),
        ("ag_attn_run", lambda **kw: attn.run(q, cache, i32(3, 2), i32(3), out=row(3, 4, 64), **kw)),
    ]


class Stream:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 77


@pytest.fixture
def lib(T, monkeypatch):
    calls = Calls()
    monkeypatch.setattr(T, "lib", calls)
    monkeypatch.setattr(T, "_raw_stream", lambda index: 5)
    return calls


@pytest.mark.parametrize("i", range(6))
def test_tensors_on_another_device_than_the_current(T, monkeypatch, lib, i):
    name, call = calls_of_all_runs(T)[i]
    monkeypatch.setattr(T, "_current", lambda: 0)
    for kw in ({}, {"stream": Stream(1)}, {"stream": Stream(0)}):
        with pytest.raises(T.AgmmError) as e:
            call(**kw)
        assert e.value.code == -6
    assert lib.names == []
    monkeypatch.setattr(T, "_current", lambda: 1)
    call()
    call(stream=Stream(1))
    assert lib.names == [name, name]
    with pytest.raises(T.AgmmError):
        call(stream=Stream(0))
    assert lib.names == [name, name]
    lib.names.clear()


def test_no_rotated_elements(T):
    """A rotated part of 0 elements is refused, as any other that the header does not allow."""
    for rot in (0, 3, -2, 66):
        with pytest.raises(T.AgmmError) as e:
            T.Rope(64, rot_dim=rot)
        assert e.value.code == -1


@pytest.mark.parametrize("storage,row", [("mxfp8", 64), ("mxfp4", 32)])
def test_coded_cache_without_scales(T, storage, row):
    pool = Fake((4, 2, 16, row), torch.uint8)
    scale = Fake((4, 2, 16, 4), torch.uint8)
    for scales in ((), (scale,), (None, scale)):
        with pytest.raises(ValueError):
            T.PagedCache(pool, pool, *scales, storage=storage)
    assert T.PagedCache(pool, pool, scale, scale, storage=storage).head_dim == 64


def test_magnitude_past_32_bits(T):
    for m in (1e39, -1e300):
        with pytest.raises(T.AgmmError) as e:
            T.Rope(64, magnitude=m)
        assert e.value.code == -1
