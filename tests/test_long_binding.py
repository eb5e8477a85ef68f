"""CPU-only checks of what the Python binding of include/agmm_long.h refuses before it calls the library, with
stand-ins for tensors on a GPU."""
import pytest
import torch

from test_attention_binding import Calls, Fake, Stream


@pytest.fixture(scope="module")
def L():
    import all_gather_gemm_amd.long_context
    return all_gather_gemm_amd.long_context


@pytest.fixture(scope="module")
def T():
    import all_gather_gemm_amd.attention
    return all_gather_gemm_amd.attention


class F(Fake):
    """Also what the binding of agmm_long.h asks a tensor."""

    def is_contiguous(self):
        return True

    def new_empty(self, shape, dtype=None):
        return F(shape, dtype or self.dtype, self.device)

    def get_device(self):
        return self.device.index

    def numel(self):
        return self.shape.numel()


row = lambda *s: F(s)                    # noqa: E731
i32 = lambda *s: F(s, torch.int32)       # noqa: E731
f32 = lambda *s: F(s, torch.float32)     # noqa: E731


@pytest.fixture
def lib(T, L, monkeypatch):
    class Sized(Calls):
        def __getattr__(self, name):
            if name.endswith("_bytes"):
                return lambda *a: 64
            return super().__getattr__(name)
    calls = Sized()
    monkeypatch.setattr(T, "lib", calls)
    monkeypatch.setattr(L, "lib", calls)
    monkeypatch.setattr(T, "_raw_stream", lambda index: 5)
    monkeypatch.setattr(torch, "empty_like", lambda x: F(x.shape, x.dtype, x.device))
    return calls


@pytest.fixture
def parts(T, L, monkeypatch, lib):
    monkeypatch.setattr(T, "_result", lambda make, stream, device: make())
    cache = T.PagedCache(row(4, 2, 16, 64), row(4, 2, 16, 64))
    prefix = L.PrefixAttention.__new__(L.PrefixAttention)
    prefix.handle, prefix.torch_dtype, prefix.q_heads, prefix.head_dim = 1, torch.bfloat16, 4, 64
    prefix.desc, prefix._scratch, prefix.close = T.ag_attn_desc(), {}, lambda: None
    attn = T.DecodeAttention.__new__(T.DecodeAttention)
    attn.handle, attn.torch_dtype, attn.q_heads, attn.head_dim = 1, torch.bfloat16, 4, 64
    attn.desc, attn.close = T.ag_attn_desc(), lambda: None
    attn.desc.kv_heads = 2
    index = L.PageIndex(cache, F((4, 2, 2, 64), torch.int8), F((4, 2), torch.uint8))
    adder = L.AttentionMass(4, 2, 64)
    lib.names.clear()
    return dict(cache=cache, prefix=prefix, attn=attn, index=index, adder=adder, evictor=L.Evictor(8, 1, 2))


def calls_of(p):
    q, t, n = row(3, 4, 64), i32(3, 2), i32(3)
    return {
        "ag_prefix_run": lambda **kw: p["prefix"].run(q, p["cache"], i32(1, 2), i32(1), t, n, **kw),
        "ag_attn_run_heads": lambda **kw: p["attn"].run(q, p["cache"], i32(3, 2, 5), n, **kw),
        "ag_index_update": lambda **kw: p["index"].update(t, n, **kw),
        "ag_index_select": lambda **kw: p["index"].select(q, t, n, 8, **kw),
        "ag_mass_add": lambda **kw: p["adder"].add(f32(3, 2, 40), q, f32(3, 4), p["cache"], t, n, **kw),
        "ag_evict_choose": lambda **kw: p["evictor"].choose(p["cache"], t, n, f32(3, 2, 40), **kw),
        "ag_evict_move": lambda **kw: p["evictor"].move(p["cache"], t, i32(3, 2, 8), n, Moved((3, 2), torch.int32),
                                                        **kw),
    }


class Moved(F):
    def data_ptr(self):
        return 8192


NAMES = ["ag_prefix_run", "ag_attn_run_heads", "ag_index_update", "ag_index_select", "ag_mass_add", "ag_evict_choose",
         "ag_evict_move"]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_on_another_device_than_the_current(T, monkeypatch, lib, parts, name):
    call = calls_of(parts)[name]
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


def test_prefix_refusals(T, monkeypatch, lib, parts):
    monkeypatch.setattr(T, "_current", lambda: 1)
    q, t, n, cache, run = row(3, 4, 64), i32(3, 2), i32(3), parts["cache"], parts["prefix"].run
    for bad in (
            lambda: run(q, cache, i32(2, 2), i32(2), t, n),                          # groups without starts
            lambda: run(q, cache, i32(2, 2), i32(2), t, n, starts=i32(2)),
            lambda: run(q, cache, i32(2, 2), i32(1), t, n),
            lambda: run(q, cache, i32(1, 2, 2), i32(1), t, n),
            lambda: run(q, cache, i32(1, 2), F((1,), torch.int64), t, n),
            lambda: run(q, cache, i32(1, 2), i32(1), i32(2, 2), n),
            lambda: run(q, cache, i32(1, 2), i32(1), t, i32(2)),
            lambda: run(row(3, 5, 64), cache, i32(1, 2), i32(1), t, n),
            lambda: run(q, cache, i32(1, 2), i32(1), t, n, out=row(3, 4, 32))):
        with pytest.raises(ValueError):
            bad()
    assert lib.names == []


def test_table_of_heads_refusals(T, monkeypatch, lib, parts):
    monkeypatch.setattr(T, "_current", lambda: 1)
    for shape in ((3, 1, 5), (3, 4, 5), (2, 2, 5), (3,), (3, 2, 5, 1)):
        with pytest.raises(ValueError):
            parts["attn"].run(row(3, 4, 64), parts["cache"], i32(*shape), i32(3))
    assert lib.names == []


def test_index_refusals(T, L, monkeypatch, lib, parts):
    monkeypatch.setattr(T, "_current", lambda: 1)
    codes, scales, cache = F((4, 2, 2, 64), torch.int8), F((4, 2), torch.uint8), parts["cache"]
    for bad in (lambda: L.PageIndex(cache, codes), lambda: L.PageIndex(cache, scales=scales),
                lambda: L.PageIndex(cache, F((4, 2, 64, 2), torch.int8), scales),
                lambda: L.PageIndex(cache, F((4, 2, 2, 64), torch.uint8), scales),
                lambda: L.PageIndex(cache, codes, F((4, 1), torch.uint8)),
                lambda: L.PageIndex(cache, F((4, 2, 2, 64), torch.int8, "cuda:0"), scales)):
        with pytest.raises(ValueError):
            bad()
    codes.is_contiguous = lambda: False
    with pytest.raises(ValueError):
        L.PageIndex(cache, codes, scales)
    x, t, n = parts["index"], i32(3, 2), i32(3)
    for bad in (lambda: x.update(i32(2, 2), n), lambda: x.update(t, n, i32(2)),
                lambda: x.select(row(3, 4, 32), t, n, 8), lambda: x.select(row(3, 4, 64), i32(2, 2), n, 8),
                lambda: x.select(row(3, 4, 64), t, i32(4), 8), lambda: x.select(row(3, 4, 64), t, n, 0),
                lambda: x.select(F((3, 4, 64), torch.float16), t, n, 8)):
        with pytest.raises(ValueError):
            bad()
    assert lib.names == []


def test_mass_refusals(T, L, monkeypatch, lib, parts):
    monkeypatch.setattr(T, "_current", lambda: 1)
    q, t, n, lse, c, add = row(3, 4, 64), i32(3, 2), i32(3), f32(3, 4), parts["cache"], parts["adder"].add
    for bad in (lambda: add(f32(3, 1, 40), q, lse, c, t, n), lambda: add(f32(2, 2, 40), q, lse, c, t, n),
                lambda: add(F((3, 2, 40)), q, lse, c, t, n), lambda: add(f32(3, 2, 40), q, f32(3, 2), c, t, n),
                lambda: add(f32(3, 2, 40), q, lse, c, t, n, out=f32(3, 2, 41)),
                lambda: add(f32(3, 2, 40), q, lse, c, t, F((3,), torch.int64))):
        with pytest.raises(ValueError):
            bad()
    lse.is_contiguous = lambda: False
    with pytest.raises(ValueError):
        add(f32(3, 2, 40), q, lse, c, t, n)
    assert lib.names == []


def test_mass_geometry(T, L):
    for kw in (dict(q_heads=3, kv_heads=2, head_dim=64), dict(q_heads=4, kv_heads=2, head_dim=36),
               dict(q_heads=4, kv_heads=2, head_dim=64, window=-1)):
        with pytest.raises(T.AgmmError):
            L.AttentionMass(**kw)
    with pytest.raises(ValueError):
        L.AttentionMass(4, 2, 64, storage="int8")


def test_evictor_refusals(T, L, monkeypatch, lib, parts):
    monkeypatch.setattr(T, "_current", lambda: 1)
    for a in ((0,), (8, -1, 2), (8, 1, -2), (8, 5, 4), (8, 9, 0)):
        with pytest.raises(ValueError):
            L.Evictor(*a)
    e, c, t, n = parts["evictor"], parts["cache"], i32(3, 2), i32(3)
    other = T.PagedCache(F((4, 2, 16, 64), device="cuda:0"), F((4, 2, 16, 64), device="cuda:0"))
    for bad in (lambda: e.choose(c, t, n, f32(3, 1, 40)), lambda: e.choose(c, i32(2, 2), n, f32(3, 2, 40)),
                lambda: e.move(c, t, i32(3, 1, 8), n, Moved((3, 2), torch.int32)),
                lambda: e.move(c, t, i32(3, 2, 8), n, Moved((2, 2), torch.int32)),
                lambda: e.move(c, t, i32(3, 2, 8), n, i32(3, 2)),                     # onto itself
                lambda: e.move(c, t, i32(3, 2, 8), n, Moved((3, 2), torch.int32), to=other)):
        with pytest.raises(ValueError):
            bad()
    assert lib.names == []
