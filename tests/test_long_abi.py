"""CPU-only checks of the functions of include/agmm_long.h: they are exported, they refuse what they document
before they touch a device, and their scratch sizes are the documented layout's."""
import ctypes
import math
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def L():
    import all_gather_gemm_amd.long_context
    return all_gather_gemm_amd.long_context


def test_exports_every_declared_symbol(L):
    with open(os.path.join(ROOT, "include", "agmm_long.h")) as fh:
        text = re.sub(r"/\*.*?\*/", "", fh.read(), flags=re.S)
    names = set(re.findall(r"\b(ag_\w+)\s*\(", text))
    assert names == set(L.EXPORTED)
    for n in names:
        assert hasattr(L.lib, n), n


def test_header_is_c(L, tmp_path):
    (tmp_path / "probe.c").write_text('#include "agmm_long.h"\n#include <stdio.h>\n'
                                      'int main(void){printf("%zu\\n", sizeof(ag_page_index));return 0;}')
    exe = str(tmp_path / "probe")
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(tmp_path / "probe.c"), "-o",
                    exe], check=True)
    assert int(subprocess.run([exe], capture_output=True, check=True).stdout) == ctypes.sizeof(L.ag_page_index)


def cache(L, **kw):
    c = L.ag_kv_cache()
    base = dict(dtype=1, storage=0, head_dim=128, kv_heads=2, page_size=16, num_pages=4, k=4096,
                v=8192, page_stride=8192, head_stride=4096, row_stride=256)
    if kw.get("storage"):
        base.update(k_scale=16384, v_scale=20480, scale_page=128, scale_head=64, scale_row=4)
    for k, v in dict(base, **kw).items():
        setattr(c, k, v)
    return c


def desc(L, **kw):
    d = L.ag_attn_desc()
    L.lib.ag_attn_desc_init(ctypes.byref(d))
    for k, v in dict(dict(q_heads=8, kv_heads=2), **kw).items():
        setattr(d, k, v)
    return d


def test_prefix_scratch(L):
    # the groups' plans; for each strip of 128 rows, unfilled one of a group and workgroup a piece of 128 padded
    # rows, with their maxima and sums; and the same of each row for the own tokens
    al = lambda x: (x + 255) & ~255  # noqa: E731
    for dim, padded, wgs in ((64, 64, 512), (80, 128, 512), (256, 256, 256)):
        for batch, groups, q, kv in ((1, 1, 8, 1), (100, 3, 64, 8), (7, 20, 6, 2), (0, 0, 4, 4), (300, 300, 1, 1)):
            slots = kv * (batch * (q // kv) // 128 + min(batch, groups)) + wgs
            want = al(32 * groups) + slots * 128 * padded * 4 + al(slots * 1024)
            want = al(want + batch * q * (padded + 2) * 4)
            d = desc(L, head_dim=dim, q_heads=q, kv_heads=kv)
            assert L.lib.ag_prefix_scratch_bytes(ctypes.byref(d), batch, groups) == want
    d = ctypes.byref(desc(L))
    assert L.lib.ag_prefix_scratch_bytes(None, 1, 1) == INVALID
    assert L.lib.ag_prefix_scratch_bytes(d, -1, 1) == INVALID
    assert L.lib.ag_prefix_scratch_bytes(d, 1, -1) == INVALID
    assert L.lib.ag_prefix_scratch_bytes(d, 1 << 31, 1) == UNSUPPORTED
    assert L.lib.ag_prefix_scratch_bytes(d, 1 << 62, 1 << 62) == UNSUPPORTED
    assert L.lib.ag_prefix_scratch_bytes(ctypes.byref(desc(L, head_dim=36)), 1, 1) == UNSUPPORTED


def test_runs_without_a_handle(L):
    c = ctypes.byref(cache(L))
    assert L.lib.ag_prefix_run(None, c, 64, 0, 0, 64, 0, 1, 64, None, 1, 64, 0, 1, 64, 1, 64, 0, 0, None, 256, 1 << 40,
                               None) == INVALID
    assert L.lib.ag_attn_run_heads(None, c, 64, 0, 0, 64, 0, 0, 1, 64, 1, 64, 0, 0, None, None) == INVALID


def index(L, codes=4096, scales=64):
    return ctypes.byref(L.ag_page_index(codes, scales))


def update(L, c=None, x=None, table=64, pages=2, starts=None, lens=64, batch=1):
    return L.lib.ag_index_update(ctypes.byref(c or cache(L)), x or index(L), table, 8, pages, starts, lens, batch, None)


@pytest.mark.parametrize("rc,kw", [
    (INVALID, dict(table=None)), (INVALID, dict(table=66)), (INVALID, dict(lens=None)), (INVALID, dict(starts=65)),
    (INVALID, dict(batch=-1)), (INVALID, dict(pages=-1)), (UNSUPPORTED, dict(pages=1 << 27)),
    (UNSUPPORTED, dict(batch=(1 << 20) + 1)), (UNSUPPORTED, dict(pages=1 << 62)),
    (0, dict(batch=0, table=None, lens=None)), (0, dict(pages=0, table=None)),
])
def test_update_refusals(L, rc, kw):
    assert update(L, **kw) == rc


def test_index_refusals(L):
    assert update(L, x=index(L, codes=4104)) == INVALID
    assert update(L, x=index(L, scales=None)) == INVALID
    assert update(L, c=cache(L, head_dim=100)) == UNSUPPORTED
    assert update(L, c=cache(L, dtype=7)) == INVALID
    assert L.lib.ag_index_update(ctypes.byref(cache(L)), None, 64, 8, 2, None, 64, 1, None) == INVALID


def select(L, c=None, x=None, q=64, heads=8, table=64, pages=2, lens=64, batch=1, budget=4, sink=1, recent=1, out=64,
           out_lens=64, scratch=64, bytes=1 << 40):
    return L.lib.ag_index_select(ctypes.byref(c or cache(L)), x or index(L), q, 0, 0, heads, table, 8, pages, lens,
                                 batch, budget, sink, recent, out, out_lens, scratch, bytes, None)


@pytest.mark.parametrize("rc,kw", [
    (INVALID, dict(budget=0)), (INVALID, dict(budget=-1)), (INVALID, dict(sink=-1)), (INVALID, dict(recent=0)),
    (INVALID, dict(sink=4)), (INVALID, dict(recent=5)), (INVALID, dict(sink=1 << 62, recent=1 << 62)),
    (INVALID, dict(heads=3)), (INVALID, dict(heads=0)), (UNSUPPORTED, dict(heads=258)),
    (UNSUPPORTED, dict(budget=1 << 31)), (INVALID, dict(q=63)), (INVALID, dict(table=None)), (INVALID, dict(lens=62)),
    (INVALID, dict(out=None)), (INVALID, dict(out_lens=66)), (INVALID, dict(scratch=72, pages=300)),
    (INVALID, dict(bytes=2399, pages=300)), (INVALID, dict(scratch=None, pages=300)), (UNSUPPORTED, dict(batch=(1 << 20) + 1)), (UNSUPPORTED, dict(pages=1 << 27)),
    (0, dict(batch=0, q=None, table=None, lens=None, out=None, out_lens=None, scratch=None)),
])
def test_select_refusals(L, rc, kw):
    assert select(L, **kw) == rc


def test_index_scratch(L):
    c = ctypes.byref(cache(L))
    for pages, batch in ((0, 3), (1, 1), (256, 7), (257, 7), (1001, 64)):   # (up to 256 there is none)
        assert L.lib.ag_index_scratch_bytes(c, pages, batch) == \
            (4 * 2 * batch * (-(-pages // 4) * 4) if pages > 256 else 0)
    assert L.lib.ag_index_scratch_bytes(c, -1, 1) == INVALID
    assert L.lib.ag_index_scratch_bytes(c, 1, -1) == INVALID
    assert L.lib.ag_index_scratch_bytes(c, 1 << 31, 1) == UNSUPPORTED
    assert L.lib.ag_index_scratch_bytes(c, 1, (1 << 20) + 1) == UNSUPPORTED


def add(L, d=None, c=None, q=64, lse=64, table=64, pages=2, lens=64, batch=1, mass=64, mass_batch=64, mass_head=32,
        out=4096, out_batch=64, out_head=32, tokens=32, decay=0.5):
    return L.lib.ag_mass_add(ctypes.byref(d or desc(L)), ctypes.byref(c or cache(L)), q, 0, 0, lse, table, 8, pages,
                             lens, batch, mass, mass_batch, mass_head, out, out_batch, out_head, tokens, decay, None)


@pytest.mark.parametrize("rc,kw", [
    (INVALID, dict(q=63)), (INVALID, dict(lse=None)), (INVALID, dict(lse=66)), (INVALID, dict(mass=None)),
    (INVALID, dict(out=4098)), (INVALID, dict(tokens=-1)), (UNSUPPORTED, dict(tokens=1 << 31)),
    (INVALID, dict(decay=math.nan)), (INVALID, dict(decay=math.inf)), (INVALID, dict(table=None)),
    (INVALID, dict(lens=None)), (INVALID, dict(batch=-1)), (UNSUPPORTED, dict(pages=1 << 27)),
    (INVALID, dict(out=64, out_head=33)), (INVALID, dict(out=64, out_batch=65, batch=2)),
    (0, dict(batch=0, q=None, lse=None, mass=None, out=None, table=None, lens=None)),
    (0, dict(tokens=0, mass=None, out=None)),
])
def test_mass_refusals(L, rc, kw):
    assert add(L, **kw) == rc


def test_mass_geometry(L):
    for kw in (dict(kv_heads=4), dict(dtype=0), dict(head_dim=64), dict(storage=1)):
        assert add(L, d=desc(L, **kw)) == INVALID
    assert add(L, d=desc(L, window=-1)) == INVALID
    assert add(L, d=desc(L, scale=math.inf)) == INVALID


def choose(L, c=None, mass=64, tokens=32, table=64, pages=2, lens=64, batch=1, budget=4, sink=1, recent=1, kept=64,
           out_mass=None, out_lens=64):
    return L.lib.ag_evict_choose(ctypes.byref(c or cache(L)), mass, 64, 32, tokens, table, 8, pages, lens, batch,
                                 budget, sink, recent, kept, out_mass, out_lens, None)


@pytest.mark.parametrize("rc,kw", [
    (INVALID, dict(budget=0)), (INVALID, dict(sink=-1)), (INVALID, dict(recent=-1)), (INVALID, dict(sink=4)),
    (INVALID, dict(tokens=-1)), (UNSUPPORTED, dict(tokens=1 << 31)), (INVALID, dict(mass=None)),
    (INVALID, dict(mass=66)), (INVALID, dict(kept=None)), (INVALID, dict(out_mass=66)), (INVALID, dict(out_lens=None)),
    (INVALID, dict(table=None)), (INVALID, dict(lens=None)), (UNSUPPORTED, dict(budget=1 << 31)),
    (UNSUPPORTED, dict(batch=(1 << 20) + 1)),
    (0, dict(batch=0, mass=None, table=None, lens=None, kept=None, out_lens=None)),
])
def test_choose_refusals(L, rc, kw):
    assert choose(L, **kw) == rc


def move(L, c=None, to=None, table=64, pages=2, to_table=64, to_pages=2, kept=64, budget=4, lens=64, batch=1):
    return L.lib.ag_evict_move(ctypes.byref(c or cache(L)), table, 8, pages, ctypes.byref(to or cache(L)), to_table, 8,
                               to_pages, kept, budget, lens, batch, None)


@pytest.mark.parametrize("rc,kw", [
    (INVALID, dict(table=None)), (INVALID, dict(to_table=66)), (INVALID, dict(kept=None)), (INVALID, dict(lens=None)),
    (INVALID, dict(budget=-1)), (INVALID, dict(batch=-1)), (INVALID, dict(to_pages=-1)),
    (UNSUPPORTED, dict(budget=1 << 30)), (UNSUPPORTED, dict(to_pages=1 << 27)),
    (0, dict(batch=0, table=None, to_table=None, kept=None, lens=None)), (0, dict(budget=0, kept=None)),
])
def test_move_refusals(L, rc, kw):
    assert move(L, **kw) == rc


def test_tables_near_31_bits(L):
    """Pages of 16: tables of 2^31 - 2^20 tokens and more are refused, before anything is launched."""
    for pages in ((1 << 27) - (1 << 16), (1 << 27) - 1):
        assert select(L, pages=pages) == add(L, pages=pages) == choose(L, pages=pages) == UNSUPPORTED
        assert move(L, pages=pages) == move(L, to_pages=pages) == UNSUPPORTED


def test_move_between_unlike_caches(L):
    for kw in (dict(dtype=0), dict(storage=1), dict(head_dim=64), dict(kv_heads=1)):
        assert move(L, to=cache(L, **kw)) == INVALID
