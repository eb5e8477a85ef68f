"""CPU-only checks of the functions of include/agmm_attn.h: they are exported, their structs have
the header's layout, they refuse what they document before they touch a device, and the rotary
frequencies are the formulas'."""
import ctypes
import math
import os
import re
import subprocess

import pytest

import attention_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def T():
    import all_gather_gemm_amd.attention
    return all_gather_gemm_amd.attention


def test_exports_every_declared_symbol(T):
    with open(os.path.join(ROOT, "include", "agmm_attn.h")) as fh:
        text = re.sub(r"/\*.*?\*/", "", fh.read(), flags=re.S)
    names = set(re.findall(r"\b(ag_(?:rope|kv|attn)_\w+)\s*\(", text))
    assert names == set(T.EXPORTED)
    for n in names:
        assert hasattr(T.lib, n), n


def test_struct_layout_matches_header(T, tmp_path):
    structs = {"ag_rope_desc": T.ag_rope_desc, "ag_kv_cache": T.ag_kv_cache,
               "ag_attn_desc": T.ag_attn_desc}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "agmm_attn.h"',
             "int main(void){"]
    for name, cls in structs.items():
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    (tmp_path / "probe.c").write_text("\n".join(lines + ["return 0;}"]))
    exe = str(tmp_path / "probe")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "probe.c"), "-o", exe],
                   check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    got = {tuple(line.split()[:2]): int(line.split()[2]) for line in out.splitlines()}
    for name, cls in structs.items():
        assert got[(name, "size")] == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert got[(name, f)] == getattr(cls, f).offset, (name, f)


def _rope(T, **kw):
    d = T.ag_rope_desc()
    T.lib.ag_rope_desc_init(ctypes.byref(d))
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(head_dim=1), dict(head_dim=1025), dict(rot_dim=0), dict(rot_dim=3),
    dict(rot_dim=130), dict(rot_start=2), dict(rot_start=-1), dict(pairing=2), dict(scaling=5),
    dict(base=1.0), dict(base=math.inf), dict(scaling=1, factor=0.0), dict(magnitude=math.nan),
    dict(scaling=2, rot_dim=2, factor=2.0), dict(scaling=3, original_len=0.0),
    dict(scaling=4, original_len=8.0, low=4.0, high=4.0), dict(head_dim=1024, rot_dim=514),
])
def test_rope_refusals(T, bad):
    d, h = _rope(T, **bad), ctypes.c_void_p()
    out = (ctypes.c_double * 512)()
    assert T.lib.ag_rope_create(ctypes.byref(d), ctypes.byref(h)) == INVALID
    assert T.lib.ag_rope_thetas(ctypes.byref(d), out) == INVALID


@pytest.mark.parametrize("rot,kw", [
    (128, {}), (64, dict(scaling="linear", factor=4.0)),
    (128, dict(scaling="base", factor=8.0, base=500000.0)),
    (128, dict(scaling="turns", factor=8.0, original_len=8192.0, low=1.0, high=4.0)),
    (96, dict(scaling="index", factor=40.0, original_len=4096.0, low=1.0, high=32.0)),
    (6, dict(scaling="index", factor=2.0, original_len=100.0, low=1.0, high=32.0)),
])
def test_rope_frequencies(T, rot, kw):
    c = dict(kw, scaling=T._SCALINGS[kw.get("scaling", "none")])
    d = _rope(T, head_dim=max(rot, 2), rot_dim=rot, **c)
    out = (ctypes.c_double * (rot // 2))()
    assert T.lib.ag_rope_thetas(ctypes.byref(d), out) == 0
    # a power and a few products in doubles on either side
    assert list(out) == pytest.approx(ref.thetas(rot, **kw), rel=1e-13)


def test_rope_given_frequencies(T):
    th = (ctypes.c_double * 4)(1.0, 0.5, -0.25, 7.0)
    d = _rope(T, head_dim=8, rot_dim=8, thetas=th, scaling=9)   # the rest is not read
    out = (ctypes.c_double * 4)()
    assert T.lib.ag_rope_thetas(ctypes.byref(d), out) == 0 and list(out) == list(th)
    th[1] = math.inf
    assert T.lib.ag_rope_thetas(ctypes.byref(d), out) == INVALID


def _cache(T, **kw):
    c = T.ag_kv_cache()
    base = dict(dtype=1, storage=0, head_dim=128, kv_heads=2, page_size=16, num_pages=4, k=4096,
                v=8192, page_stride=8192, head_stride=4096, row_stride=256)
    if kw.get("storage"):
        base.update(k_scale=16384, v_scale=20480, scale_page=128, scale_head=64, scale_row=4)
    for k, v in dict(base, **kw).items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("rc,bad", [
    (INVALID, dict(dtype=2)), (INVALID, dict(storage=3)), (INVALID, dict(head_dim=0)),
    (INVALID, dict(page_size=0)), (INVALID, dict(kv_heads=0)), (INVALID, dict(num_pages=-1)),
    (UNSUPPORTED, dict(head_dim=264)), (UNSUPPORTED, dict(head_dim=100)),
    (UNSUPPORTED, dict(storage=1, head_dim=80)), (UNSUPPORTED, dict(storage=2, head_dim=16)),
    (UNSUPPORTED, dict(num_pages=1 << 27)), (UNSUPPORTED, dict(num_pages=1 << 31)),
    (UNSUPPORTED, dict(num_pages=(1 << 62) + 1)),
    (UNSUPPORTED, dict(page_stride=1 << 32)), (UNSUPPORTED, dict(row_stride=1 << 40)),
    (UNSUPPORTED, dict(storage=1, scale_page=1 << 32)),
    (INVALID, dict(page_stride=8200)), (INVALID, dict(row_stride=-256)), (INVALID, dict(k=4104)),
    (INVALID, dict(v=None)), (INVALID, dict(k_scale=4096)),
    (INVALID, dict(storage=1, k_scale=None)), (INVALID, dict(storage=1, scale_row=2)),
    (INVALID, dict(storage=2, v_scale=20482)),
])
def test_cache_refusals(T, rc, bad):
    c = ctypes.byref(_cache(T, **bad))
    assert T.lib.ag_kv_append(c, 64, 256, 128, 64, 256, 128, 64, 1, None) == rc
    assert T.lib.ag_kv_read(c, 64, 1, 64, 256, 128, 64, 256, 128, None) == rc


def test_argument_refusals(T):
    c = ctypes.byref(_cache(T))
    assert T.lib.ag_kv_append(None, 64, 256, 128, 64, 256, 128, 64, 1, None) == INVALID
    assert T.lib.ag_kv_append(c, 64, 256, 128, 64, 256, 128, 64, -1, None) == INVALID
    assert T.lib.ag_kv_append(c, 65, 256, 128, 64, 256, 128, 64, 1, None) == INVALID
    assert T.lib.ag_kv_append(c, 64, 256, 128, None, 256, 128, 64, 1, None) == INVALID
    assert T.lib.ag_kv_append(c, 64, 256, 128, 64, 256, 128, 60, 1, None) == INVALID
    assert T.lib.ag_kv_read(c, 64, 1, 64, 256, 128, 63, 256, 128, None) == INVALID
    # nothing to do is no error, and touches nothing
    assert T.lib.ag_kv_append(c, None, 0, 0, None, 0, 0, None, 0, None) == 0
    assert T.lib.ag_kv_read(c, None, 0, None, 0, 0, None, 0, 0, None) == 0
    assert T.lib.ag_kv_append_rope(c, None, 64, 0, 0, 1, 64, 0, 0, 64, 0, 0, 64, 0, 0, 64, 64, 1,
                                   None) == INVALID
    assert T.lib.ag_rope_run(None, 64, 0, 0, 0, 64, 0, 0, 0, 64, 0, 1, 1, 1, 0, None) == INVALID
    assert T.lib.ag_attn_run(None, c, 64, 0, 0, 64, 0, 1, 64, 1, 64, 0, 0, None, None) == INVALID
    assert T.lib.ag_rope_destroy(None) == 0 and T.lib.ag_attn_destroy(None) == 0


def _attn(T, **kw):
    d = T.ag_attn_desc()
    T.lib.ag_attn_desc_init(ctypes.byref(d))
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("rc,bad", [
    (INVALID, dict(dtype=-1)), (INVALID, dict(storage=3)), (INVALID, dict(q_heads=3, kv_heads=2)),
    (INVALID, dict(kv_heads=0)), (INVALID, dict(window=-1)), (INVALID, dict(num_wgs=1025)),
    (INVALID, dict(scale=-1.0)), (INVALID, dict(scale=math.nan)), (INVALID, dict(soft_cap=-2.0)),
    (INVALID, dict(soft_cap=math.inf)), (UNSUPPORTED, dict(head_dim=320)),
    (UNSUPPORTED, dict(head_dim=36)), (UNSUPPORTED, dict(storage=1, head_dim=72)),
])
def test_attention_refusals(T, rc, bad):
    d, h = _attn(T, **bad), ctypes.c_void_p()
    assert T.lib.ag_attn_workspace_bytes(ctypes.byref(d)) == rc
    assert T.lib.ag_attn_create(ctypes.byref(d), None, 0, ctypes.byref(h)) == rc


def test_attention_workspace(T):
    # two partial results (the group's rows, each padded and with its maximum and sum) and three
    # counters for each wave: 4 a workgroup, two workgroups a compute unit, one for rows of 256 16-bit
    # elements
    al = lambda x: (x + 255) & ~255  # noqa: E731
    for hd, padded, wgs in ((64, 64, 512), (80, 128, 512), (128, 128, 512), (136, 256, 256)):
        for q_heads, rows in ((8, 4), (64, 16)):
            d = _attn(T, head_dim=hd, q_heads=q_heads, kv_heads=2)
            assert T.lib.ag_attn_workspace_bytes(ctypes.byref(d)) == \
                al(8 * wgs * rows * (padded + 2) * 4) + al(12 * wgs * 4)


def test_binding_refuses_cpu_tensors(T):
    import torch
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        T.PagedCache(k, k)
    with pytest.raises(ValueError):
        T.PagedCache(k, k, storage="int8")
