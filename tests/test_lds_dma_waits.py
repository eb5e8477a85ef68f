"""Wait states in front of the loads from memory to LDS, in the built gfx950 code (CPU: the code is only listed).

Such a load takes its LDS address from m0 and needs one wait state behind the write of m0, and 5 behind a vector
instruction's write of a scalar register that it reads. The compiler keeps those where it makes the load itself; where
the load is inline asm, as here, it does not look."""
import os
import re
import shutil
import subprocess

import pytest

import all_gather_gemm_amd.build as build

OBJDUMP = os.path.join(build.LLVM_BIN, "llvm-objdump")
pytestmark = pytest.mark.skipif(not (os.path.exists(build.LIB) and shutil.which(OBJDUMP)),
                                reason="no built library or no llvm-objdump")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects():
    """The gfx950 code objects of the built library, one for each source with kernels."""
    with open(build.LIB, "rb") as fh:
        b = fh.read()
    at = b.find(MAGIC)
    while at >= 0:
        count = int.from_bytes(b[at + 24:at + 32], "little")
        off = at + 32
        for _ in range(count if count < 16 else 0):
            o, size, tl = (int.from_bytes(b[off + 8 * i:off + 8 * i + 8], "little") for i in range(3))
            triple = b[off + 24:off + 24 + tl]
            off += 24 + tl
            if triple.endswith(b"gfx950") and size:
                yield b[at + o:at + o + size]
        at = b.find(MAGIC, at + 1)


def listing(co, path):
    path.write_bytes(co)
    text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--demangle", str(path)], check=True,
                          capture_output=True, text=True).stdout
    kernels, now = {}, None
    for line in text.splitlines():
        if line.endswith(">:"):
            now = kernels.setdefault(line.split("<", 1)[1][:-2], [])
        elif now is not None and line.startswith("\t"):
            now.append(line.split("//")[0].strip())
    return kernels


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    path = tmp_path_factory.mktemp("code") / "co"
    out = {}
    for co in code_objects():
        out.update(listing(co, path))
    return out


def is_lds_load(x):
    return x.startswith(("buffer_load", "global_load")) and ("load_lds" in x or re.search(r"\blds\b", x))


def without_wait(code):
    """Loads to LDS whose m0 the instruction right in front of them writes."""
    return [f"{a} | {b}" for a, b in zip(code, code[1:])
            if is_lds_load(b) and re.match(r"[sv]_\w+ m0\b", a)]


def scalars(text):
    out = {int(n) for n in re.findall(r"\bs(\d+)\b", text)}
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        out |= set(range(int(a), int(b) + 1))
    return out


def too_young(code):
    """Loads to LDS that read a scalar register less than 5 wait states behind a vector instruction's write of it."""
    out = []
    for i, x in enumerate(code):
        if not is_lds_load(x):
            continue
        waits = 0
        for y in reversed(code[max(0, i - 5):i]):
            if waits >= 5:
                break
            if y.startswith("v_") and scalars(y.partition(" ")[2].split(",")[0]) & scalars(x):
                out.append(f"{y} | {x}")
                break
            waits += int(y.split()[1]) + 1 if y.startswith("s_nop") else 1
    return out


@pytest.mark.parametrize("code, found", [
    (["s_mov_b32 m0, s9", "global_load_lds_dwordx4 v[4:5], off"], 1),
    (["s_add_i32 m0, s9, 0x8000", "s_nop 0", "global_load_lds_dwordx4 v[4:5], off"], 0),
    (["s_mov_b32 m0, s9", "v_add_u32_e32 v1, v2, v3", "buffer_load_dwordx4 v26, s[36:39], 0 offen lds"], 0),
    (["s_add_i32 m0, s1, 4", "buffer_load_dwordx4 v26, s[36:39], 0 offen lds"], 1),
    (["s_mov_b32 m0, s9", "global_load_dwordx4 v[0:3], v[4:5], off"], 0),
])
def test_what_counts(code, found):
    assert len(without_wait(code)) == found


@pytest.mark.parametrize("kernel", ["prefix_kernel<", "agmm_persistent<", ""])
def test_m0(kernels, kernel):
    mine = {n: c for n, c in kernels.items() if kernel in n}
    assert any(is_lds_load(x) for c in mine.values() for x in c)
    assert {n: w[:2] for n, w in ((n, without_wait(c)) for n, c in mine.items()) if w} == {}


@pytest.mark.parametrize("code, found", [
    (["v_readfirstlane_b32 s36, v20", "s_nop 0", "buffer_load_dwordx4 v26, s[36:39], 0 offen lds"], 1),
    (["v_readlane_b32 s39, v20, 3", "s_nop 3", "buffer_load_dwordx4 v26, s[36:39], 0 offen lds"], 1),
    (["v_readfirstlane_b32 s36, v20", "s_nop 4", "buffer_load_dwordx4 v26, s[36:39], 0 offen lds"], 0),
    (["v_readfirstlane_b32 s40, v20", "s_nop 0", "buffer_load_dwordx4 v26, s[36:39], 0 offen lds"], 0),
    (["v_add_u32_e32 v1, s36, v20", "s_nop 0", "buffer_load_dwordx4 v26, s[36:39], 0 offen lds"], 0),
])
def test_what_is_too_young(code, found):
    assert len(too_young(code)) == found


def test_scalars(kernels):
    assert {n: w[:2] for n, w in ((n, too_young(c)) for n, c in kernels.items()) if w} == {}
