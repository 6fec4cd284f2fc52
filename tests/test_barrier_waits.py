"""LDS writes and barriers in the built libraries (no device work): a barrier orders the waves of
a block, not what they still have in flight, so what one wave wrote to LDS is there for the others
behind a barrier only if it waited for the write (lgkmcnt) before the barrier; and a word that
the others go on to overwrite has to have been read."""
import os
import re
import subprocess
import tempfile

import pytest

from dense_gemm_nt_amd import build
from tests import test_kernel_resources as k

LIBS = {"gemm_nt": (build.LIB, build.stale, build.build), "gemm_rows": (build.ROWS_LIB, build.stale_rows, build.build_rows),
        "gemm_layer": (build.LAYER_LIB, build.stale_layer, build.build_layer)}


def unwaited(text, ops=("ds_write", "ds_store", "ds_read_b32", "ds_load_b32")):
    """(kernel, operation) of every LDS operation of `ops` that a barrier follows (text order) with
    no wait for it between; and how many of them there are."""
    found, seen, name, out = [], 0, None, None
    for line in text.splitlines():
        m = re.match(r"^[0-9a-f]+ <(\S+)>:$", line)
        if m:
            name, out = m.group(1), None
            continue
        s = line.split("//")[0].strip()
        if s.startswith(ops):
            out, seen = s, seen + 1
        elif s.startswith("s_waitcnt"):
            if "lgkmcnt(0)" in s or s == "s_waitcnt 0":
                out = None
        elif s.startswith("s_barrier") and out:
            found.append((name, out))
            out = None
    return found, seen


def test_finds_a_missing_wait():
    text = "0000 <a>:\n ds_write_b32 v1, v2 // x\n s_cbranch_execz 4\n s_barrier\n"
    assert unwaited(text) == ([("a", "ds_write_b32 v1, v2")], 1)
    assert unwaited(text.replace("s_barrier", "s_waitcnt vmcnt(1) lgkmcnt(0)\n s_barrier")) == ([], 1)
    assert unwaited(text.replace("s_barrier", "s_waitcnt lgkmcnt(1)\n s_barrier"))[0]
    assert unwaited("0000 <a>:\n ds_read_b32 v1, v2\n s_barrier\n")[0]


@pytest.mark.skipif(not os.path.exists(k.OBJDUMP), reason="llvm-objdump not installed")
@pytest.mark.parametrize("name", LIBS)
def test_writes_are_waited_for_before_barriers(name):
    lib, stale, make = LIBS[name]
    if stale():
        make()
    seen = 0
    for co in k._code_objects(lib):
        with tempfile.TemporaryDirectory() as d:
            path = os.path.join(d, "co.o")
            open(path, "wb").write(co)
            text = subprocess.run([k.OBJDUMP, "-d", "--no-show-raw-insn", path], check=True, capture_output=True,
                                  text=True).stdout
        found, n = unwaited(text)
        seen += n
        assert not found, found[:8]
    assert seen > 0
