"""Compile-time resources of the row-indexed kernels' library (no device work), as
tests/test_kernel_resources.py reads them: no scratch, no spilled vector
registers, registers that fit the occupancy the LDS allows; and the wait
states between a matrix instruction and the stores of its results."""
import os
import re
import subprocess
import tempfile

import pytest

from tests import test_kernel_resources as k


@pytest.fixture(scope="module")
def lib():
    from dense_gemm_nt_amd import build
    if build.stale_rows():
        build.build_rows()
    return build.ROWS_LIB


@pytest.fixture(scope="module")
def kernels(lib):
    return k._read_kernels(lib)


def _count(kernels, part):
    return sum(part in n for n in kernels)


def test_every_family_is_built(kernels):
    # four tile forms with adapters, 2 in x 3 out types; the four-wave tile; the
    # ping-pong tile in two layouts; routed: two tiles and three layouts
    assert _count(kernels, "gemm_nt_kernel_lora") == 4 * 6 and _count(kernels, "gemm_nt_w4_lora") == 6
    assert _count(kernels, "gemm_nt_pp2_lora") == 2 * 6
    assert _count(kernels, "gemm_nt_kernel_routed") == 2 * 6 and _count(kernels, "gemm_nt_pp2_routed") == 3 * 6
    # the 128 x 128 tile for MN-major weights, with adapters and routed
    assert _count(kernels, "rows_tile") == 2 * 6
    assert not [n for n in kernels if re.search(r"gemm_nt_(kernel|pp2|w4)I", n)]    # the plain tiles are not


def test_no_scratch_no_spills(kernels):
    for n, m in kernels.items():
        assert m[".private_segment_fixed_size"] == 0, (n, m[".private_segment_fixed_size"])
        assert m[".vgpr_spill_count"] == 0, (n, m[".vgpr_spill_count"])
        assert not m[".uses_dynamic_stack"], n


def test_lds_and_register_budget(kernels):
    for n, m in kernels.items():
        assert m[".group_segment_fixed_size"] <= k.LDS_BYTES, n
        waves = -(-m[".max_flat_workgroup_size"] // 64)
        assert -(-waves // 4) * m[".vgpr_count"] <= k.REGS_PER_SIMD_LANE, n
    # the two-stage ring and the tile for MN-major weights run two blocks a compute unit
    two = [n for n in kernels if "gemm_nt_kernel_lora" in n and "Li4ELi2E" in n or "rows_tile" in n]
    assert len(two) == 6 + 12
    for n in two:
        waves = kernels[n][".max_flat_workgroup_size"] // 64
        assert 2 * kernels[n][".group_segment_fixed_size"] <= k.LDS_BYTES, n
        assert 2 * (waves // 4) * kernels[n][".vgpr_count"] <= k.REGS_PER_SIMD_LANE, (n, kernels[n][".vgpr_count"])


def _registers(text):
    out = set()
    for m in re.finditer(r"\b([va])\[(\d+):(\d+)\]|\b([va])(\d+)\b", text):
        if m.group(1):
            out |= {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
        else:
            out.add((m.group(4), int(m.group(5))))
    return out


@pytest.mark.skipif(not os.path.exists(k.OBJDUMP), reason="llvm-objdump not installed")
def test_waits_before_results_are_stored(lib):
    """No LDS or memory store stands within the wait states of a matrix instruction
    whose result it stores (text order, in the kernels with MFMA loops of their own)."""
    checked = 0
    for co in k._code_objects(lib):
        with tempfile.TemporaryDirectory() as d:
            path = os.path.join(d, "co.o")
            open(path, "wb").write(co)
            text = subprocess.run([k.OBJDUMP, "-d", "--no-show-raw-insn", path], check=True, capture_output=True,
                                  text=True).stdout
        name, recent = None, []
        for line in text.splitlines():
            m = re.match(r"^[0-9a-f]+ <(\S+)>:$", line)
            if m:
                name, recent = m.group(1), []
                continue
            if name is None or not any(f in name for f in ("lora_shrink", "lora_grad", "rows_tile")):
                continue
            s = line.split("//")[0].strip()
            if not s:
                continue
            op = s.split()[0]
            args = s[len(op):]
            recent = [(left - 1, r) for left, r in recent if left > 1]
            if op.startswith("v_mfma"):
                # 8 or 16 passes and 3, at most
                recent.append((20 if "32x32" in op else 12, _registers(args.split(",")[0])))
                checked += 1
            elif op == "s_nop":
                n = int(args)
                recent = [(left - n, r) for left, r in recent if left > n]
            elif re.match(r"(ds_write|ds_store|global_store|buffer_store)", op):
                hit = [left for left, r in recent if r & _registers(args)]
                assert not hit, (name, s, hit)
    assert checked > 0


def _scalars(text):
    out = {"vcc"} if "vcc" in text else set()
    for m in re.finditer(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text):
        out |= set(range(int(m.group(1)), int(m.group(2)) + 1)) if m.group(1) else {int(m.group(3))}
    return out


@pytest.mark.skipif(not os.path.exists(k.OBJDUMP), reason="llvm-objdump not installed")
def test_scalars_are_settled_before_loads(lib):
    """A scalar that a vector instruction wrote is read by a memory instruction five wait
    states later at the earliest (text order).  The compiler sees to that for its
    own loads, but not for those written in asm, whose scalars it may have put
    away in vector registers."""
    checked = 0
    for co in k._code_objects(lib):
        with tempfile.TemporaryDirectory() as d:
            path = os.path.join(d, "co.o")
            open(path, "wb").write(co)
            text = subprocess.run([k.OBJDUMP, "-d", "--no-show-raw-insn", path], check=True, capture_output=True,
                                  text=True).stdout
        recent = []
        for line in text.splitlines():
            if re.match(r"^[0-9a-f]+ <(\S+)>:$", line):
                recent = []
                continue
            s = line.split("//")[0].strip()
            if not s:
                continue
            op = s.split()[0]
            args = s[len(op):]
            if re.match(r"(buffer|global)_", op):
                checked += 1
                hit = [left for left, r in recent if r & _scalars(args)]
                assert not hit, (s, hit)
            states = int(args, 0) + 1 if op == "s_nop" else 1
            recent = [(left - states, r) for left, r in recent if left > states]
            if re.match(r"v_(readlane|readfirstlane|cmp)", op):
                recent.append((5, _scalars(args.split(",")[0])))
    assert checked > 0


@pytest.mark.skipif(not os.path.exists(k.OBJDUMP), reason="llvm-objdump not installed")
def test_scalars_are_settled_before_loads_of_the_first_library():
    """The same of libgemm_nt.so, whose persistent kernel keeps scalars in vector registers."""
    from dense_gemm_nt_amd import build
    if build.stale():
        build.build()
    test_scalars_are_settled_before_loads(build.LIB)
