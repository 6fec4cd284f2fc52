"""Compile-time resources of the layer library's kernels (no device work), as
tests/test_kernel_resources.py reads them: no scratch, no spilled vector
registers, registers that fit the occupancy the LDS allows; and the wait
states before memory instructions that read scalars or store results."""
import os
import re
import subprocess
import tempfile

import pytest

from tests import test_kernel_resources as k
from tests import test_rows_resources as r


@pytest.fixture(scope="module")
def lib():
    from dense_gemm_nt_amd import build
    if build.stale_layer():
        build.build_layer()
    return build.LAYER_LIB


@pytest.fixture(scope="module")
def kernels(lib):
    return k._read_kernels(lib)


def _count(kernels, part):
    return sum(part in n for n in kernels)


def test_every_family_is_built(kernels):
    # the gated block's tiles, 2 in x 3 out types; its sums' gradients, one out type each
    assert _count(kernels, "gemm_nt_kernel_gated") == 5 * 6 and _count(kernels, "gemm_nt_kernel_gategrad") == 4 * 2
    assert _count(kernels, "gemm_nt_w4_gated") == 6 and _count(kernels, "gemm_nt_w4_gategrad") == 2
    assert _count(kernels, "gemm_nt_pp2_gatedI") == 6 and _count(kernels, "gemm_nt_pp2_gategrad") == 2
    assert _count(kernels, "gemm_nt_pp2_gated_dx") == 6 and _count(kernels, "gemm_nt_pp2_gated_dw") == 6
    # 8-bit integers, three out types
    assert _count(kernels, "gemm_nt_kernel_int8") == 5 * 3 and _count(kernels, "gemm_nt_pp2_int8") == 3
    assert _count(kernels, "gemm_nt_w4_int8") == 3 and _count(kernels, "int8_few") == 2 * 3
    # the update's tiles; the 128 x 128 tile for MN-major B: the update's, and the input gradient's
    assert _count(kernels, "gemm_nt_kernel_ortho") == 3 and _count(kernels, "gemm_nt_pp2_ortho") == 2
    assert _count(kernels, "rows_tile") == 1 + 6
    # and the 64 x 64 one
    assert _count(kernels, "tile64") == 1 + 6


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
    # the two-stage ring, the 64 x 64 tiles and the tile for MN-major B run two blocks a compute unit
    two = [n for n in kernels if ("gemm_nt_kernel" in n and ("Li4ELi2E" in n or "Li64ELi64ELi64E" in n)) or "rows_tile" in n or "tile64" in n]
    assert len(two) == (2 * 6 + 2) + 2 * 3 + 2 + 7 + 7
    for n in two:
        waves = kernels[n][".max_flat_workgroup_size"] // 64
        assert 2 * kernels[n][".group_segment_fixed_size"] <= k.LDS_BYTES, n
        assert 2 * (waves // 4) * kernels[n][".vgpr_count"] <= k.REGS_PER_SIMD_LANE, (n, kernels[n][".vgpr_count"])


@pytest.mark.skipif(not os.path.exists(k.OBJDUMP), reason="llvm-objdump not installed")
def test_scalars_are_settled_before_loads(lib):
    r.test_scalars_are_settled_before_loads(lib)


@pytest.mark.skipif(not os.path.exists(k.OBJDUMP), reason="llvm-objdump not installed")
def test_waits_before_results_are_stored(lib):
    """No LDS or memory store stands within the wait states of a matrix instruction whose result
    it stores (text order, every kernel)."""
    checked = 0
    for co in k._code_objects(lib):
        with tempfile.TemporaryDirectory() as d:
            path = os.path.join(d, "co.o")
            open(path, "wb").write(co)
            text = subprocess.run([k.OBJDUMP, "-d", "--no-show-raw-insn", path], check=True, capture_output=True,
                                  text=True).stdout
        recent = []
        for line in text.splitlines():
            s = line.split("//")[0].strip()
            if re.match(r"^[0-9a-f]+ <(\S+)>:$", line):
                recent = []
                continue
            if not s:
                continue
            op = s.split()[0]
            args = s[len(op):]
            recent = [(left - 1, regs) for left, regs in recent if left > 1]
            if op.startswith("v_mfma"):
                recent.append((20, r._registers(args.split(",")[0])))      # 16 passes and 3, at most
                checked += 1
            elif op == "s_nop":
                recent = [(left - int(args), regs) for left, regs in recent if left > int(args)]
            elif re.match(r"(ds_write|ds_store|global_store|buffer_store)", op):
                assert not [regs for _, regs in recent if regs & r._registers(args)], s
    assert checked > 0
