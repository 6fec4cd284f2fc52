"""The kernels of a feed-forward layer's products on perf/more_operators.py's listed cases: the
program to put under rocprofv3, and the table of profiles/layer_kernels.md from what it
writes, as profile_rows makes them for the row-indexed products.

    P="python3 -m dense_gemm_nt_amd.profile_layer run"
    rocprofv3 --kernel-trace --output-format csv -d OUT -o trace -- $P
    rocprofv3 --pmc FETCH_SIZE --output-format csv -d OUT -o fetch -- $P
    rocprofv3 --pmc WRITE_SIZE --output-format csv -d OUT -o write -- $P
    rocprofv3 --pmc SQ_VALU_MFMA_BUSY_CYCLES GRBM_GUI_ACTIVE SQ_LDS_BANK_CONFLICT SQ_INSTS_VALU \\
        --output-format csv -d OUT -o sq -- $P
    python3 -m dense_gemm_nt_amd.profile_layer table OUT > profiles/layer_kernels.md
"""
from __future__ import annotations

import sys

from . import profile_rows as p

CASES = "more_operators"


def product(case, i, n):
    """The update's two squares share a kernel: in turn X X^T and the polynomial's A^2, once a
    step each."""
    if case["op"] == "ortho" and n == 2 * p.cases_module(CASES).STEPS:
        return "A^2" if i % 2 else "X X^T"
    return None


def main():
    if sys.argv[1:] == ["run"]:
        p.run(CASES)
    elif len(sys.argv) == 3 and sys.argv[1] == "table":
        lines, scale = p.table(sys.argv[2], CASES, product)
        print(p.heading("products of a feed-forward layer", "libgemm_layer.so", CASES, "profile_layer", scale))
        print("\n".join(lines))
    else:
        raise SystemExit(__doc__)


if __name__ == "__main__":
    main()
