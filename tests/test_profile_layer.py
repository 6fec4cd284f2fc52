"""The table of the layer products' kernels: its heading, and the products that share a kernel."""
import csv

import pytest

from dense_gemm_nt_amd import profile_layer as l
from dense_gemm_nt_amd import profile_rows as p


def _write(path, rows):
    with open(path, "w", newline="") as f:
        w = csv.DictWriter(f, fieldnames=list(rows[0]))
        w.writeheader()
        w.writerows(rows)


@pytest.fixture
def folder(tmp_path):
    """Files of a call of two squares and a step for every case, a begin before the steps."""
    trace, counted = [], {"fetch": [], "write": [], "sq": []}

    def dispatch(name, ns, fetch=0, write=0):
        i = len(trace) + 1
        trace.append(dict(Dispatch_Id=i, Kernel_Name=name, Grid_Size_X=1024, Grid_Size_Y=1, Grid_Size_Z=1,
                          Workgroup_Size_X=256, Workgroup_Size_Y=1, Workgroup_Size_Z=1, Start_Timestamp=100,
                          End_Timestamp=100 + ns))
        for k, c in (("fetch", {"FETCH_SIZE": fetch}), ("write", {"WRITE_SIZE": write}),
                     ("sq", {"SQ_VALU_MFMA_BUSY_CYCLES": 0, "GRBM_GUI_ACTIVE": 8000.0, "SQ_LDS_BANK_CONFLICT": 0})):
            counted[k] += [dict(Dispatch_Id=i, Kernel_Name=name, Counter_Name=a, Counter_Value=b) for a, b in c.items()]
    for case in p.cases_module(l.CASES).listed():
        dispatch("at::normal_kernel", 5, 1, 1)
        for call in range(p.CALLS):
            dispatch("void gnt::begin(gnt::Args)", 4000)
            for step in range(p.cases_module(l.CASES).STEPS):
                dispatch("void gnt::square<1>(gnt::Args)", 7000)
                dispatch("void gnt::square<1>(gnt::Args)", 2000)
                dispatch("void gnt::step(gnt::Args)", 9000)
    dispatch("__amd_rocclr_copyBuffer", 9, p.COPY_MB * 1024, p.COPY_MB * 1024)
    _write(tmp_path / "trace_kernel_trace.csv", trace)
    for k, rows in counted.items():
        _write(tmp_path / ("%s_counter_collection.csv" % k), rows)
    return str(tmp_path)


def test_products_that_share_a_kernel_are_apart(folder):
    lines, _ = p.table(folder, l.CASES, l.product)
    at = next(i for i, s in enumerate(lines) if s.startswith("| **ortho_small**"))
    assert [s.split(" | ")[0] for s in lines[at + 1:at + 5]] == ["| begin", "| square<1>: X X^T", "| square<1>: A^2", "| step"]
    assert [s.split(" | ")[2] for s in lines[at + 1:at + 5]] == ["4.0", "7.0", "2.0", "9.0"]
    # elsewhere a kernel's launches are one
    assert [s.split(" | ")[0] for s in lines[1:4]] == ["| begin", "| square<1>", "| step"]


def test_headings_name_their_own_files():
    scale = {"fetch": 2.0, "write": 1.0}
    text = p.heading("products of a feed-forward layer", "libgemm_layer.so", l.CASES, "profile_layer", scale)
    for part in ("# Kernels of the products of a feed-forward layer", "`libgemm_layer.so`", "`perf/more_operators.py`",
                 "`dense_gemm_nt_amd/profile_layer.py`", "FETCH_SIZE x 2.000", "%d MiB" % p.COPY_MB):
        assert part in text, part
    assert "gemm_rows" not in text and "profile_rows" not in text and "perf/operators" not in text
    assert "%" not in text
    old = open(p.os.path.join(p.ROOT, "profiles", "rows_kernels.md")).read()
    rows = p.heading("products whose weight is picked per row", "libgemm_rows.so", "operators", "profile_rows", scale)
    assert old.splitlines()[0] == rows.splitlines()[0] and old.splitlines()[2] == rows.splitlines()[2]
