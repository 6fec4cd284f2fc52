"""The table of the row-indexed kernels from rocprofv3's files, on made ones."""
import csv

from dense_gemm_nt_amd import profile_rows as p


def _write(path, rows):
    with open(path, "w", newline="") as f:
        w = csv.DictWriter(f, fieldnames=list(rows[0]))
        w.writeheader()
        w.writerows(rows)


def test_table(tmp_path):
    n = len(p.cases_module().listed())
    trace, counted = [], {"fetch": [], "write": [], "sq": []}

    def dispatch(name, ns, fetch, write, busy):
        i = len(trace) + 1
        trace.append(dict(Dispatch_Id=i, Kernel_Name=name, Grid_Size_X=1024, Grid_Size_Y=2, Grid_Size_Z=1,
                          Workgroup_Size_X=256, Workgroup_Size_Y=1, Workgroup_Size_Z=1, Start_Timestamp=100,
                          End_Timestamp=100 + ns))
        for k, c in (("fetch", {"FETCH_SIZE": fetch}), ("write", {"WRITE_SIZE": write}),
                     ("sq", {"SQ_VALU_MFMA_BUSY_CYCLES": busy, "GRBM_GUI_ACTIVE": 8000.0,
                             "SQ_LDS_BANK_CONFLICT": 3000.0})):
            counted[k] += [dict(Dispatch_Id=i, Kernel_Name=name, Counter_Name=a, Counter_Value=b) for a, b in c.items()]

    for case in range(n):
        dispatch("at::normal_kernel", 5, 1, 1, 0)
        for call in range(p.CALLS):
            slow = 50000 if call < p.WARM else 0
            dispatch("void gnt::(anonymous namespace)::first<0, 1>(gnt::Args)", 2000 + slow, 1024, 512, 512000.0)
            dispatch("void gnt::second(gnt::Args)", 3000, 0, 0, 0.0)
    dispatch("__amd_rocclr_copyBuffer", 9, p.COPY_MB * 512, p.COPY_MB * 1024, 0)
    _write(tmp_path / "trace_kernel_trace.csv", trace)
    for k, rows in counted.items():
        _write(tmp_path / ("%s_counter_collection.csv" % k), rows)
    lines, scale = p.table(str(tmp_path))
    assert scale == {"fetch": 2.0, "write": 1.0} and len(lines) == 3 * n
    # 1 MiB x 2 read, half a MiB written in 2 us; 512000 / 1024 of 8000 / 8 cycles
    assert lines[1] == "| first<0, 1> | 4x2x1 | 2.0 | 2.1 | 0.5 | 1.31 | 50 % | 3 |"
    assert lines[2].startswith("| second | 4x2x1 | 3.0 | 0.0 | 0.0 | 0.00 | 0 % |")
