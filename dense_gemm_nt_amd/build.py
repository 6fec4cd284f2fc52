"""Compile the HIP library (gfx950) in place: ``python -m dense_gemm_nt_amd.build``."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
# the host side and one translation unit per group of kernel instantiations,
# compiled in parallel and linked into one shared library
SOURCES = [os.path.join(CSRC, f) for f in (
    "gemm_nt.hip", "launch_tiles_a.hip", "launch_tiles_b.hip",
    "launch_pp2.hip", "launch_pp2_km.hip", "launch_pp2_mk.hip", "launch_pp2_mm.hip",
    "launch_pp2_f8_e4e4.hip", "launch_pp2_f8_e4e5.hip", "launch_pp2_f8_e5e4.hip",
    "launch_pp2_f8_e5e5.hip", "launch_pp2_grouped.hip", "launch_pp2_persistent.hip", "launch_w4.hip")]
HEADERS = [os.path.join(CSRC, f) for f in ("gemm_nt_common.hpp", "gemm_nt_kernel.hpp",
                                           "gemm_nt_pp2.hpp", "gemm_nt_w4.hpp", "gemm_nt_trace.hpp",
                                           "gemm_nt_launch.hpp", "gemm_nt_ext.hpp", "gemm_nt_plan.hpp",
                                           "launch_pp2.hip",
                                           "launch_pp2_f8.hip", "launch_tiles_a.hip")] + \
    [os.path.join(ROOT, "include", "gemm_nt.h")]
LIB = os.path.join(PKG, "libgemm_nt.so")
# the row-indexed products (include/gemm_rows.h): a library of its own, whose
# tiles are the headers above with an addition
ROWS = os.path.join(CSRC, "rows")
ROWS_SOURCES = [os.path.join(ROWS, f) for f in (
    "rows_lora.hip", "rows_route.hip", "rows_routed.hip", "launch_lora_tiles.hip",
    "launch_lora_tiles_b.hip", "launch_lora_w4.hip", "launch_lora_pp2.hip",
    "launch_lora_pp2_km.hip", "launch_routed_tiles.hip", "launch_routed_pp2.hip",
    "launch_routed_pp2_km.hip", "launch_routed_pp2_mm.hip", "launch_rows_tile.hip")]
ROWS_HEADERS = [os.path.join(ROWS, f) for f in ("rows_common.hpp", "rows_group.hpp",
                                                "rows_host.hpp", "rows_index.hpp", "rows_launch.hpp",
                                                "rows_tile.hpp")] + \
    [os.path.join(ROOT, "include", "gemm_rows.h")]
ROWS_LIB = os.path.join(PKG, "libgemm_rows.so")
# the products of a feed-forward layer (include/gemm_layer.h), likewise
LAYER = os.path.join(CSRC, "layer")
LAYER_SOURCES = [os.path.join(LAYER, f) for f in (
    "layer_gated.hip", "layer_int8.hip", "launch_gated_tiles.hip", "launch_gated_tiles_b.hip",
    "launch_gategrad_tiles.hip", "launch_gategrad_tiles_b.hip", "launch_gated_w4.hip",
    "launch_gategrad_w4.hip", "launch_gated_pp2.hip", "launch_gategrad_pp2.hip", "launch_gated_dx.hip",
    "launch_gated_dx_tile.hip", "launch_gated_dw.hip", "launch_int8_tiles.hip", "launch_int8_pp2.hip", "layer_ortho.hip",
    "launch_ortho.hip")]
LAYER_HEADERS = [os.path.join(LAYER, f) for f in ("layer_common.hpp", "layer_host.hpp", "layer_launch.hpp",
                                                  "paired_ext.hpp", "int8_ext.hpp", "ortho_common.hpp",
                                                  "ortho_ext.hpp", "tile64.hpp")] + \
    [os.path.join(ROOT, "include", "gemm_layer.h")]
LAYER_LIB = os.path.join(PKG, "libgemm_layer.so")
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def flags() -> list:
    return ["--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC",
            "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
            # packed FP32 VALU forms are kept out of the generated code
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wno-unused-command-line-argument"]


def command(out: str, extra=()) -> list:
    """One hipcc line that compiles and links every source (used by tools that
    want a single command, e.g. with extra -R remarks)."""
    return [hipcc(), *flags(), "-shared", *extra, *SOURCES, "-o", out]


def _run(cmd):
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(ln for ln in res.stdout.splitlines() if "packed-fp32-ops" not in ln)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed: %s\n%s" % (" ".join(cmd), out))
    return out


def build(verbose: bool = False, jobs: int = 0, out: str = LIB, defines=(), sources=None) -> str:
    """Compile every source and link them into `out` (the library by default;
    `defines` are extra -D flags, e.g. for an instrumented copy)."""
    sources = SOURCES if sources is None else sources
    tmpdir = tempfile.mkdtemp(prefix="gemm_nt_build_")
    try:
        objs = [os.path.join(tmpdir, os.path.basename(src) + ".o") for src in sources]
        cmds = [[hipcc(), *flags(), *defines, "-c", src, "-o", obj] for src, obj in zip(sources, objs)]
        jobs = jobs or max(1, min(len(cmds), os.cpu_count() or 1, 8))
        if verbose:
            for c in cmds:
                print(" ".join(c), flush=True)
        with concurrent.futures.ThreadPoolExecutor(jobs) as ex:
            list(ex.map(_run, cmds))
        tmp = out + ".tmp%d" % os.getpid()
        link = [hipcc(), "--offload-arch=" + ARCH, "-shared", "-fPIC", *objs, "-o", tmp]
        if verbose:
            print(" ".join(link), flush=True)
        _run(link)
        os.replace(tmp, out)
    finally:
        shutil.rmtree(tmpdir, ignore_errors=True)
    return out


def build_rows(verbose: bool = False, jobs: int = 0) -> str:
    """The library of the row-indexed products."""
    return build(verbose, jobs, ROWS_LIB, sources=ROWS_SOURCES)


def build_layer(verbose: bool = False, jobs: int = 0) -> str:
    """The library of a feed-forward layer's products."""
    return build(verbose, jobs, LAYER_LIB, sources=LAYER_SOURCES)


def stale_layer() -> bool:
    if not os.path.exists(LAYER_LIB):
        return True
    t = os.path.getmtime(LAYER_LIB)
    return any(os.path.getmtime(f) > t for f in LAYER_SOURCES + LAYER_HEADERS + ROWS_HEADERS + HEADERS)


def stale_rows() -> bool:
    if not os.path.exists(ROWS_LIB):
        return True
    t = os.path.getmtime(ROWS_LIB)
    return any(os.path.getmtime(f) > t for f in ROWS_SOURCES + ROWS_HEADERS + HEADERS)


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in SOURCES + HEADERS)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
    print(build_rows(verbose="-v" in sys.argv))
    print(build_layer(verbose="-v" in sys.argv))
