"""Build libtq.so in-tree for sm_103a (GB300) with nvcc.

Each translation unit compiles in parallel to an object under ``_build/``, then
one link produces ``quantised_kv_cache_gb300/_lib/libtq.so``. No cmake, no
torch extension machinery: the library is a plain C-ABI shared object.

Usage: ``python -m quantised_kv_cache_gb300.build [--force] [--verbose]``.
"""

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libtq.so")

SOURCES = ["tq_host.cpp", "tq_append.cu", "tq_decode.cu", "tq_dequant.cu", "tq_kivi.cu", "tq_noalloc.cu", "tq_decode2.cu", "tq_append2.cu",
           "tq_append_tc.cu", "tq_append_small.cu", "tq_append_bulk.cu", "tq_selftest.cu", "tq_q8_host.cpp",
           "tq_rotary.cu", "tq_q8_append.cu", "tq_q8_attend.cu", "tq_q8_prompt.cu", "tq_q8_weights.cu",
           "tq_q8_evict.cu", "tq_q8_bounds.cu", "tq_q8_select.cu", "tq_q8_scores.cu", "tq_q8_listed.cu",
           "tq_q8_listed_many.cu", "tq_q8_shared.cu", "tq_q8_prefix_many.cu", "tq_q8_own_many.cu", "tq_q8_both_many.cu"]
HEADERS = ["tq_internal.h", "tq_device.cuh", "tq_ptx.cuh", "tq_tcgen05.cuh", "tq_q8.h", "tq_q8_host.h", "tq_q8.cuh",
           "tq_q8_attend.cuh", "tq_q8_rows.cuh", "tq_q8_few.cuh", "tq_q8_many.cuh", "tq_q8_select.cuh", "tq_q8_solo.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    cand = [os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found (set NVCC or put /usr/local/cuda/bin on PATH)")


def _flags():
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr", "-diag-suppress=177",
                   "-I", os.path.join(ROOT, "include")]


def _newest_input_mtime():
    paths = [os.path.join(CSRC, s) for s in SOURCES + HEADERS] + [os.path.join(ROOT, "include", "tq.h"),
                                                                  os.path.abspath(__file__)]
    return max(os.path.getmtime(p) for p in paths)


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest_input_mtime():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    nvcc = nvcc_path()
    flags = _flags() + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD, src + ".o")
        cmd = [nvcc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode:
            raise RuntimeError(f"nvcc failed on {src}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode:
        raise RuntimeError("link failed")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills / shared memory")
    args = ap.parse_args()
    extra = ["-Xptxas", "-v"] if args.ptxas_info else None
    print(build(force=args.force or args.ptxas_info, verbose=args.verbose or args.ptxas_info, extra_flags=extra))
