"""Build the CUDA library libspecverify.so in-tree with nvcc (sm_103a only).

    python -m speculative_decoding_verify_07_gb300.build

Each translation unit compiles in parallel; the shared object lands in
speculative_decoding_verify_07_gb300/lib/.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "lib")
OBJDIR = os.path.join(ROOT, "_build")
LIB = os.path.join(LIBDIR, "libspecverify.so")
SOURCES = ["spec_verify.cu", "spec_kernel.cu", "spec_commit.cu", "spec_api.cu", "spec_noalloc.cu", "spec_draft.cu",
           "spec_cache.cu", "spec_attend.cu", "spec_attend_rows.cu", "spec_attend_wide.cu",
           "spec_recur.cu", "spec_conv.cu", "spec_scan.cu", "spec_shared.cu", "spec_attend_rows_common.cu",
           "spec_attend_rows_own.cu", "spec_attend_wide_common.cu", "spec_attend_wide_own.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def build(verbose: bool = False, ptxas_info: bool = False, defines: tuple[str, ...] = (), lib: str = LIB,
          objdir: str = OBJDIR) -> str:
    """Compiles and links the library.  A variant with other `defines` (NAME=VALUE) gets its own lib and objdir."""
    os.makedirs(os.path.dirname(lib), exist_ok=True)
    os.makedirs(objdir, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    extra += [f"-D{d}" for d in defines]

    def compile_one(src):
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-c",
               os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    for _, log in results:
        if (verbose or ptxas_info) and log:
            print(log, file=sys.stderr)
    objs = [o for o, _ in results]
    tmp = lib + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="--ptxas" in sys.argv))
