"""Build the sm_100a CUDA library in-tree: lut_clustered_weight_b200/libcq_b200.so,
and the CPython module _cq_bind.so (tensor checks of some entry points) beside it.

    python lut_clustered_weight_b200/build.py [--force] [-v] [--ptxas-info]

(Run it by path: importing the package itself loads the library.)

Every .cu under csrc/ is compiled with nvcc for sm_100a only and linked into
one shared library whose exported symbols are the C ABI of include/cq.h.
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
CSRC = PKG / "csrc"
INCLUDE = PKG.parent / "include"
BUILD = PKG / "_build"
LIB = PKG / "libcq_b200.so"
BIND_SRC = CSRC / "bind.cpp"
BIND = PKG / "_cq_bind.so"

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and Path(c).exists():
            return c
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _bind_cmd(out: Path) -> list[str]:
    """g++ command of the CPython module: torch's headers and libraries (found
    without importing torch), and the CUDA library beside it."""
    torch = Path(importlib.util.find_spec("torch").submodule_search_locations[0])
    cuda = Path(nvcc()).resolve().parent.parent
    inc = [torch / "include", torch / "include/torch/csrc/api/include", cuda / "include",
           sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
            *[f"-isystem{i}" for i in inc], str(BIND_SRC), "-o", str(out), f"-L{PKG}",
            "-l:libcq_b200.so", "-Wl,-rpath,$ORIGIN", f"-L{torch / 'lib'}", "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _sources():
    return sorted(CSRC.glob("*.cu"))


def _deps():
    return sorted(list(CSRC.glob("*.cuh")) + list(CSRC.glob("*.h")) + list(INCLUDE.glob("*.h")))


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> Path:
    BUILD.mkdir(exist_ok=True)
    newest_dep = max((p.stat().st_mtime for p in _deps()), default=0)
    srcs = _sources()
    objs = []
    jobs = []
    for s in srcs:
        o = BUILD / (s.stem + ".o")
        objs.append(o)
        if force or ptxas_info or not o.exists() or o.stat().st_mtime < max(s.stat().st_mtime, newest_dep):
            cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-I", str(INCLUDE), "-c", str(s), "-o", str(o)]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if (verbose or ptxas_info) and (r.stderr or r.stdout):
            print(r.stdout + r.stderr, flush=True)

    with ThreadPoolExecutor(max_workers=min(8, max(1, len(jobs)))) as ex:
        list(ex.map(run, jobs))
    if jobs or force or not LIB.exists():
        tmp = PKG / f".libcq_b200.{os.getpid()}.so"
        cmd = [nvcc(), *ARCH, "-shared", "-o", str(tmp), *map(str, objs), "-lcudart"]
        run(cmd)
        os.replace(tmp, LIB)
    newest = max(p.stat().st_mtime for p in (BIND_SRC, INCLUDE / "cq.h"))
    if force or not BIND.exists() or BIND.stat().st_mtime < newest:
        tmp = PKG / f"._cq_bind.{os.getpid()}.so"
        run(_bind_cmd(tmp))
        os.replace(tmp, BIND)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills / smem")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose, ptxas_info=a.ptxas_info))


if __name__ == "__main__":
    sys.exit(main())
