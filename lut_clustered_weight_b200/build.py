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
import re
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
CSRC = PKG / "csrc"
INCLUDE = PKG.parent / "include"
BUILD = PKG / "_build"
LIB = PKG / "libcq_b200.so"
BIND_SRC = CSRC / "bind.cpp"
BIND = PKG / "_cq_bind.so"
BIND_STAMP = BUILD / "bind.stamp"

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and Path(c).exists():
            return c
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _torch() -> Path:
    """torch's folder, found without importing it."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch not found")
    return Path(spec.submodule_search_locations[0])


def torch_version() -> str:
    text = (_torch() / "version.py").read_text()
    return re.search(r"__version__ *= *['\"](.*?)['\"]", text)[1]


def _bind_cmd(out: Path) -> list[str]:
    """g++ command of the CPython module: torch's headers and libraries, and the
    CUDA library beside it."""
    torch = _torch()
    cuda = Path(nvcc()).resolve().parent.parent
    inc = [torch / "include", torch / "include/torch/csrc/api/include", cuda / "include",
           sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
            f'-DCQ_TORCH_VERSION="{torch_version()}"',
            *[f"-isystem{i}" for i in inc], str(BIND_SRC), "-o", str(out), f"-L{PKG}",
            "-l:libcq_b200.so", "-Wl,-rpath,$ORIGIN", f"-L{torch / 'lib'}", "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _bind_lacks() -> str | None:
    """What is not here that the CPython module is built with, or None."""
    try:
        torch = _torch()
    except RuntimeError as e:
        return str(e)
    if shutil.which("g++") is None:
        return "g++ not found"
    for f in (torch / "include/torch/csrc/Exceptions.h", torch / "lib/libc10_cuda.so",
              Path(sysconfig.get_paths()["include"]) / "Python.h"):
        if not f.exists():
            return f"{f} not found"
    return None


def build_bind(force: bool = False, verbose: bool = False) -> None:
    """The CPython module, where its source, the C interface, torch or Python changed
    (it holds torch's C++ interface).  Without a compiler, torch's headers or a
    torch with CUDA it is left out with a warning: the package works without it, but
    for the calls that it marshals."""
    lacks = _bind_lacks()
    if lacks:
        warnings.warn(f"{BIND.name} is not built: {lacks}", stacklevel=2)
        return
    stamp = f"torch {torch_version()} {sysconfig.get_config_var('SOABI')}"
    newest = max(p.stat().st_mtime for p in (BIND_SRC, INCLUDE / "cq.h"))
    if (not force and BIND.exists() and BIND.stat().st_mtime >= newest and BIND_STAMP.exists()
            and BIND_STAMP.read_text() == stamp):
        return
    tmp = BIND.with_name(f"._cq_bind.{os.getpid()}.so")
    _run(_bind_cmd(tmp), verbose)
    os.replace(tmp, BIND)
    BIND_STAMP.write_text(stamp)


def _run(cmd, verbose: bool = False, show: bool = False) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiler failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if (verbose or show) and (r.stderr or r.stdout):
        print(r.stdout + r.stderr, flush=True)


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
        _run(cmd, verbose, ptxas_info)

    with ThreadPoolExecutor(max_workers=min(8, max(1, len(jobs)))) as ex:
        list(ex.map(run, jobs))
    if jobs or force or not LIB.exists():
        tmp = PKG / f".libcq_b200.{os.getpid()}.so"
        cmd = [nvcc(), *ARCH, "-shared", "-o", str(tmp), *map(str, objs), "-lcudart"]
        run(cmd)
        os.replace(tmp, LIB)
    build_bind(force, verbose)
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
