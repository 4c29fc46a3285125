"""Build ``libvn.so`` in-tree with nvcc for sm_103a (GB300).

Usage: ``python -m virtual_noise_perturbed_gb300.build [--force] [-v]``.

Each ``csrc/*.cu`` file is compiled in parallel to ``_build/*.o`` and the
objects are linked into ``virtual_noise_perturbed_gb300/libvn.so`` (CUDA
runtime linked statically; the driver API is reached through the runtime's
entry-point query, so no link against libcuda is needed). ``csrc/vn_torch.cpp``, the
centre network's calls on torch tensors, is compiled beside them with the host compiler
into ``_binding.so``, which links to the library. A rebuild happens
only when a source or header is newer than the libraries, or when ``_binding.so`` was built for another
Python or torch than this one. Builds take a file lock,
so processes that start together (the ranks of one job, test workers) build
once: the others wait, then find the library current.
"""

from __future__ import annotations

import argparse
import concurrent.futures as cf
import fcntl
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libvn.so")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = [os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libvn.so")


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def binding_source() -> str:
    return os.path.join(CSRC, "vn_torch.cpp")


def _inputs() -> list:
    return sources() + [binding_source()] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) \
        + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _made_for() -> str:
    """What _binding.so is tied to: the interpreter's ABI, and torch's version and place."""
    try:
        torch_version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch_version = "?"
    return f"{sys.version} {sysconfig.get_config_var('SOABI')} torch {torch_version} in {_torch_dir()}"


def _stamp() -> str:
    return os.path.join(BUILD, "binding.made_for")


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    try:
        with open(_stamp()) as f:
            if f.read() != _made_for():
                return False
    except FileNotFoundError:
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(p) <= t for p in _inputs())


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)
    return r


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile and link libvn.so unless it is current; returns its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with open(os.path.join(BUILD, ".lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        try:
            if not force and up_to_date():  # another process built it while this one waited
                return LIB
            _compile_and_link(verbose, extra_flags)
        finally:
            fcntl.flock(lock, fcntl.LOCK_UN)
    return LIB


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("torch is required to build _binding.so")
    return list(spec.submodule_search_locations)[0]


def _compile_and_link(verbose: bool, extra_flags) -> None:
    cc = nvcc()
    flags = CFLAGS + list(extra_flags or [])
    torch_dir, cuda = _torch_dir(), os.path.dirname(os.path.dirname(os.path.realpath(cc)))
    cxx = os.environ.get("CXX") or "g++"
    bobj = os.path.join(BUILD, "vn_torch.o")
    objs = []
    cmds = [[cxx, "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE, "-I", os.path.join(torch_dir, "include"),
             "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
             "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
             "-c", binding_source(), "-o", bobj]]
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmds.append([cc, *ARCH, *flags, "-c", src, "-o", obj])
    with cf.ThreadPoolExecutor(max_workers=min(len(cmds), os.cpu_count() or 4)) as ex:
        list(ex.map(lambda c: _run(c, verbose), cmds))
    tmp = LIB + ".tmp"
    _run([cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static", "-Xlinker", "-soname=libvn.so"], verbose)
    os.replace(tmp, LIB)
    if os.path.exists(_stamp()):
        os.remove(_stamp())
    tmp = BINDING + ".tmp"
    _run([cxx, "-shared", "-o", tmp, bobj, "-L", PKG, "-l:libvn.so", "-Wl,-rpath,$ORIGIN",
          "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"],
         verbose)
    os.replace(tmp, BINDING)
    with open(_stamp(), "w") as f:
        f.write(_made_for())


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills per kernel")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_info else []
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose or a.ptxas_info, extra_flags=extra))
    return 0


if __name__ == "__main__":
    sys.exit(main())
