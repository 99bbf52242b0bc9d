"""Build liblucetree.so in-tree: every csrc/*.cu compiled for sm_103a in
parallel, then linked into one shared library with the extern "C" ABI of
include/lucetree.h."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.machinery
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build", "lucetree")
LIB = os.path.join(PKG, "liblucetree.so")
MARSHAL_SRC = os.path.join(PKG, "binding", "marshal.cpp")
# named for the Python that it is built for: another one neither loads nor reuses it
SUFFIX = importlib.machinery.EXTENSION_SUFFIXES[0]
MARSHAL = os.path.join(PKG, "_marshal" + SUFFIX)
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags():
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                   "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build_marshal(force: bool = False) -> str | None:
    """The binding's tensor checks as a Python extension (host code, against the
    installed torch).  The binding makes the same checks in Python where it is
    missing, so a host without Python's headers, or without torch (where only the C
    library is of use), gets a notice."""
    import sysconfig

    try:
        import torch
    except ImportError as e:
        print(f"the binding's tensor checks are not built: {e}", file=sys.stderr)
        return None
    # what was tried last, and how it went; a failure is tried again with `force`
    stamp = os.path.join(BUILD, "marshal" + SUFFIX + ".last")
    key = f"{torch.__version__} {os.path.getmtime(MARSHAL_SRC)}"
    last = open(stamp).read() if os.path.exists(stamp) else ""
    if not force and last == "failed " + key:
        return None
    if not force and last == "built " + key and os.path.exists(MARSHAL):
        return MARSHAL

    def note(how):
        os.makedirs(BUILD, exist_ok=True)
        with open(stamp, "w") as f:
            f.write(f"{how} {key}")

    root = os.path.dirname(torch.__file__)
    inc = os.path.join(root, "include")
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or "g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
           f'-DMARSHAL_TORCH_VERSION="{torch.__version__}"', "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], MARSHAL_SRC, "-o", tmp, "-L", os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = (r.stderr or f"exit code {r.returncode}") if r.returncode != 0 else ""
    except OSError as e:
        why = str(e)
    if why:
        print(f"the binding's tensor checks stay in Python:\n{why[-2000:]}", file=sys.stderr)
        if os.path.exists(MARSHAL):  # of an older source
            os.remove(MARSHAL)
        note("failed")
        return None
    os.replace(tmp, MARSHAL)
    note("built")
    return MARSHAL


def build(force: bool = False, verbose: bool = False, extra: list | None = None) -> str:
    if not force and up_to_date():
        build_marshal()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = _flags() + (extra or [])

    def one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        marshal = ex.submit(build_marshal, force)
        objs = list(ex.map(one, sources()))
        marshal.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
