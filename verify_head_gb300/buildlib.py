"""Build libverifyhead.so (sm_103a) in-tree with nvcc.

Each .cu file under csrc/ is compiled in parallel, then linked into one
shared library next to this file.  Only one -gencode (sm_103a); host code is
portable (x86_64 and aarch64).  Beside it _marshal_<versions>.so, the compiled
argument marshalling of the norm and log-probability calls: it needs Python's
and torch's headers, and where they are missing the binding marshals in Python.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libverifyhead.so")
LIB_DEBUG = os.path.join(HERE, "libverifyhead_debug.so")  # -DVH_DEBUG: device-side index guards
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA library cannot be built")
    return path


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def marshal_path() -> str:
    """Where the marshalling for the running interpreter and torch lies.  It reads tensors by torch's own layout, so a
    file that was compiled against another Python, torch or C++ ABI must not be loaded: the name says which they were."""
    import torch
    tag = "-".join((sysconfig.get_config_var("SOABI") or sys.implementation.cache_tag, torch.__version__,
                    str(getattr(torch.version, "git_version", ""))[:10], f"abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"))
    return os.path.join(HERE, "_marshal_" + re.sub(r"[^0-9A-Za-z.]+", "_", tag) + ".so")


def build_marshal(force: bool = False):
    """Compiles the marshalling with the host compiler against the running torch; returns its path, or None (with the
    compiler's message on stderr) where that is not possible."""
    deps = (MARSHAL_SRC, os.path.join(ROOT, "include", "verifyhead.h"))
    try:
        import torch
        out = marshal_path()
        if not force and os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps):
            return out
        top = os.path.dirname(torch.__file__)
        cuda = os.path.dirname(os.path.dirname(nvcc()))
        inc = [os.path.join(top, "include"), os.path.join(top, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
        lib = os.path.join(top, "lib")
        tmp = out + f".tmp{os.getpid()}"
        cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *("-I" + p for p in inc), MARSHAL_SRC,
               "-o", tmp, "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath," + lib]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(r.stderr[-2000:])
        os.replace(tmp, out)
        return out
    except (ImportError, OSError, RuntimeError, AttributeError) as e:
        print(f"the compiled marshalling was not built (calls are marshalled in Python): {e}", file=sys.stderr)
        return None


def build(force: bool = False, verbose: bool = False, extra_flags=(), debug: bool = False) -> str:
    """Compile and link libverifyhead.so (debug: libverifyhead_debug.so with
    -DVH_DEBUG, whose kernels guard their indices and report failures in the
    workspace error word); returns its path."""
    lib = LIB_DEBUG if debug else LIB
    if not force and up_to_date(lib):
        if not debug:
            build_marshal()
        return lib
    obj_dir = os.path.join(BUILD_DIR, "debug") if debug else BUILD_DIR
    os.makedirs(obj_dir, exist_ok=True)
    nv = nvcc()
    flags = list(extra_flags) + (["-DVH_DEBUG"] if debug else [])

    def compile_one(src):
        obj = os.path.join(obj_dir, os.path.basename(src) + ".o")
        cmd = [nv, *ARCH, *NVCC_FLAGS, *flags, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        marshal = None if debug else ex.submit(build_marshal, force)
        results = list(ex.map(compile_one, sources()))
        if marshal is not None:
            marshal.result()
    if verbose:
        for _, log in results:
            if log.strip():
                print(log)
    objs = [o for o, _ in results]
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nv, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
           "-Xlinker", "-rpath=/usr/local/cuda/lib64"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))
