"""Build the CUDA library (libpagedkv.so) in-tree with nvcc for sm_103a, and the
Python binding's native part (binding/calls.cpp) with g++ against this torch.

Each translation unit is compiled in parallel with
``-gencode arch=compute_103a,code=sm_103a -O3 -lineinfo`` and the objects are
linked into ``paged_kv_decode_16_gb300/_build/libpagedkv.so`` (static CUDA
runtime, so loading it needs no GPU).  Rebuilds only when a source or header
is newer than the library.  The library needs neither torch nor Python's headers
(build_library; ``python build.py`` without a torch); the binding is built after it
and for itself.  Concurrent builds (two test processes, a test and
the benchmark) take an exclusive file lock on ``_build/.lock`` and compile
into an object directory of their own, so they never share a half-written
object; the second one to get the lock finds the library up to date.
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import fcntl
import glob
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libpagedkv.so")
BINDING = os.path.join(HERE, "binding", "calls.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("CUDA_HOME", ""), "/usr/local/cuda"):
        p = os.path.join(cand, "bin", "nvcc") if cand else ""
        if p and os.path.exists(p):
            return p
    p = shutil.which("nvcc")
    if not p:
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedkv.so")
    return p


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _inputs() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.hpp")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def binding_path() -> str:
    """The native module of the Python binding; its name holds the torch and Python
    versions that it was built against."""
    import torch
    tag = re.sub(r"[^0-9A-Za-z]+", "_", f"{torch.__version__}_py{sysconfig.get_python_version()}")
    return os.path.join(OUT_DIR, f"_pagedkv_calls_{tag}.so")


def _newest(paths) -> float:
    return max(os.path.getmtime(f) for f in paths)


def library_up_to_date() -> bool:
    return os.path.exists(LIB) and _newest(_inputs()) <= os.path.getmtime(LIB)


def binding_up_to_date() -> bool:
    calls = binding_path()
    header = os.path.join(INCLUDE, "pagedkv.h")
    return os.path.exists(calls) and _newest((BINDING, header, __file__)) <= os.path.getmtime(calls)


def _compile_binding(out: str) -> subprocess.CompletedProcess:
    """g++ of binding/calls.cpp into an object (a C++ file against torch's headers)."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    cmd = ["g++", "-c", BINDING, "-o", out, "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE,
           "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"),
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    return subprocess.run(cmd, capture_output=True, text=True)


def _link_binding(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    out = binding_path()
    tmp = f"{out}.tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", OUT_DIR, "-lpagedkv", "-L", libs,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr)
    os.replace(tmp, out)


@contextlib.contextmanager
def _build_lock():
    os.makedirs(OUT_DIR, exist_ok=True)
    with open(os.path.join(OUT_DIR, ".lock"), "w") as f:
        fcntl.flock(f, fcntl.LOCK_EX)
        try:
            yield
        finally:
            fcntl.flock(f, fcntl.LOCK_UN)


def build_library(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile every source for sm_103a and link libpagedkv.so; return its path.  Needs
    nvcc and a host compiler, nothing else."""
    if not force and library_up_to_date():
        return LIB
    with _build_lock():
        if force or not library_up_to_date():  # (built by another process meanwhile)
            _build_library_locked(verbose, ptxas_verbose)
        return LIB


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """The library and the Python binding's native part; return the library's path.  Where
    the binding does not compile, the library is there all the same when this raises."""
    if not force and library_up_to_date() and binding_up_to_date():
        return LIB
    with _build_lock():
        library = force or not library_up_to_date()
        binding = force or not binding_up_to_date()
        with tempfile.TemporaryDirectory() as tmp, cf.ThreadPoolExecutor(max_workers=1) as ex:
            obj = os.path.join(tmp, "calls.o")
            calls = ex.submit(_compile_binding, obj) if binding else None
            if library:
                _build_library_locked(verbose, ptxas_verbose)
            if calls:
                r = calls.result()
                if r.returncode != 0:
                    raise RuntimeError("the Python binding's native part does not compile:\n"
                                       + r.stderr)
                _link_binding(obj)
    return LIB


def _build_library_locked(verbose: bool, ptxas_verbose: bool) -> None:
    nvcc = _nvcc()
    obj_dir = os.path.join(OUT_DIR, f"obj{os.getpid()}")
    os.makedirs(obj_dir, exist_ok=True)
    common = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
              *ARCH]
    if ptxas_verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src: str):
        obj = os.path.join(obj_dir, os.path.basename(src) + ".o")
        cmd = [nvcc, "-c", src, "-o", obj, *common]
        if src.endswith(".cpp"):
            cmd = [nvcc, "-x", "cu", "-c", src, "-o", obj, *common]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    objs = []
    errors = []
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        for src, obj, r in ex.map(compile_one, sources()):
            if verbose or ptxas_verbose:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                errors.append(f"{os.path.basename(src)}:\n{r.stderr}")
            objs.append(obj)
    if errors:
        raise RuntimeError("nvcc failed:\n" + "\n".join(errors))
    # the temporary name keeps the .so suffix: nvcc picks the link step from it
    tmp = os.path.join(OUT_DIR, f"libpagedkv.tmp{os.getpid()}.so")
    cmd = [nvcc, "-shared", *ARCH, "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr)
    os.replace(tmp, LIB)
    shutil.rmtree(obj_dir, ignore_errors=True)


def main(argv) -> None:
    """The library, and the binding where there is a torch to build it against."""
    options = dict(force="--force" in argv, verbose=True, ptxas_verbose="-v" in argv)
    try:
        import torch  # noqa: F401
    except ImportError:
        print(build_library(**options))
        sys.stderr.write("no torch: the Python binding's native part is not built\n")
        return
    print(build(**options))


if __name__ == "__main__":
    main(sys.argv[1:])
