"""Build libpkv.so in-tree with nvcc for sm_103a (GB300).

Each .cu translation unit compiles in parallel to an object file, then nvcc
links them into ``paged_kv_attention_21_gb300/_build/libpkv.so`` with the
CUDA runtime linked statically (the tensor-map encoder is fetched from the
driver at run time, so libcuda is not linked).  Beside them g++ compiles the
binding's argument checks (``csrc/marshal.cpp``, against torch's headers) into
``_build/_marshal.so``.  The library needs nvcc alone: without torch it is built
by itself, and where the binding's module does not compile it is linked all the
same before that is reported.
"""
from __future__ import annotations

import concurrent.futures
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libpkv.so")
MARSHAL_PATH = os.path.join(OUT_DIR, "_marshal.so")
STAMP_PATH = os.path.join(OUT_DIR, "_marshal.for")  # what _marshal.so was built against
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler",
              "-fPIC,-ffp-contract=off", "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libpkv")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps(binding: bool):
    names = [f for f in os.listdir(CSRC) if f.endswith(".cpp") == binding]
    return [os.path.join(CSRC, f) for f in names] + [os.path.join(INCLUDE, "pkv.h"), __file__]


def _torch_dir():
    """Where torch is installed, or None."""
    spec = importlib.util.find_spec("torch")
    return None if spec is None else list(spec.submodule_search_locations)[0]


def _binding_for():
    """The torch and Python whose ABI the binding's module is bound to; None without torch."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "unknown"
    return "torch %s at %s, python %s\n" % (version, torch_dir, sys.version.split()[0])


def _compile_marshal():
    """The binding's extension module, where there is torch; raises with the compiler's output."""
    torch_dir, stamp = _torch_dir(), _binding_for()
    if torch_dir is None:
        return
    lib = os.path.join(torch_dir, "lib")
    tmp = MARSHAL_PATH + ".tmp.%d" % os.getpid()
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE,
           "-I", os.path.join(torch_dir, "include"),
           "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include"),
           os.path.join(CSRC, "marshal.cpp"), "-o", tmp,
           "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on marshal.cpp:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, MARSHAL_PATH)
    with open(STAMP_PATH, "w") as f:
        f.write(stamp)


def _newer(path, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps)


def library_up_to_date() -> bool:
    return _newer(LIB_PATH, _deps(False))


def binding_up_to_date() -> bool:
    """Built from the current source, for the installed torch and this Python (or no torch)."""
    stamp = _binding_for()
    if stamp is None:
        return True
    if not _newer(MARSHAL_PATH, _deps(True)) or not os.path.exists(STAMP_PATH):
        return False
    with open(STAMP_PATH) as f:
        return f.read() == stamp


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every kernel TU and link libpkv.so, and the binding's module beside it;
    returns the library's path."""
    os.makedirs(OUT_DIR, exist_ok=True)
    if not force and library_up_to_date():
        if not binding_up_to_date():
            _compile_marshal()
        return LIB_PATH
    nvcc = _nvcc()
    srcs = sources()

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH_FLAGS, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        marshal = ex.submit(_compile_marshal)
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB_PATH + ".tmp.%d" % os.getpid()
    cmd = [nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB_PATH)
    marshal.result()  # the library stands, whatever became of the binding's module
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
