"""Compile the CUDA library libattn.so (sm_103a) in-tree.

Each translation unit is compiled by its own nvcc process (in parallel), then
linked into ``causal_streaming_softmax_gb300/libattn.so``.  Objects go to
``causal_streaming_softmax_gb300/_build/``.  A rebuild happens only when a
source or header is newer than the library.

``_marshal.so`` beside it is a small Python extension (host code) that hands
PyTorch tensors to the library's serving calls; it is compiled by g++ against
the installed PyTorch's headers in the same way.  It reads PyTorch's objects
through those headers, so it belongs to one build of PyTorch and Python: it
carries that build's key, and is made again, or left alone, where another is
installed.  The library does not need it.
"""
import concurrent.futures
import glob
import importlib.util
import os
import runpy
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libattn.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
MARSHAL_KEY = os.path.join(BUILD, "marshal.key")  # what MARSHAL was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
              "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libattn.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "attn.h"), __file__]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def marshal_key(version=None, cuda=None, git_version=None) -> str:
    """What _marshal.so is built for: the installed (or the given) PyTorch's
    version, CUDA version and revision, and this Python's ABI."""
    if version is None:
        v = runpy.run_path(os.path.join(_torch(), "version.py"))
        version, cuda, git_version = v["__version__"], v.get("cuda"), v.get("git_version")
    return "torch %s cuda %s %s %s" % (version, cuda, git_version,
                                       sysconfig.get_config_var("SOABI"))


def marshal_up_to_date() -> bool:
    if not os.path.exists(MARSHAL) or not os.path.exists(MARSHAL_KEY):
        return False
    with open(MARSHAL_KEY) as f:
        if f.read() != marshal_key():
            return False
    t = os.path.getmtime(MARSHAL)
    return all(os.path.getmtime(p) <= t for p in (MARSHAL_SRC, os.path.join(INCLUDE, "attn.h"),
                                                  __file__))


def _torch() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("PyTorch not found: its headers are required to build _marshal.so")
    return spec.submodule_search_locations[0]


def marshal_missing():
    """What keeps _marshal.so from being built here (None: nothing)."""
    if importlib.util.find_spec("torch") is None:
        return "PyTorch"
    if not os.path.exists(os.path.join(_torch(), "lib", "libc10_cuda.so")):
        return "a PyTorch with CUDA"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    return None


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    """Compile the Python extension that marshals the serving calls."""
    if not force and marshal_up_to_date():
        return MARSHAL
    torch, cuda, key = _torch(), os.path.dirname(os.path.dirname(_nvcc())), marshal_key()
    inc = [os.path.join(torch, "include"),
           os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    lib = os.path.join(torch, "lib")
    tmp = MARSHAL + ".tmp.%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           '-DCSS_BUILT_FOR="%s"' % key] + \
        [x for p in inc for x in ("-isystem", p)] + [MARSHAL_SRC, "-o", tmp, "-L" + lib,
         "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on %s:\n%s%s" % (MARSHAL_SRC, r.stdout, r.stderr))
    os.makedirs(BUILD, exist_ok=True)
    if os.path.exists(MARSHAL_KEY):
        os.remove(MARSHAL_KEY)  # never a key beside another build's library
    os.replace(tmp, MARSHAL)
    with open(MARSHAL_KEY, "w") as f:
        f.write(key)
    return MARSHAL


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    missing = marshal_missing()
    if missing and verbose:
        print("_marshal.so is left out: it needs %s" % missing, file=sys.stderr)
    if not force and up_to_date() and (missing or marshal_up_to_date()):
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + ARCH + NVCC_FLAGS + list(extra_flags) + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose and r.stderr.strip():
            print(r.stderr, file=sys.stderr)
        return obj

    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        marshal = None if missing else ex.submit(build_marshal, force, verbose)
        objs = [] if not force and up_to_date() else list(ex.map(compile_one, srcs))
    if objs:
        _link(nvcc, objs, verbose)
    if marshal is not None:
        marshal.result()  # raises what stopped it, the library being there
    return LIB


def _link(nvcc: str, objs, verbose: bool) -> None:
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)


if __name__ == "__main__":
    flags = [a for a in sys.argv[1:] if a.startswith("-X") or a.startswith("--")]
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=[f for f in flags if f != "--force"]))
