"""Build libslope.so (the C-ABI CUDA library) in-tree with nvcc for sm_100a,
and its debug build libslope_debug.so (-DSLOPE_DEBUG_BOUNDS: bounds checks on
every plain global-memory access of the kernels, for tests), and with g++
the Python module _calls.so (csrc/calls.cpp)."""
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "slope_api.cu")
LIB = os.path.join(HERE, "libslope.so")
LIB_DEBUG = os.path.join(HERE, "libslope_debug.so")
CALLS = os.path.join(HERE, "_calls.so")


def deps():
    """What the library is built from."""
    csrc = os.path.join(HERE, "csrc")
    return [os.path.join(csrc, f) for f in os.listdir(csrc)] + [os.path.join(ROOT, "include", "slope.h")]


NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-shared", "-Xptxas", "-v"]


def nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _build_one(lib: str, extra, force: bool, verbose: bool) -> str:
    if not force and os.path.exists(lib):
        newest = max(os.path.getmtime(d) for d in deps())
        if os.path.getmtime(lib) >= newest:
            return lib
    cmd = [nvcc()] + NVCC_FLAGS + list(extra) + ["-o", lib, SRC]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"nvcc failed building {os.path.basename(lib)}")
    if verbose:
        sys.stderr.write(res.stderr)
    return lib


def calls_key() -> str:
    """What a built _calls.so belongs to: this Python and this torch."""
    import torch
    return f"{sysconfig.get_config_var('SOABI')} {sys.hexversion:#x} torch {torch.__version__} {int(torch._C._GLIBCXX_USE_CXX11_ABI)}"


def calls_current() -> bool:
    """Whether _calls.so is there and was built for this Python and this torch."""
    try:
        with open(CALLS, "rb") as f:  # calls.cpp keeps its key as a string
            return b"slope calls for " + calls_key().encode() + b"\0" in f.read()
    except OSError:
        return False


def build_calls(force: bool = False) -> str:
    """Build _calls.so: Python's and torch's headers, no device code."""
    src, lib = os.path.join(HERE, "csrc", "calls.cpp"), CALLS
    deps = [src, os.path.join(ROOT, "include", "slope.h")]
    if not force and calls_current() and os.path.getmtime(lib) >= max(map(os.path.getmtime, deps)):
        return lib
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    include = [sysconfig.get_paths()["include"], os.path.join(home, "include"),
               os.path.join(home, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f'-DSLOPE_CALLS_KEY="{calls_key()}"', f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
           + [f"-isystem{d}" for d in include] + ["-o", lib, src, "-L" + os.path.join(home, "lib"),
                                                  "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"])
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"g++ not started ({e})") from e
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("g++ failed building _calls.so")
    return lib


def build(force: bool = False, verbose: bool = False, debug: bool = True) -> str:
    """Build libslope.so and _calls.so (and, with debug=True, libslope_debug.so
    beside them, in parallel); returns the release library's path.  Without
    torch's C++ headers or g++ the library is built all the same."""
    from concurrent.futures import ThreadPoolExecutor
    with ThreadPoolExecutor(3) as ex:
        calls = ex.submit(build_calls, force)
        rel = ex.submit(_build_one, LIB, [], force, verbose)
        if debug:
            ex.submit(_build_one, LIB_DEBUG, ["-DSLOPE_DEBUG_BOUNDS"], force, False).result()
        try:
            calls.result()
        except (RuntimeError, ImportError) as e:  # the library itself needs nvcc alone
            sys.stderr.write(f"_calls.so not built ({e}); the int8 path's calls go through ctypes without it\n")
        return rel.result()


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
