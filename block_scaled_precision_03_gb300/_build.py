"""Build libbsq.so in-tree with nvcc for sm_103a, and the native Python
binding _binding.so with the host compiler.

Each .cu file is compiled in parallel into _build/, then linked into
block_scaled_precision_03_gb300/libbsq.so (CUDA runtime linked statically,
driver entry points resolved at run time).  binding.cpp is compiled against the
installed PyTorch beside them, and again when that is another one; the library
does not wait for it, and stands where it cannot be built.  Usage:

    python -m block_scaled_precision_03_gb300._build [--force] [-v]
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libbsq.so")
BINDING = os.path.join(HERE, "_binding.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
SOURCES = ["api.cu", "quantize.cu", "convert.cu", "gemm.cu", "gemm2.cu", "api_ops.cu", "moe.cu",
           "norm.cu", "head.cu", "linear.cu", "gemv.cu", "clip.cu", "adamw.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    return "nvcc"


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "bsq.h"))
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def _made_for() -> str:
    """What the binding is compiled against besides the sources: this Python and
    the installed PyTorch, whose version file is read without importing it."""
    import importlib.util
    torch = importlib.util.find_spec("torch")
    version = "none"
    if torch is not None and torch.origin:
        with open(os.path.join(os.path.dirname(torch.origin), "version.py")) as f:
            version = f.read()
    return f"{sys.version}\n{version}"


def _lib_current() -> bool:
    return os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps()


def _binding_current() -> bool:
    if not os.path.exists(BINDING) or os.path.getmtime(BINDING) < _deps():
        return False
    try:
        with open(os.path.join(BUILD, "binding.for")) as f:
            return f.read() == _made_for()
    except FileNotFoundError:
        return False


def _compile_binding():
    import sysconfig
    try:
        import torch
    except ImportError as e:
        raise RuntimeError(f"the Python binding needs PyTorch: {e}") from e
    root = os.path.dirname(torch.__file__)
    tmp = BINDING + f".{os.getpid()}.tmp"
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", abi,
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{os.path.join(root, 'lib')}"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"g++ could not be run for binding.cpp: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(os.path.join(BUILD, "binding.for"), "w") as f:
        f.write(_made_for())


def build(force: bool = False, verbose: bool = False) -> str:
    """Build what is out of date; returns the library's path.  Where the binding
    cannot be built the library is built all the same, before the error."""
    os.makedirs(BUILD, exist_ok=True)
    lib, binding = force or not _lib_current(), force or not _binding_current()
    with ThreadPoolExecutor(1) as ex:
        beside = ex.submit(_compile_binding) if binding else None
        if lib:
            _build_lib(verbose)
        if beside:
            beside.result()
    return LIB


def _build_lib(verbose: bool) -> None:
    flags = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE] + ARCH
    if verbose:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc(), *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".{os.getpid()}.tmp"
    r = subprocess.run([nvcc(), "-shared", *ARCH, "-o", tmp, *objs, "-cudart", "static"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
