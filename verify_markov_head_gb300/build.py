"""Build the CUDA library libdspark.so in-tree (nvcc, sm_103a only).

Each translation unit under csrc/ is compiled separately (in parallel) and
linked into verify_markov_head_gb300/_lib/libdspark.so with the CUDA runtime
linked statically, so the library needs nothing from the Python environment.
Beside it, where PyTorch is installed, the Python module of the serving
operators (csrc/serve_py.cpp) is built with its headers; its version is in the
module's name.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT, "libdspark.so")
ROOT = os.path.dirname(HERE)
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(SRC, f) for f in os.listdir(SRC) if f.endswith(".cu"))


def _stale(lib):
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(SRC, f) for f in os.listdir(SRC)] + [os.path.join(ROOT, "include", "dspark.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def torch_dir():
    """PyTorch's folder, None where there is none."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def serve_lacks():
    """What the Python module's build needs and does not find, None where all is there."""
    torch = torch_dir()
    if torch is None:
        return "PyTorch"
    if not os.path.exists(os.path.join(torch, "include", "c10", "cuda", "CUDAStream.h")):
        return "PyTorch's CUDA headers"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    return None if shutil.which("g++") else "g++"


def serve_module() -> str:
    """Where the Python module of this PyTorch is built."""
    version: dict = {}
    with open(os.path.join(torch_dir(), "version.py")) as f:      # (without importing torch)
        for line in f:
            if line.startswith("__version__"):
                exec(line, version)
    return os.path.join(OUT, f"_serve-{version['__version__']}.so")


def _compile_serve(cc):
    """Object file of the Python module, and what its link needs."""
    torch = torch_dir()
    obj = os.path.join(OUT, "serve_py.o")
    dirs = [os.path.join(ROOT, "include"), os.path.join(torch, "include"),
            os.path.join(torch, "include", "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
            os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", *(f"-I{d}" for d in dirs), "-c", os.path.join(SRC, "serve_py.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on serve_py.cpp:\n{r.stderr}")
    return obj, os.path.join(torch, "lib")


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    lacks = serve_lacks()
    if not force and not _stale(LIB) and (lacks or not _stale(serve_module())):
        return LIB
    os.makedirs(OUT, exist_ok=True)
    cc = nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT, os.path.basename(src).replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        serve = None if lacks else ex.submit(_compile_serve, cc)
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if serve is None:
        if verbose:
            print(f"the serving operators' Python module is not built: no {lacks}", file=sys.stderr)
        return LIB
    serve_obj, torch_lib = serve.result()            # (the library stands whatever came of the module)
    module = serve_module()
    tmp = module + f".tmp{os.getpid()}"
    r = subprocess.run(["g++", "-shared", "-o", tmp, serve_obj, "-L", torch_lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
                        "-lc10", "-L", OUT, "-l:libdspark.so", "-Wl,-rpath,$ORIGIN"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, module)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
