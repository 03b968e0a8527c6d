"""In-tree build of libmoe_w4.so (sm_103a only) with nvcc.

Each .cu under csrc/ is compiled to an object in parallel, then linked into
bit_quantized_expert_moe_gb300/libmoe_w4.so.  The Python binding of the 16-bit
expert operators (csrc/expert16_binding.cpp) is compiled beside them with g++
and linked against that library and torch; where torch or Python's headers are not
installed the library is built without it.  Run as a module or call build().
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_w4.so")
BINDING_SRC = os.path.join(CSRC, "expert16_binding.cpp")
BINDING = os.path.join(PKG, "_expert16.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps() -> list[str]:
    out = sources() + [BINDING_SRC, os.path.abspath(__file__)]
    out += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    out += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return out


def binding_lacks() -> str | None:
    """What the binding needs and this machine does not have."""
    if importlib.util.find_spec("torch") is None:
        return "torch"
    if not os.path.exists(os.path.join(sysconfig.get_path("include"), "Python.h")):
        return "Python's headers"
    return None


def _torch_version() -> str:
    """Where torch lies, its version and the CUDA and commit it was built from, without importing it."""
    where = os.path.dirname(importlib.util.find_spec("torch").origin)
    with open(os.path.join(where, "version.py")) as f:
        return where + "\n" + f.read()


def _built_against() -> str:
    """The torch and the interpreter whose C++ and C interfaces the binding is compiled for."""
    return f"{sysconfig.get_config_var('SOABI')}\n{_torch_version()}"


def _binding_current() -> bool:
    try:
        with open(os.path.join(BUILD, "expert16.against")) as f:
            return f.read() == _built_against()
    except OSError:
        return False


def up_to_date() -> bool:
    lacks = binding_lacks()
    made = [LIB] if lacks else [LIB, BINDING]
    if not all(os.path.exists(p) for p in made) or not (lacks or _binding_current()):
        return False
    t = min(os.path.getmtime(p) for p in made)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _binding_object() -> str:
    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    obj = os.path.join(BUILD, "expert16_binding.o")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}",
           "-isystem", inc, "-isystem", os.path.join(inc, "torch/csrc/api/include"),
           "-isystem", sysconfig.get_path("include"), "-isystem", cuda, "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    # by name and not by path: it asks for the library beside itself ($ORIGIN), wherever
    # the tree lies by then
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, f"-L{os.path.dirname(LIB)}",
           f"-l:{os.path.basename(LIB)}", f"-L{lib}", "-ltorch_python", "-ltorch_cpu",
           "-ltorch", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(os.path.join(BUILD, "expert16.against"), "w") as f:
        f.write(_built_against())


def build(verbose: bool = False, force: bool = False, extra: list[str] | None = None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    extra = extra or []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    lacks = binding_lacks()
    with ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 1)) as ex:
        binding = None if lacks else ex.submit(_binding_object)
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    # the C library is there by now, whatever becomes of the binding
    if lacks:
        print(f"{LIB} is built; without {lacks} the Python binding of the 16-bit expert operators is not", file=sys.stderr)
    else:
        _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
