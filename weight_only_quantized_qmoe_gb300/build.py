"""Build libqmoe.so (the C-ABI library) in-tree with nvcc for sm_103a, and
_ops_torch.so (the operators on torch tensors, a CPython module that calls the
library) with g++ against torch's headers.  The library needs no torch; without
one the module is left out.

Every translation unit is compiled in parallel; the objects go to
``<repo>/_build`` and the libraries next to this file.  No cmake.
"""
from __future__ import annotations

import concurrent.futures
import os
import platform
import re
import shutil
import subprocess
import sys
import sysconfig
from importlib.util import find_spec

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(HERE, "libqmoe.so")
SOURCES = ["qmoe_api.cu", "qmoe_route.cu", "qmoe_decode.cu", "qmoe_prefill.cu", "qmoe_decode_b2.cu",
           "qmoe_decode_b3.cu", "qmoe_decode_b4.cu", "qmoe_decode_b8.cu",
           "qmoe_decode_b1.cu", "qmoe_fused.cu", "qmoe_fused_w22.cu", "qmoe_fused_w23.cu",
           "qmoe_fused_w24.cu", "qmoe_fused_w32.cu", "qmoe_fused_w33.cu", "qmoe_fused_w34.cu",
           "qmoe_fused_w42.cu", "qmoe_fused_w43.cu", "qmoe_fused_w44.cu",
           "qmoe_ops_api.cu", "qmoe_sort.cu", "qmoe_mx4.cu", "qmoe_mx4_gemm.cu", "qmoe_norm.cu", "qmoe_norm_grad.cu"]
TORCH_MODULE = os.path.join(HERE, "_ops_torch.so")
TORCH_SOURCE = "qmoe_ops_torch.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc_path() -> str:
    for cand in (os.environ.get("CUDA_HOME"), "/usr/local/cuda"):
        if cand and os.path.exists(os.path.join(cand, "bin", "nvcc")):
            return os.path.join(cand, "bin", "nvcc")
    found = shutil.which("nvcc")
    if not found:
        raise RuntimeError("nvcc not found: set CUDA_HOME")
    return found


def _newer(target: str, suffixes) -> bool:
    """The target is there and no older than the sources of these kinds."""
    if not os.path.exists(target):
        return False
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(suffixes)]
    files += [os.path.join(INCLUDE, "qmoe.h"), os.path.abspath(__file__)]
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in files)


def library_up_to_date() -> bool:
    return _newer(LIB_PATH, (".cu", ".cuh", ".h"))


def torch_version() -> str:
    """The torch and the Python that the module belongs to (without importing torch)."""
    with open(os.path.join(list(find_spec("torch").submodule_search_locations)[0], "version.py")) as f:
        found = re.search(r"^__version__\s*=\s*['\"]([^'\"]+)", f.read(), re.M)
    return f"{found.group(1) if found else '?'} {sys.version.split()[0]} {platform.machine()}"


def _built_for() -> str:
    """What torch_version() was when the module was built."""
    try:
        with open(TORCH_MODULE + ".torch") as f:
            return f.read()
    except OSError:
        return ""


def module_up_to_date() -> bool:
    """The module on torch tensors is current, or there is no torch to build it against."""
    return find_spec("torch") is None or (_newer(TORCH_MODULE, (".cpp",)) and _built_for() == torch_version())


def up_to_date() -> bool:
    return library_up_to_date() and module_up_to_date()


def torch_module_commands(nvcc: str, obj: str):
    """The compile and the link command of the module on torch tensors."""
    spec = find_spec("torch")
    if spec is None:
        raise RuntimeError("torch not found: its headers are needed for " + TORCH_SOURCE)
    torch_dir = list(spec.submodule_search_locations)[0]
    cuda = os.path.dirname(os.path.dirname(nvcc))
    inc = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    compile_cmd = ["g++", "-O2", "-std=c++20", "-fPIC", "-Wall", *[f"-I{d}" for d in inc], "-c",
                   os.path.join(CSRC, TORCH_SOURCE), "-o", obj]
    link_cmd = ["g++", "-shared", obj, "-o", TORCH_MODULE + ".tmp", "-L" + os.path.join(torch_dir, "lib"), "-lc10",
                "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-L" + HERE, "-l:libqmoe.so",
                "-Wl,-rpath,$ORIGIN"]
    return compile_cmd, link_cmd


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is not current; the module on torch tensors only where there is a torch."""
    with_library = force or not library_up_to_date()
    with_module = find_spec("torch") is not None and (force or not module_up_to_date())
    if not with_library and not with_module:
        return LIB_PATH
    nvcc = nvcc_path()
    objdir = os.path.join(ROOT, "_build")
    os.makedirs(objdir, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        torch_obj = None
        if with_module:
            compile_torch, link_torch = torch_module_commands(nvcc, os.path.join(objdir, TORCH_SOURCE.replace(".cpp", ".o")))
            torch_obj = ex.submit(_run, compile_torch, "g++ for " + TORCH_SOURCE)
        if with_library:
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB_PATH + ".tmp"
            _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcuda"], "link of " + os.path.basename(LIB_PATH))
            os.replace(tmp, LIB_PATH)
        if with_module:
            torch_obj.result()
            _run(link_torch, "link of " + os.path.basename(TORCH_MODULE))
            os.replace(TORCH_MODULE + ".tmp", TORCH_MODULE)
            with open(TORCH_MODULE + ".torch", "w") as f:
                f.write(torch_version())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
