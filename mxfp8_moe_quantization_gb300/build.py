"""Build libfp8moe.so in-tree with nvcc for sm_103a (GB300), and the module
that marshals PyTorch tensors for the small calls with the host compiler.

Each translation unit compiles in parallel; the CUDA objects link into
``mxfp8_moe_quantization_gb300/libfp8moe.so``, the binding into ``_binding.so``
beside it.  A rebuild happens only when a source or header is newer than the
libraries, or when the binding was made for another PyTorch or Python (it is
compiled against their internals).  No cmake, one -gencode.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfp8moe.so")
BINDING = os.path.join(HERE, "_binding.so")
STAMP = os.path.join(BUILD, "binding.for")   # what BINDING was compiled against

SOURCES = ["api.cu", "quant.cu", "colwise.cu", "colwise_cluster.cu", "colwise_jagged.cu", "dual.cu", "tensorwise.cu", "blockwise.cu", "routing.cu", "swizzle.cu",
           "grouped_mm.cu", "blockwise_mm.cu", "layer.cu", "norm.cu", "router.cu", "swiglu.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills", "-I", INCLUDE]


def _nvcc() -> str:
    for cand in [os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"]:
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    out = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    out.append(os.path.join(INCLUDE, "fp8moe.h"))
    out.append(os.path.abspath(__file__))
    return out


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def _made_for() -> str:
    import torch
    return "\n".join([torch.__version__, os.path.realpath(_torch_dir()), sys.version, os.uname().machine])


def _stamped() -> str:
    try:
        with open(STAMP) as f:
            return f.read()
    except OSError:
        return ""


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING) or _stamped() != _made_for():
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(p) <= t for p in _deps())


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile every .cu for sm_103a and link libfp8moe.so; return its path."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    torch_dir = _torch_dir()
    binding_obj = os.path.join(BUILD, "binding.o")

    def run(what, cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")

    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))

    def compile_binding():
        run("binding", [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-I", os.path.join(torch_dir, "include"),
                        "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include"),
                        "-I", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "binding.cpp"), "-o", binding_obj])

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, SOURCES))
        binding.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = BINDING + ".tmp"
    torch_lib = os.path.join(torch_dir, "lib")
    run("binding link", [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, binding_obj, "-L", HERE, "-l:libfp8moe.so",
                         "-L", torch_lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
                         "-L", os.path.join(cuda, "lib64"), "-lcudart", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_lib}"])
    os.replace(tmp, BINDING)
    with open(STAMP + ".tmp", "w") as f:
        f.write(_made_for())
    os.replace(STAMP + ".tmp", STAMP)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
