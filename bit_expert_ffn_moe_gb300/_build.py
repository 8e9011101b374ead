"""In-tree build of libmoe_gb300.so (nvcc, sm_103a only) and of the extension module that calls it on torch tensors."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libmoe_gb300.so")
TORCH_OPS = os.path.join(BUILD, "moe_torch_ops.so")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")

NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "-lineinfo",
              "-Xcompiler", "-fPIC", "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _torch_ops_commands(obj: str, out: str):
    """Compile and link commands of csrc/torch_ops.cpp against the torch that runs this."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    compile_ = ["g++", "-std=c++20", "-O2", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
                *["-isystem" + i for i in inc], "-c", os.path.join(CSRC, "torch_ops.cpp"), "-o", obj]
    libs = os.path.join(root, "lib")
    link = ["g++", "-shared", obj, "-o", out, "-L" + libs, "-Wl,-rpath," + libs, "-Wl,-rpath,$ORIGIN", "-ltorch_python", "-ltorch",
            "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-L" + BUILD, "-l:" + os.path.basename(LIB)]
    return compile_, link


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(TORCH_OPS):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(TORCH_OPS))
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every translation unit in parallel and link the shared library."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    procs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [nvcc, *NVCC_FLAGS, "-c", src, "-o", obj]
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    torch_obj = os.path.join(BUILD, "torch_ops.o")
    torch_tmp = TORCH_OPS + ".tmp.%d" % os.getpid()
    torch_compile, torch_link = _torch_ops_commands(torch_obj, torch_tmp)
    procs.append((torch_compile[-3], subprocess.Popen(torch_compile, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out))
        elif verbose and out.strip():
            sys.stderr.write(out)
    if failed:
        msg = "\n".join("%s:\n%s" % (s, o) for s, o in failed)
        raise RuntimeError("compilation failed:\n" + msg)
    tmp = LIB + ".tmp.%d" % os.getpid()
    subprocess.run([nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-Xlinker", "-soname," + os.path.basename(LIB), *objs,
                    "-o", tmp], check=True)
    os.replace(tmp, LIB)
    subprocess.run(torch_link, check=True)
    os.replace(torch_tmp, TORCH_OPS)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
