"""In-tree build of libmoe_gb300.so (nvcc, sm_103a only) and of the extension module that calls it on torch tensors."""
from __future__ import annotations

import glob
import importlib.util
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


def _torch_id() -> str:
    """The torch that the extension module has to be built against: where it is and its version; "" without one."""
    try:
        spec = importlib.util.find_spec("torch")
    except ValueError:  # (sys.modules["torch"] is None or half imported)
        spec = None
    if spec is None or not spec.origin:
        return ""
    root = os.path.dirname(os.path.abspath(spec.origin))
    with open(os.path.join(root, "version.py")) as f:
        return "%s %s %s" % (sys.version.split()[0], root, f.read())


def _stamp() -> str:
    return TORCH_OPS + ".torch"


def _older(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(p) > t for p in deps)


def _lib_stale() -> bool:
    return _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _torch_ops_stale(torch_id: str) -> bool:
    if _older(TORCH_OPS, glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(INCLUDE, "*.h"))) or not os.path.exists(_stamp()):
        return True
    with open(_stamp()) as f:
        return f.read() != torch_id


def build(force: bool = False, verbose: bool = False, torch_ops: bool = True) -> str:
    """Compile every translation unit in parallel and link the shared library and, with torch_ops and where there is a torch, the
    extension module.  The library needs neither torch nor the module."""
    torch_id = _torch_id() if torch_ops else ""
    lib = force or _lib_stale()
    ops = torch_id != "" and (force or _torch_ops_stale(torch_id))
    if not lib and not ops:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    procs = []
    objs = []
    for src in sources() if lib else []:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [nvcc, *NVCC_FLAGS, "-c", src, "-o", obj]
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    torch_src = os.path.join(CSRC, "torch_ops.cpp")
    torch_tmp = TORCH_OPS + ".tmp.%d" % os.getpid()
    if ops:
        torch_compile, torch_link = _torch_ops_commands(os.path.join(BUILD, "torch_ops.o"), torch_tmp)
        procs.append((torch_src, subprocess.Popen(torch_compile, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out))
        elif verbose and out.strip():
            sys.stderr.write(out)

    def check(failures):
        if failures:
            raise RuntimeError("compilation failed:\n" + "\n".join("%s:\n%s" % f for f in failures))
    check([f for f in failed if f[0] != torch_src])
    if lib:
        tmp = LIB + ".tmp.%d" % os.getpid()
        subprocess.run([nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-Xlinker", "-soname," + os.path.basename(LIB),
                        *objs, "-o", tmp], check=True)
        os.replace(tmp, LIB)
    check(failed)
    if ops:
        subprocess.run(torch_link, check=True)
        os.replace(torch_tmp, TORCH_OPS)
        with open(_stamp(), "w") as f:
            f.write(torch_id)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
