"""In-tree build for sm_103a: libspecverify.so (nvcc, translation units compiled in
parallel) and the Python binding of the verify step's operators (g++).

The library links the CUDA runtime statically (nvcc's default), so it does not
depend on which libcudart the Python process has loaded; device pointers and
streams are shared through the driver's primary context. The binding
(csrc/binding.cpp) is compiled against the headers of the installed torch and
linked to the library beside it.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRCS = [os.path.join(PKG, "csrc", n) for n in ("spec_verify.cu", "verify_step.cu", "paged_step.cu")]
BINDING_SRC = os.path.join(PKG, "csrc", "binding.cpp")
OUT_DIR = os.path.join(PKG, "_lib")
OUT = os.path.join(OUT_DIR, "libspecverify.so")
BINDING_OUT = os.path.join(OUT_DIR, "_binding.so")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc_path():
    for cand in (os.environ.get("CUDA_HOME"), os.environ.get("CUDA_PATH"), "/usr/local/cuda"):
        if cand and os.path.exists(os.path.join(cand, "bin", "nvcc")):
            return os.path.join(cand, "bin", "nvcc")
    found = shutil.which("nvcc")
    if found:
        return found
    raise RuntimeError("nvcc not found (set CUDA_HOME)")


def _run(cmd):
    res = subprocess.run(cmd, capture_output=True, text=True)
    log = " ".join(cmd) + "\n" + res.stdout + res.stderr
    if res.returncode != 0:
        raise RuntimeError(os.path.basename(cmd[0]) + " failed:\n" + res.stderr[-4000:])
    return log


def _binding_object(out):
    import torch
    from torch.utils import cpp_extension

    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], os.path.join(ROOT, "include"),
           os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")]
    abi = int(getattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", True))
    return _run(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}", *(f"-I{p}" for p in inc), "-c",
                 BINDING_SRC, "-o", out])


def build(verbose=False):
    os.makedirs(OUT_DIR, exist_ok=True)
    obj = os.path.join(OUT_DIR, "binding.o")
    lib = [nvcc_path(), ARCH, "-O3", "-lineinfo", "-std=c++17", "--shared", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
           "-I", os.path.join(ROOT, "include"), "--threads", "0", "-o", OUT, *SRCS]
    with ThreadPoolExecutor(2) as pool:
        jobs = [pool.submit(_run, lib), pool.submit(_binding_object, obj)]
        log = jobs[0].result()
        jobs[1].result()
    import torch

    tl = os.path.join(os.path.dirname(torch.__file__), "lib")
    _run(["g++", "-shared", "-o", BINDING_OUT, obj, f"-L{OUT_DIR}", "-l:libspecverify.so", f"-L{tl}", "-lc10", "-lc10_cuda",
          "-ltorch", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"])
    with open(os.path.join(OUT_DIR, "build.log"), "w") as f:
        f.write(log)
    if verbose:
        print(log)
    return OUT


if __name__ == "__main__":
    print(build(verbose=True))
