"""Build libfbob.so in-tree with nvcc for sm_103a, and the Python binding of
the operators around the attention (``bind/``) against torch's headers.

Every translation unit under ``csrc/`` is compiled in parallel to an object
file under ``_build/`` and linked into ``exact_second_order_attn_gb300/libfbob.so``.
The CUDA runtime is linked statically; the CUDA driver is reached through the
runtime's entry-point query, so the library loads on machines without a GPU.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfbob.so")
BIND = os.path.join(PKG, "bind")
EXT = os.path.join(PKG, "_fbob_model" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-diag-suppress", "177", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _deps():
    return [os.path.join(d, f) for d in (CSRC, INCLUDE, BIND) for f in os.listdir(d)]


def _torch_stamp():
    """What the binding is compiled against (a file of this name marks it built)."""
    import torch
    return os.path.join(BUILD, "torch-" + torch.__version__)


def _compile(nvcc, src, verbose_ptxas=False):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc, *ARCH, *COMMON, "-c", src, "-o", obj]
    if verbose_ptxas and src.endswith(".cu"):
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _compile_binding():
    import torch
    root = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "model_bind.o")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-w", "-c", os.path.join(BIND, "model_bind.cpp"),
           "-o", obj, "-I", os.path.join(root, "include"), "-I", os.path.join(root, "include/torch/csrc/api/include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           "-I", INCLUDE, f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the binding did not compile:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = EXT + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", PKG, "-l:libfbob.so", "-Wl,-rpath,$ORIGIN",
           "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the binding did not link:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)
    open(_torch_stamp(), "w").close()


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int | None = None) -> str:
    """Compile and link libfbob.so and the binding if any source is newer than
    they are, or the binding is another torch's; return libfbob.so's path."""
    srcs = sources()
    if not force and os.path.exists(LIB) and os.path.exists(EXT) and os.path.exists(_torch_stamp()):
        t = min(os.path.getmtime(LIB), os.path.getmtime(EXT))
        if all(os.path.getmtime(p) <= t for p in _deps()):
            return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or max(1, min(len(srcs), os.cpu_count() or 4))
    with cf.ThreadPoolExecutor(jobs + 1) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(lambda s: _compile(nvcc, s, verbose_ptxas), srcs))
    if verbose_ptxas:
        for _, log in results:
            if log.strip():
                sys.stderr.write(log)
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
