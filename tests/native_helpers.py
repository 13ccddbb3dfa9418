"""Host functions of the library's headers, compiled for the CPU and called
through ctypes."""

from __future__ import annotations

import ctypes
import os
import subprocess

from exact_second_order_attn_gb300 import build as b


def compiled(tmp, source, nvcc=False):
    """The shared object of C++ ``source`` (extern "C" functions), which may
    include the library's internal headers; ``nvcc``: those with device code."""
    src, lib = os.path.join(tmp, "host.cu" if nvcc else "host.cpp"), os.path.join(tmp, "host.so")
    with open(src, "w") as f:
        f.write(source)
    cuda = os.path.join(os.path.dirname(os.path.dirname(b._nvcc())), "include")
    cc = [b._nvcc(), *b.ARCH, *b.COMMON] if nvcc else [os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-fPIC"]
    r = subprocess.run([*cc, "-shared", src, "-o", lib, "-I", b.CSRC, "-I", b.INCLUDE, "-I", cuda],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(lib)
