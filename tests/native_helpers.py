"""Host functions of the library's headers, compiled for the CPU and called
through ctypes."""

from __future__ import annotations

import ctypes
import os
import subprocess

from exact_second_order_attn_gb300 import build as b


def compiled(tmp, source):
    """The shared object of C++ ``source`` (extern "C" functions), which may
    include the library's internal headers."""
    src, lib = os.path.join(tmp, "host.cpp"), os.path.join(tmp, "host.so")
    with open(src, "w") as f:
        f.write(source)
    cuda = os.path.join(os.path.dirname(os.path.dirname(b._nvcc())), "include")
    r = subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-shared", "-fPIC", src, "-o", lib, "-I", b.CSRC,
                        "-I", b.INCLUDE, "-I", cuda], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(lib)
