"""Host code of the library's headers, compiled for the tests that look at its launch plans on the CPU."""
from __future__ import annotations

import ctypes
import importlib.util
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_nf4_quantised_amd", "csrc")


def host_library(folder, source: str) -> ctypes.CDLL:
    """`source`, which may include the headers of csrc/, as a library of host code alone."""
    spec = importlib.util.spec_from_file_location("_nf4_build", os.path.join(ROOT, "bit_nf4_quantised_amd", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    cpp, lib = os.path.join(folder, "plan.cpp"), os.path.join(folder, "plan.so")
    with open(cpp, "w") as f:
        f.write(source)
    res = subprocess.run([build.hipcc(), "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-shared", "-I", CSRC,
                          cpp, "-o", lib], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    return ctypes.CDLL(lib)
