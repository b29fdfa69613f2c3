"""Kernels whose waves pass values between their lanes through LDS without a workgroup barrier order the accesses by wavefront
fences, in the code that the compiler is left with: a scheduling barrier alone orders no memory. Compiles, runs nothing."""
import importlib.util
import os
import re
import subprocess

import pytest

from plan_helpers import CSRC, ROOT


def _functions(source, folder):
    """The optimised device functions of a source by name, as LLVM IR."""
    spec = importlib.util.spec_from_file_location("_nf4_build", os.path.join(ROOT, "bit_nf4_quantised_amd", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    out = os.path.join(folder, source + ".ll")
    res = subprocess.run([build.hipcc()] + build.COMMON + ["--offload-device-only", "-emit-llvm", "-S", os.path.join(CSRC, source),
                                                            "-o", out], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    return dict(re.findall(r"^define [^@]*@([\w.]+)\(.*?\{\n(.*?)^\}", open(out).read(), flags=re.S | re.M))


@pytest.mark.slow
@pytest.mark.parametrize("source,kernel,exchanges", [("rope.hip", "rope_dw_kernel", 1), ("attn_kv4.hip", "attn_kv4_few_kernel", 3)])
def test_exchanges_between_lanes_are_fenced(source, kernel, exchanges, tmp_path):
    found = {n: body for n, body in _functions(source, tmp_path).items() if kernel in n}
    assert found
    for name, body in found.items():
        order = re.findall(r"fence syncscope\(\"wavefront\"\) (\w+)|(wave)\.barrier\(", body)
        steps = [a or b for a, b in order]
        assert len(steps) >= 3 * exchanges and steps == ["release", "wave", "acquire"] * (len(steps) // 3), (name, steps)
