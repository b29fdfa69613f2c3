"""What the library exports under C names: the calls that the header declares and nothing else. A helper that left it under a
plain name could be replaced by another library's function of that name in the same process, or replace it."""
import shutil
import subprocess

import pytest

q = pytest.importorskip("bit_nf4_quantised_amd")


@pytest.mark.skipif(shutil.which("nm") is None, reason="no nm")
def test_c_names_are_those_of_the_header():
    out = subprocess.run(["nm", "-D", "--defined-only", q.LIB_PATH], capture_output=True, text=True, check=True).stdout
    names = {line.split()[2] for line in out.splitlines() if line.split()[1] in "TW"}
    assert {n for n in names if not n.startswith("_")} == set(q.EXPORTED)
