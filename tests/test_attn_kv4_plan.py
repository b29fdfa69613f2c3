"""Plans of attention over a 4-bit cache: every launch fits, whatever the kernel's workgroups are. No kernel runs here."""
import pytest

from kv4_cases import CASES, name_of, sequences
from plan_helpers import Kv4Plans

THREADS = (1 << 32) - 1     # of a launch


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    return Kv4Plans(tmp_path_factory.mktemp("kv4_plan"))


def test_launches_of_workgroups_of_512_threads_fit(plan):
    """64 sequences of three row tiles, over 65528 key heads, are 1.5 times what a launch of 512-thread workgroups holds."""
    heads, n = 65528, 768
    seqs = [(n * i, n, 0, 70) for i in range(64)]
    few, many = plan(seqs, heads, heads, 8)
    assert few["kernel"] == -1 and many["kernel"] == 3
    assert 64 * 3 * heads * 512 > THREADS
    assert many["launches"] == 2 and many["threads"] <= THREADS


@pytest.mark.parametrize("heads,kv", [(65528, 65528), (65535, 1), (4096, 64), (32, 8)])
@pytest.mark.parametrize("nq", [1, 17, 33, 65, 300, 1025, 16384])
@pytest.mark.parametrize("nk", [1, 4000, (1 << 30) - 1])
def test_every_launch_fits(plan, heads, kv, nq, nk):
    if -(-nq * (heads // kv) // 32) * kv > (1 << 24) - 1:       # refused
        return
    for p in plan([(nq * i, nq, 0, nk) for i in range(130)], heads, kv, 128):
        assert p["threads"] <= THREADS and p["groups"] < 1 << 31


@pytest.mark.parametrize("case", CASES, ids=name_of)
def test_cases_take_the_kernels_that_they_are_for(plan, case):
    few, many = plan(sequences(case), case.heads, case.kv, case.d, case.book, case.window)
    taken = few if case.nq * case.heads // case.kv <= 32 else many
    assert (taken["kernel"], taken["several"] > 0) == (case.kernel, case.several)


def test_cases_cover_every_kernel():
    have = {(c.kernel, c.d <= 64, c.book == "fp4", c.several) for c in CASES}
    assert len(have) == 4 * 2 * 2 * 2
