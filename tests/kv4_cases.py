"""Batches that take each kernel of the attention over a 4-bit cache: every number of rows a workgroup (16, 32, 128 and 256, the
kernels 0 to 3), both padded head sizes, tables and E2M1, one range of keys and several. A CPU test holds the kernels that they
are planned for to what is said here; the GPU tests run them."""
from collections import namedtuple

Case = namedtuple("Case", "kernel several heads kv d book nq nks causal window", defaults=(True, 0))

CASES = [
    Case(0, False, 4, 2, 64, "nf4", 1, [70, 33]),
    Case(0, False, 4, 2, 64, "fp4", 1, [70, 33]),
    Case(0, False, 4, 2, 40, "int4", 1, [33]),
    Case(0, False, 4, 2, 128, "nf4", 1, [70, 33]),
    Case(0, False, 4, 2, 96, "fp4", 3, [70, 2, 33]),
    Case(0, True, 4, 2, 64, "nf4", 1, [1000, 3, 500]),
    Case(0, True, 4, 2, 40, "fp4", 1, [1300]),
    Case(0, True, 4, 2, 128, "nf4", 1, [1000, 3, 500]),
    Case(0, True, 4, 2, 128, "fp4", 2, [1300]),
    Case(0, True, 4, 2, 72, "int4", 3, [1000, 40], False),
    Case(1, False, 8, 1, 64, "fp4", 5, [70]),
    Case(1, False, 8, 1, 64, "nf4", 5, [70]),
    Case(1, False, 8, 1, 128, "fp4", 5, [33]),
    Case(1, False, 8, 1, 128, "nf4", 5, [70]),
    Case(1, True, 8, 1, 64, "fp4", 5, [1000]),
    Case(1, True, 12, 4, 64, "nf4", 13, [500, 480, 500]),
    Case(1, True, 8, 1, 128, "fp4", 5, [500]),
    Case(1, True, 4, 2, 128, "nf4", 31, [1000]),
    Case(2, False, 8, 1, 64, "fp4", 5, [33]),
    Case(2, False, 8, 1, 64, "nf4", 5, [33]),
    Case(2, False, 8, 1, 128, "fp4", 65, [33]),
    Case(2, False, 8, 1, 128, "nf4", 5, [33]),
    Case(2, True, 8, 1, 64, "fp4", 65, [300]),
    Case(2, True, 8, 1, 64, "nf4", 5, [500]),
    Case(2, True, 8, 1, 128, "fp4", 65, [300]),
    Case(2, True, 8, 1, 128, "nf4", 5, [300]),
    Case(2, True, 8, 1, 80, "int4", 65, [700], True, 500),
    Case(2, True, 8, 1, 80, "fp4", 65, [700], False),
    Case(3, False, 16, 4, 64, "nf4", 33, [33 + i % 5 for i in range(40)]),
    Case(3, False, 16, 4, 40, "int4", 33, [33] * 40, False),
    Case(3, False, 16, 4, 64, "fp4", 62, [300] * 64 + [135] * 32),
    Case(3, False, 16, 4, 128, "nf4", 33, [33 + i % 5 for i in range(40)]),
    Case(3, False, 16, 4, 128, "fp4", 33, [33] * 40),
    Case(3, False, 16, 4, 96, "nf4", 70, [100, 7, 130] * 14, True, 50),
    Case(3, True, 16, 4, 64, "nf4", 33, [4100, 4100, 4000]),
    Case(3, True, 32, 8, 64, "fp4", 128, [1000] + [100] * 64),
    Case(3, True, 5, 5, 128, "nf4", 129, [4100, 4100, 4000]),
    Case(3, True, 8, 8, 128, "fp4", 129, [2000] * 8),
    Case(3, True, 32, 8, 80, "int4", 257, [2500, 700], True, 1500),
    Case(3, True, 32, 8, 128, "nf4", 257, [2500, 100], False),
]


def sequences(c):
    """(q0, nq, k0, nk) of a case, with keys that no sequence has between them."""
    seqs, at = [], 2
    for i, n in enumerate(c.nks):
        seqs.append((i * c.nq, c.nq, at, n))
        at += n + 3
    return seqs


def name_of(c):
    return f"kernel{c.kernel}-{'several' if c.several else 'one'}-d{c.d}-{c.book}-{c.nq}x{len(c.nks)}" + \
        ("" if c.causal else "-all") + (f"-w{c.window}" if c.window else "")
