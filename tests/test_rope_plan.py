"""The rotation's workgroups: as many as there is work, up to a limit that queries and keys share, for every number of heads.
No kernel runs here."""
import ctypes

import pytest

from plan_helpers import host_library

GRID, SUMS, PER = 65536, 4096, 4     # most workgroups without and with sums of dw; heads of an item


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    lib = host_library(tmp_path_factory.mktemp("rope_plan"), """
#include "rope_plan.h"
extern "C" int plan(long long tokens, int heads, int kv_heads, int d, int sums, int* q_groups, int* per) {
  nf4::RopeArgs a{};
  a.tokens = tokens;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.d = d;
  const int groups = nf4::rope_plan(a, sums != 0);
  *q_groups = a.q_groups;
  *per = a.per;
  return groups;
}
""")

    def call(tokens, heads, kv, d, sums):
        q, per = ctypes.c_int(), ctypes.c_int()
        n = lib.plan(ctypes.c_longlong(tokens), heads, kv, d, int(sums), ctypes.byref(q), ctypes.byref(per))
        return n, q.value, per.value
    return call


def _full(tokens, heads, d, per):
    """Workgroups that leave no group of lanes an item more than another."""
    return -(-tokens * -(-heads // per) // (32 if d <= 64 else 16))


@pytest.mark.parametrize("heads,kv", [(1, 0), (8, 2), (64, 8), (64, 1), (32767, 0), (32768, 0), (32768, 8), (65535, 0), (65535, 1), (65535, 65535), (1, 65535)])
@pytest.mark.parametrize("tokens", [1, 37, 200, 4096, 1 << 20, 1 << 40])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sums", [False, True])
def test_every_number_of_heads_fills_the_grid(plan, tokens, heads, kv, d, sums):
    n, q, per = plan(tokens, heads, kv, d, sums)
    assert per in (PER, 2 * PER) and (sums or per == PER)
    want_q, want_k = _full(tokens, heads, d, per), _full(tokens, kv, d, per) if kv else 0
    most = SUMS if sums else GRID
    assert 1 <= q and (n > q) == (kv > 0)
    if want_q + want_k <= most:
        assert (n, q) == (want_q + want_k, want_q)
    else:       # the limit, or nearly: a share is a whole number
        assert n <= most and (n >= most - 1 or n - q == want_k)
        # shares by the heads; the keys take what is left
        assert abs(q - most * heads / (heads + kv)) <= 1


def test_where_groups_go_on_to_further_tokens(plan):
    """The sizes of the GPU test of it."""
    q, k = 54613, 10923
    assert plan(450000, 5, 1, 128, False) == (q + k, q, 4) and q * 16 < 2 * 450000 and k * 16 < 450000
    q, k = 3413, 683
    assert plan(450000, 5, 1, 128, True) == (q + k, q, 8) and q * 16 < 450000 and k * 16 < 450000
