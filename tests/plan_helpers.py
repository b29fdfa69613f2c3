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


KV4_PLAN = r"""
#include "attn_kv4_plan.h"
// Of the sequences of up to 32 rows and of those with more: kernel (-1: none), launches, most ranges of a sequence, sequences of
// several ranges, most workgroups and most threads of a launch.
extern "C" void kv4_plan(const long long* seqs, long long count, int book, int heads, int kv_heads, int d, int window, long long* out) {
  std::vector<nf4::AttnSeq> v;
  for (long long i = 0; i < count; ++i) v.push_back({seqs[4 * i], seqs[4 * i + 2], (int)seqs[4 * i + 1], (int)seqs[4 * i + 3]});
  const nf4::Kv4Plan p = nf4::kv4_plan(v.data(), count, book, heads, kv_heads, d, window);
  for (const nf4::Kv4Class* c : {&p.few, &p.many}) {
    long long launches = 0, ranges = 0, several = 0, groups = 0;
    for (size_t from = 0; from < c->seqs.size();) {
      const nf4::AttnSeqs q = nf4::kv4_seqs(*c, from, heads / kv_heads, kv_heads, window);
      for (int i = 0; i < q.count; ++i) {
        const long long n = c->ranges(q.seq[i], window);
        ranges = std::max(ranges, n);
        several += n > 1;
      }
      groups = std::max(groups, (long long)q.first[q.count] * kv_heads);
      ++launches;
      from += (size_t)q.count;
    }
    *out++ = c->seqs.empty() ? -1 : c->kernel;
    *out++ = launches;
    *out++ = ranges;
    *out++ = several;
    *out++ = groups;
    *out++ = groups * c->k().waves * 64;
  }
}
"""
BOOKS = {"nf4": 0, "fp4": 1, "int4": 2}


class Kv4Plans:
    """The plans of attention over a 4-bit cache: few and many, each a dict of what KV4_PLAN says."""

    def __init__(self, folder):
        self._lib = host_library(folder, KV4_PLAN)

    def __call__(self, seqs, heads, kv, d, book="nf4", window=0):
        flat = [v for s in seqs for v in s]
        out = (ctypes.c_longlong * 12)()
        self._lib.kv4_plan((ctypes.c_longlong * len(flat))(*flat), ctypes.c_longlong(len(seqs)), BOOKS[book], heads, kv, d, window, out)
        names = ("kernel", "launches", "ranges", "several", "groups", "threads")
        return dict(zip(names, out[:6])), dict(zip(names, out[6:]))
