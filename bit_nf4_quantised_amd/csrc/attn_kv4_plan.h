// Which kernel takes the sequences of an attention over a 4-bit cache, in which ranges of keys and in which launches (host
// side; attn_kv4.hip).
#pragma once
#include "attn.h"

namespace nf4 {

inline int64_t kv4_keys(const AttnSeq& s, int window) { return std::max<int64_t>(1, s.nk - first_key(s, window)); }

// The kernels: rows of a workgroup, keys of a step (a range is a multiple of it), workgroups that a compute unit holds, and
// the time of a step in us with 1, 2 .. of them on it, d = 128 and d <= 64, for tables and for E2M1 each. Measured as the
// difference of 16 steps and 8 of workgroups that are all alike. Calls (us) with each of the four, NF4, d 128:
//   24 rows, 16 times 4000 keys, 8 key heads   51   36   53   67         100 rows, 4 times 8000   83   57   45   49
//   64 rows, 16 times 1000 keys                26   21   28   30         400 rows, 8000 keys      72   56   45   38
//   1200 rows, twice 4000 keys                174  135   75   64         100 rows, 1000 keys      11.5 11.8 14.2 13.6
// The estimate below chose the fastest of each, or one within 0.3 us of it.
struct Kv4Kernel {
  int rows, waves, step, most;
  double us[2][2][3];
  constexpr int64_t groups() const { return kMaxThreads / (waves * 64); }   // of a launch
};
constexpr Kv4Kernel kKv4Kernels[] = {
    {16, 4, 128, 3, {{{1.65, 2.4, 3.4}, {1.05, 1.6, 2.2}}, {{1.25, 1.55, 2.0}, {0.95, 1.1, 1.5}}}},
    {32, 4, 128, 2, {{{1.9, 2.6, 0}, {1.25, 1.95, 0}}, {{1.4, 1.8, 0}, {1.05, 1.25, 0}}}},
    {128, 4, 64, 2, {{{1.6, 2.5, 0}, {1.4, 2.25, 0}}, {{1.1, 1.6, 0}, {1.0, 1.4, 0}}}},
    {256, 8, 64, 1, {{{2.05, 0, 0}, {1.95, 0, 0}}, {{1.55, 0, 0}, {1.45, 0, 0}}}},
};

// The sequences of one launch form: their rows in tiles of the kernel's, their keys in ranges of about `chunk`.
struct Kv4Class {
  std::vector<AttnSeq> seqs;
  int kernel = 0;
  int64_t chunk = 0;
  const Kv4Kernel& k() const { return kKv4Kernels[kernel]; }
  int64_t tiles(const AttnSeq& s, int G) const { return ceil64((int64_t)s.nq * G, k().rows); }
  int ranges(const AttnSeq& s, int window) const { return (int)ceil64(kv4_keys(s, window), chunk); }
};
struct Kv4Plan {
  Kv4Class few, many;        // sequences of up to 32 rows, and of more
  int64_t part_floats = 0;   // workspace of one launch (the largest)
};

inline AttnSeqs kv4_seqs(const Kv4Class& c, size_t from, int G, int kv_heads, int window) {
  return pack_seqs(c.seqs, from, kv_heads, [&](const AttnSeq& s) { return c.tiles(s, G) * c.ranges(s, window); }, c.k().groups());
}

// Chooses the kernel among [from, to) and the length of a range by the smallest estimate: 5 us around the steps (launch, first
// loads, joining the waves), the longest range's steps at the rate of a unit that holds its share of workgroups, times the
// rounds of workgroups, and, where there are ranges to join, 3.5 us and their sums, written and read, at 3.5 TB/s.
inline double up(double x) {   // to a whole number; x is not large
  const int64_t i = (int64_t)x;
  return (double)(i + ((double)i < x));
}
inline void kv4_choose(Kv4Class& c, int from, int to, bool e2m1, int G, int kv_heads, int d, int window) {
  const size_t n = c.seqs.size();
  std::vector<double> keys(n), rows(n);
  double longest = 1;
  for (size_t i = 0; i < n; ++i) {
    keys[i] = (double)kv4_keys(c.seqs[i], window);
    rows[i] = (double)c.seqs[i].nq * G;
    longest = std::max(longest, keys[i]);
  }
  double best = -1;
  for (int x = from; x < to; ++x) {
    const Kv4Kernel& k = kKv4Kernels[x];
    for (double chunk = k.step;; chunk = up(chunk * 1.19 / k.step) * k.step) {
      const bool whole = chunk >= longest;
      double large = 0, records = 0, joined = 0, load = 0, top = 0, most = 0;
      for (size_t i = 0; i < n; ++i) {
        const double r = whole ? 1 : up(keys[i] / chunk), w = up(rows[i] / k.rows) * kv_heads;
        if (keys[i] > 0.5 * r * std::min(chunk, longest)) large += w * r;
        most = std::max(most, w * r);
        load += w * keys[i];
        top = std::max(top, up(keys[i] / (r * k.step)) * k.step);
        if (r > 1) {
          joined += rows[i] * kv_heads;
          records += rows[i] * kv_heads * r;
        }
      }
      // a sequence has to fit a launch, and so have the rows to join
      if (whole || (most <= (double)k.groups() && joined <= (double)(1 << 22))) {
        // workgroups on each of 256 units: those of more than half a range's length, or by the work
        const double full = std::max({1.0, up(large / 256), up(load / top / 256 - 0.25)});
        const int on = (int)std::min<double>(k.most, full);
        const double us = 5 + top / k.step * k.us[d <= 64][e2m1][on - 1] * up(full / on) +
                          (records > 0 ? 3.5 + records * (d + 8) * 8 / 3.5e6 : 0);
        if (best < 0 || us < best) {
          best = us;
          c.kernel = x;
          c.chunk = (int64_t)(whole ? up(longest / k.step) * k.step : chunk);
        }
      }
      if (whole) break;
    }
  }
}

inline Kv4Plan kv4_plan(const AttnSeq* seqs, int64_t count, int book, int heads, int kv_heads, int d, int window) {
  Kv4Plan p;
  const int G = heads / kv_heads;
  int64_t few_rows = 0, many_rows = 0;
  for (const AttnSeq& s : by_work(seqs, count, false)) {
    const int64_t rows = (int64_t)s.nq * G;
    (rows <= 32 ? p.few : p.many).seqs.push_back(s);
    int64_t& most = rows <= 32 ? few_rows : many_rows;
    most = std::max(most, rows);
  }
  for (Kv4Class* c : {&p.few, &p.many}) {
    if (c->seqs.empty()) continue;
    // 16 rows a workgroup for up to 32 rows, 32 for 17 to 512, 128 and 256 from 33 on
    if (c == &p.few) kv4_choose(*c, 0, few_rows <= 16 ? 1 : 2, book == 1, G, kv_heads, d, window);
    else kv4_choose(*c, many_rows <= 512 ? 1 : 2, many_rows <= 64 ? 3 : 4, book == 1, G, kv_heads, d, window);
    for (size_t from = 0; from < c->seqs.size();) {
      const AttnSeqs q = kv4_seqs(*c, from, G, kv_heads, window);
      int64_t f = 0;
      for (int i = 0; i < q.count; ++i) {
        const int ns = c->ranges(q.seq[i], window);
        if (ns > 1) f += (int64_t)q.seq[i].nq * heads * ns * (d + 8);
      }
      p.part_floats = std::max(p.part_floats, f);
      from += (size_t)q.count;
    }
  }
  return p;
}

}  // namespace nf4
