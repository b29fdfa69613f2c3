// How many workgroups a rotation gets, and which of them take queries (host side; rope.hip).
#pragma once
#include "launch.h"

#include <algorithm>

namespace nf4 {

constexpr int kRopeHeads = 4;      // heads of a token that a group of lanes takes at a time
// Workgroups at most, of queries and of keys together; past them they go on to further tokens. That is slower than more
// workgroups (4096 tokens of 64 and 8 heads, d 128, normed, 2304 and 4608 of them: 25.4 us, and 27.3 with 2048; 32768 tokens
// 199 and 229), but where each leaves partial sums of dw these have to be added (32768 tokens 386 and 354 with 4096).
constexpr int kRopeGrid = 65536, kRopeSums = 4096;

// A group takes 4 heads of a token; where sums of dw are left and there are enough groups for every lane of the
// GPU (8192 of 16 lanes), 8, two rounds of four: half as many sums to join (2048 tokens of 32 and 8 heads, d 128, 17.2 us, and
// 20.3 by fours; 256 tokens 9.5, and 8.5 by fours).
inline int rope_plan(RopeArgs& a, bool sums) {
  const int64_t lanes = a.d <= 64 ? 32 : 16;   // groups of a workgroup
  const int64_t most = sums ? kRopeSums : kRopeGrid;
  auto items = [&](int heads) { return a.tokens * ((heads + a.per - 1) / a.per); };
  a.per = 2 * kRopeHeads;
  if (!sums || items(a.heads) + items(a.kv_heads) < 8192) a.per = kRopeHeads;
  int64_t q = (items(a.heads) + lanes - 1) / lanes, k = (items(a.kv_heads) + lanes - 1) / lanes;
  if (q + k > most) {   // shares by the heads
    q = std::max<int64_t>(1, most * a.heads / (a.heads + a.kv_heads));
    k = std::min<int64_t>(k, most - q);
  }
  a.q_groups = (int)q;
  return (int)(q + k);
}

}  // namespace nf4
