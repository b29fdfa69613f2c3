// Attention over a key/value cache in 4 bits (gfx950): as attention over the bf16 values that its blocks stand
// for (kv4.h), which exist only in registers and LDS.
//
// Scores, softmax and sums are those of attn.hip: streamed keys as result rows and query rows as result columns of the
// first product, fp32 statistics, probabilities rounded to bf16 where they enter the second product (2^-8). The query
// heads that share a key head are packed with the tokens into rows (row = token * group + head in group), so a block is
// dequantised for all of them. Blocks are dequantised in the order of Kv4Table::eight(); the queries are put
// in the same order, and the output's columns back into theirs.
//
// A value block that stands for NaN enters as zeros, and the same block of its key as NaN: a query that sees the
// key gets NaN through the score, and one that does not gets nothing of it (0 times NaN would be NaN). A key's block
// of infinite maximum is NaN with every code: a score of minus infinity would pass for a hidden key.
//
// Keys of a range that end within a tile: the lanes past it take the last key again, which the mask hides.
#include "attn_kv4_plan.h"
#include "kv4.h"

namespace nf4 {

// The ranges of keys of a launch's sequences.
struct Kv4Split {
  float* part;   // per row, key head and range: d sums, maximum, sum, 6 unused
  int lo[kAttnSeqs], chunk[kAttnSeqs], ranges[kAttnSeqs];   // first key, keys a range, how many
  int64_t row0[kAttnSeqs];        // first record of a sequence in part
  int join_first[kAttnSeqs + 1];  // prefix sums of rows x key heads over the sequences of several ranges
};
// A workgroup's sequence with its ranges. Lane i reads all entries of sequence i before the workgroup knows which it needs: a
// second trip to the kernel arguments would cost its start about 0.4 us (one token of 601 keys 6.4 us, and 6.0 so).
struct Kv4Found {
  Found at;
  int lo, chunk, ranges;
  int64_t row0;
};
__device__ __forceinline__ Kv4Found kv4_find(const AttnSeqs& sq, const Kv4Split& sp, int tile) {
  const int lane = threadIdx.x & 63;
  const int lo = sp.lo[lane], chunk = sp.chunk[lane], ranges = sp.ranges[lane];
  const int64_t row0 = sp.row0[lane];
  Kv4Found f;
  f.at = find_seq(sq, tile);
  f.lo = lane_value(lo, f.at.index);
  f.chunk = lane_value(chunk, f.at.index);
  f.ranges = lane_value(ranges, f.at.index);
  f.row0 = lane_value(row0, f.at.index);
  return f;
}

__device__ __forceinline__ bool kv4_lost(uint32_t absmax) { return absmax >= kBf16Infinity; }   // absmax has no sign

// ------------------------------------------------------------------------------------------
// Few rows: 16 NR rows a workgroup, its keys one range of the sequence's, of which its four waves take 32-key tiles in
// turn; there are no barriers until the waves are joined. Products are v_mfma_f32_16x16x32_bf16: lane (n, q) = (lane
// % 16, lane / 16) holds of a result column n and rows 4 q .. 4 q + 3, of an operand row (or column) n and 8 values.
// The contraction of the first product may run over d in any order, so lane (n, q) takes the block q (d <= 64: half
// the block q / 2) of keys n and 16 + n as it lies in the cache, 16 bytes, and its dequantised dwords are the
// operand. Values go through an LDS tile of the wave's own, from which transpose loads read them across.
// Bound by the vector instructions of the tables' codes (3 a value, shared by the 8 or 16 rows that a token or two leave), then
// by memory: one token each over 16 caches of 1 to 8191 keys, 64 heads over 8, d 128, takes 25 us (63 MB, 2.5 TB/s) in NF4;
// 131071 and 60001 keys in E2M1, whose codes cost 2 instructions a value, 47 (220 MB, 4.7 TB/s). Three waves a SIMD: the
// registers of four spill (32 us for the first of these). One range with 8 or 16 waves a workgroup instead of several
// ranges and a join takes 10.3 to 13 us for 601 keys that take 8.2 so: the codes of a key head are then one unit's work.
template <int DP>
struct Kv4Few;
// d > 64: lane (n, q) holds block q of keys n and 16 + n, key and value
template <>
struct Kv4Few<128> {
  u32x4 k[2], v[2];
  uint32_t ka[2], va[2];
  __device__ __forceinline__ void load(const AttnKv4Args& a, int64_t kt, int64_t vt, int last, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t key = (uint32_t)min(16 * i + (lane & 15), last), b = (uint32_t)min(lane >> 4, a.nb - 1);
      const uint32_t ko = key * (uint32_t)a.k4.token + b, vo = key * (uint32_t)a.v4.token + b;
      k[i] = *reinterpret_cast<const u32x4*>(a.k4.codes + 16 * kt + 16u * ko);
      v[i] = *reinterpret_cast<const u32x4*>(a.v4.codes + 16 * vt + 16u * vo);
      ka[i] = a.k4.absmax[kt + ko];
      va[i] = a.v4.absmax[vt + vo];
    }
  }
  __device__ __forceinline__ uint32_t absmax(int i) const { return kv4_lost(max(ka[i], va[i])) ? kBf16Nan : ka[i]; }
  template <class Deq>
  __device__ __forceinline__ void values(uint16_t* tile, const typename Deq::Shared& tables, const AttnKv4Args& a, int lane) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Deq q(tables, a.t, a.unit, kv4_lost(va[i]) ? 0u : va[i]);
#pragma unroll
      for (int t = 0; t < 4; ++t)
        *reinterpret_cast<u32x4*>(tile + Tile<128>::elem(16 * i + (lane & 15), 4 * (lane >> 4) + t)) = q.eight(v[i][t]);
    }
  }
  // column of the lane's 8 values of the first product's step t
  static __device__ __forceinline__ int column(int t, int lane) { return 32 * (lane >> 4) + 8 * t; }
};
// d <= 64: half the block q / 2 of keys n and 16 + n, and block lane / 32 of value lane % 32
template <>
struct Kv4Few<64> {
  u32x2 k[2];
  u32x4 v;
  uint32_t ka[2], kva[2], va;
  __device__ __forceinline__ void load(const AttnKv4Args& a, int64_t kt, int64_t vt, int last, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t key = (uint32_t)min(16 * i + (lane & 15), last), b = (uint32_t)min(lane >> 5, a.nb - 1);
      const uint32_t ko = key * (uint32_t)a.k4.token + b;
      k[i] = *reinterpret_cast<const u32x2*>(a.k4.codes + 16 * kt + (16u * ko + 8u * ((uint32_t)lane >> 4 & 1u)));
      ka[i] = a.k4.absmax[kt + ko];
      kva[i] = a.v4.absmax[vt + (key * (uint32_t)a.v4.token + b)];
    }
    const uint32_t vo = (uint32_t)min(lane & 31, last) * (uint32_t)a.v4.token + (uint32_t)min(lane >> 5, a.nb - 1);
    v = *reinterpret_cast<const u32x4*>(a.v4.codes + 16 * vt + 16u * vo);
    va = a.v4.absmax[vt + vo];
  }
  __device__ __forceinline__ uint32_t absmax(int i) const { return kv4_lost(max(ka[i], kva[i])) ? kBf16Nan : ka[i]; }
  template <class Deq>
  __device__ __forceinline__ void values(uint16_t* tile, const typename Deq::Shared& tables, const AttnKv4Args& a, int lane) const {
    const Deq q(tables, a.t, a.unit, kv4_lost(va) ? 0u : va);
#pragma unroll
    for (int t = 0; t < 4; ++t)
      *reinterpret_cast<u32x4*>(tile + Tile<64>::elem(lane & 31, 4 * (lane >> 5) + t)) = q.eight(v[t]);
  }
  static __device__ __forceinline__ int column(int t, int lane) { return 16 * (lane >> 4) + 8 * t; }
};

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// maximum and sum over the four lanes of a column, in all of them
__device__ __forceinline__ float quarter_max(float v) {
  v = half_max(v);
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float quarter_sum(float v) {
  v = half_sum(v);
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// the operand whose rows are tile columns 16 dt .. 16 dt + 15 and whose contraction runs over 32 tile rows in the order of
// two 16-row score accumulators: lane quarter q takes rows 4 q .. 4 q + 3, then 16 + 4 q .. 16 + 4 q + 3
template <int DP>
__device__ __forceinline__ bf16x8 cols16(const uint16_t* t, int dt, int lane) {
  const int j = lane & 15, m = 4 * (lane >> 4) + (j >> 2), c = 2 * dt + ((j & 3) >> 1);
  const uint16_t* base = t + 4 * (j & 1);
  bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(base + Tile<DP>::elem(m, c)));
  bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(base + Tile<DP>::elem(m + 16, c)));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Running softmax of 16 rows (one per lane column) over 32 streamed keys a step, as Online.
template <int DT>
struct Online16 {
  float m, mc, l;
  f32x4 o[DT];
  __device__ __forceinline__ void init() {
    m = -INFINITY;
    mc = 0.f;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < DT; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  __device__ __forceinline__ void update(f32x4 (&s)[2], float c, float slack) {
    float mx = -INFINITY;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[t][i]);
    mx = quarter_max(mx);
    if (__any(mx > m + slack)) {
      const float mn = fmaxf(m, mx);
      const float mnc = mn == -INFINITY ? 0.f : mn * c;
      const float a = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mc - mnc);   // no key yet: l and o are zero
      m = mn;
      mc = mnc;
      l *= a;
#pragma unroll
      for (int k = 0; k < DT; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[k][i] *= a;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[t][i] = __builtin_amdgcn_exp2f(__fmaf_rn(s[t][i], c, -mc));
        l += s[t][i];
      }
  }
};

template <int DP, class Deq, int NR>
__global__ __launch_bounds__(256, NR == 1 ? 3 : 2) void attn_kv4_few_kernel(const AttnKv4Args a, const AttnSeqs sq, const Kv4Split sp) {
  constexpr int NW = 4, BN = 32, KS = DP / 32, DT = DP / 16, R = 16 * NR, P = DP + 4;
  typedef Kv4Few<DP> Blocks;
  // a wave's tile of values, later its outputs as [row][d + 4]
  __shared__ __attribute__((aligned(16))) float lds[NW][R * P];
  __shared__ float Ms[NW][R], Ls[NW][R];
  __shared__ typename Deq::Shared tables;
  static_assert(BN * DP * 2 <= R * P * 4, "the tile fits");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int G = a.f.heads / a.f.kv_heads;
  const Unit u = unit_of((int)blockIdx.x, a.f.kv_heads, 1);
  const Kv4Found found = kv4_find(sq, sp, u.tile);
  const AttnSeq s = found.at.seq;
  const int local = u.tile - found.at.first;
  const int ns = found.ranges, split = local % ns, rt = local / ns;
  const int shift = s.nk - s.nq, rows = s.nq * G;
  const int t0 = rt * R / G, t1 = min(rows - 1, rt * R + R - 1) / G;   // tokens of the row tile
  const Range first = visible(t0 + shift, s.nk, a.f.causal, a.f.window), last = visible(t1 + shift, s.nk, a.f.causal, a.f.window);
  // tiles are counted from the first key that the sequence's first row sees (none before it is read)
  const int lo = found.lo, chunk = found.chunk;
  const int k_lo = lo + max((first.lo - lo) & ~(BN - 1), split * chunk);
  const int k_hi = min(last.hi, lo + (split + 1) * chunk);
  const int64_t kbase = s.k0 * a.k4.token + (int64_t)u.kvh * a.k4.head, vbase = s.k0 * a.v4.token + (int64_t)u.kvh * a.v4.head;
  const int j_w = k_lo + wave * BN;   // the wave's first tile; its tiles are NW apart
  Blocks now, next;
  if (j_w < k_hi) now.load(a, kbase + (int64_t)j_w * a.k4.token, vbase + (int64_t)j_w * a.v4.token, k_hi - 1 - j_w, lane);

  Deq::share(tables, tid, a.t, a.unit);
  bf16x8 qf[NR][KS];
  Range mine[NR];   // keys that the lane's rows see
  Online16<DT> acc[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int row = rt * R + 16 * r + (lane & 15);
    const int tok = min(row, rows - 1) / G, head = u.kvh * G + min(row, rows - 1) % G;
    mine[r] = visible(tok + shift, s.nk, a.f.causal, a.f.window);
    const uint16_t* q = a.f.q.p + (s.q0 + tok) * a.f.q.token + (int64_t)head * a.f.q.head;
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      const int col = Blocks::column(t, lane);
      u32x4 v = u32x4{0u, 0u, 0u, 0u};
      if (row < rows && col < a.f.d) v = *reinterpret_cast<const u32x4*>(q + col);
      qf[r][t] = __builtin_bit_cast(bf16x8, kv4_order(v));
    }
    acc[r].init();
  }
  const float slack = slack_of(a.f.c);
  uint16_t* const vt = reinterpret_cast<uint16_t*>(lds[wave]);
  lds_barrier();   // the tables are there

  // the tile of keys from j, in `now`; the wave's next goes to `next`
  auto tile = [&](Blocks& now, Blocks& next, int j) __attribute__((always_inline)) {
    const int jn = j + NW * BN;
    if (jn < k_hi) next.load(a, kbase + (int64_t)jn * a.k4.token, vbase + (int64_t)jn * a.v4.token, k_hi - 1 - jn, lane);
    f32x4 sc[NR][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Deq kq(tables, a.t, a.unit, now.absmax(i));
#pragma unroll
      for (int t = 0; t < KS; ++t) {
        const bf16x8 kf = __builtin_bit_cast(bf16x8, kq.eight(now.k[i][t]));
#pragma unroll
        for (int r = 0; r < NR; ++r) sc[r][i] = mfma16(kf, qf[r][t], t ? sc[r][i] : f32x4{0.f, 0.f, 0.f, 0.f});
      }
    }
    wave_lds_order();   // the last tile's values have been read
    now.template values<Deq>(vt, tables, a, lane);
    wave_lds_order();
    // some row does not see some key
    if (j + BN > first.hi || j < last.lo) {
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        asm volatile("" : "+v"(sc[r][0]), "+v"(sc[r][1]));   // few tiles come here: keep it out of the others' way
        const int at = mine[r].lo - j - 4 * (lane >> 4);
        const uint32_t n = (uint32_t)max(mine[r].hi - mine[r].lo, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((uint32_t)(16 * (i >> 2) + (i & 3) - at) >= n) sc[r][i >> 2][i & 3] = -INFINITY;
      }
    }
    bf16x8 p[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      acc[r].update(sc[r], a.f.c, slack);
      p[r] = __builtin_bit_cast(bf16x8, u32x4{pack_bf16x2(sc[r][0][0], sc[r][0][1]), pack_bf16x2(sc[r][0][2], sc[r][0][3]),
                                              pack_bf16x2(sc[r][1][0], sc[r][1][1]), pack_bf16x2(sc[r][1][2], sc[r][1][3])});
    }
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      const bf16x8 vf = cols16<DP>(vt, dt, lane);
#pragma unroll
      for (int r = 0; r < NR; ++r) acc[r].o[dt] = mfma16(vf, p[r], acc[r].o[dt]);
    }
  };
  for (int j = j_w; j < k_hi; j += NW * BN) {
    tile(now, next, j);
    now = next;
  }

  // join the waves: each leaves its statistics and sums, which are scaled to the common maximum and added in wave order
  wave_lds_order();   // its tile has been read
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const float l = quarter_sum(acc[r].l);
    const int at = 16 * r + (lane & 15);
    if (lane < 16) {
      Ms[wave][at] = acc[r].m;
      Ls[wave][at] = l;
    }
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) *reinterpret_cast<f32x4*>(&lds[wave][at * P + 16 * dt + 4 * (lane >> 4)]) = acc[r].o[dt];
  }
  __syncthreads();
  for (int x = tid; x < R * (DP / 8); x += 256) {   // 8 columns a thread
    const int row = x / (DP / 8), c0 = x % (DP / 8) * 8, grow = rt * R + row;
    if (grow >= rows) break;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) mx = fmaxf(mx, Ms[w][row]);
    const float mxc = mx == -INFINITY ? 0.f : mx * a.f.c;
    float l = 0.f, v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = Ms[w][row] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(Ms[w][row] * a.f.c - mxc);
      l += Ls[w][row] * f;   // 0 times NaN stays NaN
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __fmaf_rn(lds[w][row * P + c0 + kv4_place_of(e)], f, v[e]);
    }
    if (c0 >= a.f.d) continue;
    const int tok = grow / G, head = u.kvh * G + grow % G;
    if (ns == 1) {
      const float inv = inverse_sum(l);
      *reinterpret_cast<u32x4*>(a.f.o.p + (s.q0 + tok) * a.f.o.token + (int64_t)head * a.f.o.head + c0) =
          u32x4{pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv),
                pack_bf16x2(v[4] * inv, v[5] * inv), pack_bf16x2(v[6] * inv, v[7] * inv)};
      if (c0 == 0 && a.f.lse) a.f.lse[(int64_t)head * a.f.lse_stride + s.q0 + tok] = lse_of(mxc, l);
    } else {
      float* part = sp.part + (found.row0 + ((int64_t)grow * a.f.kv_heads + u.kvh) * ns + split) * (int64_t)(a.f.d + 8);
      *reinterpret_cast<f32x4*>(part + c0) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(part + c0 + 4) = f32x4{v[4], v[5], v[6], v[7]};
      if (c0 == 0) {
        part[a.f.d] = l == 0.f ? -INFINITY : mxc;   // finite (0 at least) where the sum is NaN: the join reads it
        part[a.f.d + 1] = l;
      }
    }
  }
}

// ------------------------------------------------------------------------------------------
// Many rows: WV waves of 32 rows each share tiles of 64 keys in LDS, which they dequantise together, two tiles deep: while
// a tile is multiplied, the next one's codes become values and the one after it is on its way from memory. Products are
// v_mfma_f32_32x32x16_bf16 as in attn.hip. A workgroup's keys are one range of the sequence's.
// Bound by the codes, the softmax and the products together, which two waves a SIMD, in step at the barriers, overlap little: 512
// tokens each on 4096 and 1911 keys, 32 heads over 8, d 128, NF4, take 77 to 79 us (590 TFLOP/s; the vector unit and the matrix
// unit are busy 54 and 37 % of the cycles of the units at work). With 4 waves, of which two workgroups fit a unit, 95:
// twice the codes. Waves that form codes before and after their products in turn 86; products of both key halves in
// turn, and priority for them: no gain. Every row tile dequantises its keys again: 8191 tokens on as many keys take 570 us, and 517
// if the cache is read back once (11) and attended to in bf16; 512 tokens on 8191 keys 89, and 109 so.
template <int DP, int WV>
struct Kv4Many {
  static constexpr int UNITS = 64 * (DP / 32) * 2, N = (UNITS + WV * 64 - 1) / (WV * 64);   // blocks of a tile, and of a thread
  u32x4 c[N];
  uint32_t m[N], vm[N];   // the block's maximum and that of the value's block (for values the same)
  // a wave's units are the 64 keys of one block; in a tile of too few blocks waves do others' work again
  static __device__ __forceinline__ int unit(int tid, int i) { return (i * WV * 64 + tid) % UNITS; }
  static __device__ __forceinline__ bool value(int tid, int i) { return unit(tid, i) >= UNITS / 2; }
  static __device__ __forceinline__ int block(int tid, int i) { return unit(tid, i) / 64 % (DP / 32); }
  __device__ __forceinline__ void load(const AttnKv4Args& a, int64_t kt, int64_t vt, int last, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t key = (uint32_t)min(tid & 63, last), b = (uint32_t)min(block(tid, i), a.nb - 1);
      const bool val = value(tid, i);
      const uint8_t* codes = val ? a.v4.codes + 16 * vt : a.k4.codes + 16 * kt;
      const uint16_t* absmax = val ? a.v4.absmax + vt : a.k4.absmax + kt;
      const uint32_t at = key * (uint32_t)(val ? a.v4.token : a.k4.token) + b;
      c[i] = *reinterpret_cast<const u32x4*>(codes + 16u * at);
      m[i] = absmax[at];
      vm[i] = a.v4.absmax[vt + (key * (uint32_t)a.v4.token + b)];
    }
  }
  // the loaded blocks into a tile
  template <class Deq>
  __device__ __forceinline__ void store(uint16_t* kt, uint16_t* vt, const typename Deq::Shared& tables, const AttnKv4Args& a, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool val = value(tid, i);
      const Deq q(tables, a.t, a.unit, kv4_lost(max(m[i], vm[i])) ? (val ? 0u : kBf16Nan) : m[i]);
      uint16_t* tile = val ? vt : kt;
#pragma unroll
      for (int t = 0; t < 4; ++t)
        *reinterpret_cast<u32x4*>(tile + Tile<DP>::elem(tid & 63, 4 * block(tid, i) + t)) = q.eight(c[i][t]);
    }
  }
};

// Accumulator rows 8 g .. 8 g + 7 (g = 0, 2) of a 32-row result tile, whose rows are the output's columns in the order of
// eight(), exchanged between lane halves so that a lane holds 8 neighbouring columns, 16 (g / 2) + 8 (lane / 32), in order.
__device__ __forceinline__ void kv4_columns(float (&o)[8], const f32x16& v, int g) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[4 * g + k]), __float_as_uint(v[4 * g + 4 + k]), false, false);
    o[2 * k] = __uint_as_float(r[0]);
    o[2 * k + 1] = __uint_as_float(r[1]);
  }
}

template <int DP, class Deq, int WV>
__global__ __launch_bounds__(WV * 64, 2) void attn_kv4_many_kernel(const AttnKv4Args a, const AttnSeqs sq, const Kv4Split sp) {
  constexpr int BN = 64, KS = DP / 16, DT = DP / 32, R = 32 * WV;
  typedef Tile<DP> T;
  __shared__ __attribute__((aligned(16))) uint16_t K0[BN * DP], V0[BN * DP], K1[BN * DP], V1[BN * DP];
  __shared__ typename Deq::Shared tables;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int G = a.f.heads / a.f.kv_heads;
  const Unit u = unit_of((int)blockIdx.x, a.f.kv_heads, 1);
  const Kv4Found found = kv4_find(sq, sp, u.tile);
  const AttnSeq s = found.at.seq;
  const int local = found.at.next - 1 - u.tile;   // from the last rows (the most keys when causal) to the first
  const int ns = found.ranges, split = local % ns, rt = local / ns;
  const int shift = s.nk - s.nq, rows = s.nq * G;
  const int row = rt * R + wave * 32 + (lane & 31);
  const int tok = min(row, rows - 1) / G, head = u.kvh * G + min(row, rows - 1) % G;
  auto sees = [&](int r) { return visible(min(r, rows - 1) / G + shift, s.nk, a.f.causal, a.f.window); };
  const Range mine = visible(tok + shift, s.nk, a.f.causal, a.f.window);
  const Range wa = sees(rt * R + wave * 32), wb = sees(rt * R + wave * 32 + 31);   // of the wave's first and last row
  const int lo = found.lo, chunk = found.chunk;
  const int k_lo = lo + max((sees(rt * R).lo - lo) & ~(BN - 1), split * chunk);
  const int k_hi = min(sees(rt * R + R - 1).hi, lo + (split + 1) * chunk);
  const int nt = k_hi > k_lo ? (k_hi - k_lo + BN - 1) / BN : 0;
  const int64_t kbase = (s.k0 + k_lo) * a.k4.token + (int64_t)u.kvh * a.k4.head, vbase = (s.k0 + k_lo) * a.v4.token + (int64_t)u.kvh * a.v4.head;
  typedef Kv4Many<DP, WV> Many;
  Many codes;
  auto load = [&](int t) __attribute__((always_inline)) {   // past the last tile the last one again
    const int at = min(t, nt - 1) * BN;
    codes.load(a, kbase + (int64_t)at * a.k4.token, vbase + (int64_t)at * a.v4.token, k_hi - 1 - (k_lo + at), tid);
  };
  if (nt > 0) load(0);
  Deq::share(tables, tid, a.t, a.unit);
  bf16x8 qf[KS];
  {
    const uint16_t* q = a.f.q.p + (s.q0 + tok) * a.f.q.token + (int64_t)head * a.f.q.head;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int col = 8 * (2 * ks + (lane >> 5));
      u32x4 v = u32x4{0u, 0u, 0u, 0u};
      if (row < rows && col < a.f.d) v = *reinterpret_cast<const u32x4*>(q + col);
      qf[ks] = __builtin_bit_cast(bf16x8, kv4_order(v));
    }
  }
  Online<DT> acc;
  acc.init();
  const float slack = slack_of(a.f.c);
  if (nt > 0) {
    lds_barrier();   // the tables are there
    codes.template store<Deq>(K0, V0, tables, a, tid);
    load(1);
  }
  // tile t is in (Kt, Vt); tile t + 1 is made in (kn, vn). No branches around the products: a wave whose rows see nothing of a
  // tile hides all of it (branches made the compiler move the outputs between registers, 81 us against 76)
  auto tile = [&](int t, const uint16_t* Kt, const uint16_t* Vt, uint16_t* kn, uint16_t* vn) __attribute__((always_inline)) {
    lds_barrier();   // tile t is in, and every wave is done with tile t - 1
    codes.template store<Deq>(kn, vn, tables, a, tid);
    load(t + 2);
    const int j0 = k_lo + t * BN;
    f32x16 sc[2];
    bf16x8 f[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) f[ks] = T::rows(Kt, 0, ks, lane);
    sc[0] = zero16();
    sc[1] = zero16();
    keep_order();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      sc[0] = mfma(f[ks], qf[ks], sc[0]);
      f[ks] = T::rows(Kt, 32, ks, lane);
      keep_order();
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      sc[1] = mfma(f[ks], qf[ks], sc[1]);
      f[ks] = T::cols(Vt, 16 * (ks / DT), ks % DT, lane);
      keep_order();
    }
    if (j0 + BN > wa.hi || j0 < wb.lo) {
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) hide(sc[kt], mine, j0 + 32 * kt, lane, -INFINITY);
    }
    acc.update(sc, a.f.c, slack);
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      acc.o[i % DT] = mfma(f[i], pack8(sc[0], i / DT), acc.o[i % DT]);
      f[i] = T::cols(Vt, 32 + 16 * (i / DT), i % DT, lane);
    }
#pragma unroll
    for (int i = 0; i < KS; ++i) acc.o[i % DT] = mfma(f[i], pack8(sc[1], i / DT), acc.o[i % DT]);
  };
  for (int t = 0; t < nt; t += 2) {
    tile(t, K0, V0, K1, V1);
    if (t + 1 < nt) tile(t + 1, K1, V1, K0, V0);
  }

  const float l = half_sum(acc.l);
  const bool in = row < rows;   // both lanes of a row alike
  if (ns == 1) {
    const float inv = inverse_sum(l);
    uint16_t* o = a.f.o.p + (s.q0 + tok) * a.f.o.token + (int64_t)head * a.f.o.head;
#pragma unroll
    for (int i = 0; i < 2 * DT; ++i) {
      const int c = 16 * i + 8 * (lane >> 5);
      float v[8];
      kv4_columns(v, acc.o[i / 2], 2 * (i & 1));
      if (in && c < a.f.d)
        *reinterpret_cast<u32x4*>(o + c) = u32x4{pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv),
                                                 pack_bf16x2(v[4] * inv, v[5] * inv), pack_bf16x2(v[6] * inv, v[7] * inv)};
    }
    if (in && a.f.lse && lane < 32) a.f.lse[(int64_t)head * a.f.lse_stride + s.q0 + tok] = lse_of(acc.mc, l);
  } else {
    float* part = sp.part + (found.row0 + ((int64_t)row * a.f.kv_heads + u.kvh) * ns + split) * (int64_t)(a.f.d + 8);
#pragma unroll
    for (int i = 0; i < 2 * DT; ++i) {
      const int c = 16 * i + 8 * (lane >> 5);
      float v[8];
      kv4_columns(v, acc.o[i / 2], 2 * (i & 1));
      if (in && c < a.f.d) {
        *reinterpret_cast<f32x4*>(part + c) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4*>(part + c + 4) = f32x4{v[4], v[5], v[6], v[7]};
      }
    }
    if (in && lane < 32) {
      part[a.f.d] = l == 0.f ? -INFINITY : acc.mc;   // finite (0 at least) where the sum is NaN: the join reads it
      part[a.f.d + 1] = l;
    }
  }
}

// ------------------------------------------------------------------------------------------
// Joins the ranges: an item is a row and key head of a sequence of several ranges. 32 lanes hold its columns, 4 each; S groups
// of them take its ranges in turn, four at a time on their way, and are joined in order. Bound by memory where rows are many
// (2048 workgroups of 8 items of 2 ranges, 6 us) and by latency where ranges are (3.6 us for 32 items, 6.5 for 128 of over 90).
// S = 8 for more than 4 ranges, else 1: the whole attention of 8 rows over 130000 keys takes 52 us with 8 and 68 with 1, that of
// two times 2048 rows over 4000 keys (2 ranges) 110 with 8 and 86 with 1.
template <int S>
__global__ __launch_bounds__(256) void attn_kv4_join_kernel(const AttnFwdArgs a, const AttnSeqs sq, const Kv4Split sp) {
  constexpr int ITEMS = 8 / S;
  const int lane = threadIdx.x & 63, grp = (int)threadIdx.x >> 5;
  const int G = a.heads / a.kv_heads;
  const int slice = grp % S;
  // sequences with one range have no items; as kv4_find, one trip to the arguments
  const int f = lane < sq.count ? sp.join_first[lane] : 0x7FFFFFFF, next = sp.join_first[lane + 1], ranges = sp.ranges[lane];
  const int64_t row0 = sp.row0[lane], q0 = sq.seq[lane].q0;
  const int all = lane_value(next, sq.count - 1);
  const int want = (int)blockIdx.x * ITEMS + grp / S, item = min(want, all - 1);
  const int i0 = __builtin_amdgcn_readfirstlane(item);
  int si = (int)__popcll(__ballot(f <= i0)) - 1;
  int first = lane_value(f, si), ns = lane_value(ranges, si);
  int64_t base = lane_value(row0, si), tok0 = lane_value(q0, si);
  if (ITEMS > 1 && __any(item >= lane_value(next, si))) {   // the wave's second item is of a later sequence
    while (item >= sp.join_first[si + 1]) ++si;
    first = sp.join_first[si];
    ns = sp.ranges[si];
    base = sp.row0[si];
    tok0 = sq.seq[si].q0;
  }
  const int local = item - first;
  const int grow = local / a.kv_heads, kvh = local % a.kv_heads;
  const int tok = grow / G, head = kvh * G + grow % G;
  const int64_t step = a.d + 8;
  const float* part = sp.part + (base + (int64_t)local * ns) * step;
  const int c = 4 * (lane & 31), cc = min(c, a.d - 4);   // d is a multiple of 8
  float mx = -INFINITY, l = 0.f;
  f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k0 = slice; k0 < ns; k0 += 4 * S) {
    float m[4], lk[4];
    f32x4 x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float* p = part + min(k0 + q * S, ns - 1) * step;
      x[q] = *reinterpret_cast<const f32x4*>(p + cc);
      m[q] = p[a.d];
      lk[q] = p[a.d + 1];
    }
    float top = mx;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (k0 + q * S >= ns) m[q] = -INFINITY;
      top = fmaxf(top, m[q]);
    }
    if (top == -INFINITY) continue;
    const float g = __builtin_amdgcn_exp2f(mx - top);   // 0 while nothing was seen
    l *= g;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] *= g;
    mx = top;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (m[q] == -INFINITY) continue;   // past the end, or a range that the row sees nothing of
      const float w = __builtin_amdgcn_exp2f(m[q] - top);
      l = __fmaf_rn(w, lk[q], l);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __fmaf_rn(w, x[q][e], v[e]);
    }
  }
  if constexpr (S > 1) {
    __shared__ float ms[S], ls[S];
    __shared__ __attribute__((aligned(16))) float vs[S][128];
    if ((lane & 31) == 0) {
      ms[slice] = mx;
      ls[slice] = l;
    }
    *reinterpret_cast<f32x4*>(&vs[slice][4 * (lane & 31)]) = v;
    __syncthreads();
    if (slice) return;
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < S; ++k) top = fmaxf(top, ms[k]);
    l = 0.f;
    v = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const float w = ms[k] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ms[k] - top);
      l += ls[k] * w;   // 0 times NaN stays NaN
      const f32x4 x = *reinterpret_cast<const f32x4*>(&vs[k][4 * (lane & 31)]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __fmaf_rn(w, x[e], v[e]);
    }
    mx = top;
  }
  if (want >= all) return;
  const float inv = inverse_sum(l);
  if (c < a.d)
    *reinterpret_cast<u32x2*>(a.o.p + (tok0 + tok) * a.o.token + (int64_t)head * a.o.head + c) =
        u32x2{pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv)};
  if (a.lse && (lane & 31) == 0) a.lse[(int64_t)head * a.lse_stride + tok0 + tok] = lse_of(mx, l);
}

// ------------------------------------------------------------------------------------------
// Host side: launches
size_t attn_kv4_ws_floats(const AttnSeq* seqs, int64_t count, int book, int heads, int kv_heads, int d, int window) {
  return (size_t)kv4_plan(seqs, count, book, heads, kv_heads, d, window).part_floats;
}

template <int DP, class Deq>
static void kv4_launch(int kernel, const AttnKv4Args& a, const AttnSeqs& q, const Kv4Split& sp, hipStream_t stream) {
  const dim3 grid((unsigned)(q.first[q.count] * a.f.kv_heads)), wg((unsigned)kKv4Kernels[kernel].waves * 64);
  switch (kernel) {
    case 0: hipLaunchKernelGGL((attn_kv4_few_kernel<DP, Deq, 1>), grid, wg, 0, stream, a, q, sp); break;
    case 1: hipLaunchKernelGGL((attn_kv4_few_kernel<DP, Deq, 2>), grid, wg, 0, stream, a, q, sp); break;
    case 2: hipLaunchKernelGGL((attn_kv4_many_kernel<DP, Deq, 4>), grid, wg, 0, stream, a, q, sp); break;
    default: hipLaunchKernelGGL((attn_kv4_many_kernel<DP, Deq, 8>), grid, wg, 0, stream, a, q, sp); break;
  }
}

hipError_t launch_attn_kv4(const AttnKv4Args& a, int book, const AttnSeq* seqs, int64_t count, float* ws, size_t ws_floats,
                           bool* fits, hipStream_t stream) {
  const Kv4Plan plan = kv4_plan(seqs, count, book, a.f.heads, a.f.kv_heads, a.f.d, a.f.window);
  *fits = !plan.part_floats || (ws && ws_floats >= (size_t)plan.part_floats);
  if (!*fits || (plan.few.seqs.empty() && plan.many.seqs.empty())) return hipSuccess;
  const int G = a.f.heads / a.f.kv_heads;
  for (const Kv4Class* c : {&plan.few, &plan.many}) {
    for (size_t from = 0; from < c->seqs.size();) {
      const AttnSeqs q = kv4_seqs(*c, from, G, a.f.kv_heads, a.f.window);
      from += (size_t)q.count;
      Kv4Split sp{};
      sp.part = ws;
      int64_t row0 = 0;
      int most = 0;
      for (int i = 0; i < q.count; ++i) {
        const int n = c->ranges(q.seq[i], a.f.window);
        sp.lo[i] = (int)first_key(q.seq[i], a.f.window);
        sp.ranges[i] = n;
        sp.chunk[i] = (int)(ceil64(ceil64(kv4_keys(q.seq[i], a.f.window), n), c->k().step) * c->k().step);   // equal ranges
        sp.row0[i] = row0;
        const int64_t items = n > 1 ? (int64_t)q.seq[i].nq * a.f.heads : 0;
        row0 += items * n;
        sp.join_first[i + 1] = sp.join_first[i] + (int)items;
        most = std::max(most, n);
      }
      if (a.f.d <= 64) {
        if (book == 1) kv4_launch<64, Kv4E2m1>(c->kernel, a, q, sp, stream);
        else kv4_launch<64, Kv4Table>(c->kernel, a, q, sp, stream);
      } else {
        if (book == 1) kv4_launch<128, Kv4E2m1>(c->kernel, a, q, sp, stream);
        else kv4_launch<128, Kv4Table>(c->kernel, a, q, sp, stream);
      }
      const int items = sp.join_first[q.count];
      if (items && most > 4) hipLaunchKernelGGL(attn_kv4_join_kernel<8>, dim3((unsigned)items), dim3(256), 0, stream, a.f, q, sp);
      else if (items) hipLaunchKernelGGL(attn_kv4_join_kernel<1>, dim3((unsigned)((items + 7) / 8)), dim3(256), 0, stream, a.f, q, sp);
    }
  }
  return hipGetLastError();
}

}  // namespace nf4
