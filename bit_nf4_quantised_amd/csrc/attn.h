// What the attention kernels share (gfx950): tiles in LDS, products of rows and tiles, masks, the running
// softmax, work lists of sequences, and the host's helpers that make them.
#pragma once
#include "common.h"
#include "launch.h"

#include <limits.h>

#include <algorithm>
#include <vector>

namespace nf4 {

typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A row's reference maximum is raised only when a new score passes it by more than this many powers
// of two: until then the probabilities of the row grow to at most 2^kSlack, which costs no accuracy
// in fp32 sums and bf16 operands (both are relative), and the output is not rescaled.
constexpr float kSlack = 8.f;
// the same as raw scores (finite for every scale: the first score always passes -inf plus this)
__device__ __forceinline__ float slack_of(float c) { return fminf(kSlack / c, 1e30f); }

// ------------------------------------------------------------------------------------------
// LDS tiles: rows of DP bf16 in 16-byte chunks; chunk c of row m sits at slot c ^ swz(m). 16
// consecutive rows at one chunk (operand reads along a row) and 4 aligned rows at 4 aligned chunks
// (transpose reads) both fall on 16 different 16-byte bank groups.
template <int DP>
struct Tile {
  static constexpr int kChunks = DP / 8;
  static __device__ __forceinline__ int swz(int m) {
    return DP == 128 ? (((m & 3) << 2) | ((m >> 2) & 3)) : ((((m >> 1) & 1) << 2) | ((m >> 2) & 3));
  }
  static __device__ __forceinline__ int elem(int m, int c) { return m * DP + ((c ^ swz(m)) << 3); }

  // operand whose rows are tile rows m0 .. m0+31 and whose contraction runs along the tile's
  // columns 16 ks .. 16 ks + 15
  static __device__ __forceinline__ bf16x8 rows(const uint16_t* t, int m0, int ks, int lane) {
    const int m = lane & 31;
    return *reinterpret_cast<const bf16x8*>(t + m0 * DP + elem(m, 2 * ks + (lane >> 5)));
  }
  // operand whose rows are tile columns 32 dt .. 32 dt + 31 and whose contraction runs over tile rows
  // m0 .. m0+15 (m0 a multiple of 16) in the order of a score accumulator: lane half h takes rows
  // 4 h .. 4 h + 3, then 8 + 4 h .. 8 + 4 h + 3
  static __device__ __forceinline__ bf16x8 cols(const uint16_t* t, int m0, int dt, int lane) {
    const int j = lane & 15, h = lane >> 5;
    const int m = 4 * h + (j >> 2), c = 4 * dt + 2 * ((lane >> 4) & 1) + ((j & 3) >> 1);
    const uint16_t* base = t + m0 * DP + 4 * (j & 1);
    bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(base + elem(m, c)));
    bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(base + elem(m + 8, c)));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// LDS-DMA of ROWS x DP into a tile by NW waves: rows past `rows` and columns past d become zeros.
template <int DP, int ROWS, int NW>
struct TileDma {
  static constexpr int kLoads = ROWS * (DP / 8) / 64 / NW;   // per wave
  static_assert(kLoads >= 1, "a wave loads 1 KiB at least");
  uint32_t off[kLoads];
  __device__ __forceinline__ void init(int wave, int lane, int d, uint32_t stride) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int slot = (wave * kLoads + j) * 64 + lane;
      const int row = slot / Tile<DP>::kChunks, c = (slot % Tile<DP>::kChunks) ^ Tile<DP>::swz(row);
      off[j] = 8 * c < d ? (uint32_t)row * stride * 2u + (uint32_t)c * 16u : kOutOfRange;
    }
  }
  // base: the tile's first row; rows >= 0 valid rows
  __device__ __forceinline__ void load(uint16_t* tile, const uint16_t* base, int rows, int d, uint32_t stride,
                                       int wave) const {
    const uint32_t nrec = rows > 0 ? ((uint32_t)(min(rows, ROWS) - 1) * stride + (uint32_t)d) * 2u : 0u;
    __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, (int)nrec, kRsrcFlags);
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(tile + (wave * kLoads + j) * 512), 16, off[j], 0, 0, 0);
  }
};

// Keys and values of one key head of a sequence, streamed in tiles of ROWS.
template <int DP, int ROWS, int NW>
struct KvStream {
  typedef TileDma<DP, ROWS, NW> Dma;
  static constexpr int kLoads = 2 * Dma::kLoads;   // per wave and tile
  Dma kd, vd;
  const uint16_t *k, *v;
  uint32_t ks, vs;
  int nk, d;
  __device__ __forceinline__ void init(const AttnTensor& kt, const AttnTensor& vt, const AttnSeq& s, int kvh, int dd, int wave,
                                       int lane) {
    ks = (uint32_t)kt.token;
    vs = (uint32_t)vt.token;
    nk = s.nk;
    d = dd;
    k = kt.p + s.k0 * kt.token + (int64_t)kvh * kt.head;
    v = vt.p + s.k0 * vt.token + (int64_t)kvh * vt.head;
    kd.init(wave, lane, d, ks);
    vd.init(wave, lane, d, vs);
  }
  __device__ __forceinline__ void load(uint16_t* kt, uint16_t* vt, int j, int wave) const {   // keys from j
    kd.load(kt, k + (int64_t)j * ks, nk - j, d, ks, wave);
    vd.load(vt, v + (int64_t)j * vs, nk - j, d, vs, wave);
  }
};

// Rows in registers as the operand whose columns are those rows (contraction along d): lane column
// lane % 32, chunk 2 ks + lane / 32 for every ks. `row` is the lane's row, or null for zeros.
template <int DP>
__device__ __forceinline__ void load_rows(bf16x8 (&f)[DP / 16], const uint16_t* row, int d, int lane) {
#pragma unroll
  for (int ks = 0; ks < DP / 16; ++ks) {
    const int c = 8 * (2 * ks + (lane >> 5));
    u32x4 v = u32x4{0u, 0u, 0u, 0u};
    if (row && c < d) v = *reinterpret_cast<const u32x4*>(row + c);
    f[ks] = __builtin_bit_cast(bf16x8, v);
  }
}

// the instructions before stay before, those after stay after
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// maximum and sum over the two lane halves (lane and lane ^ 32), in both
__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// accumulator rows 8 s .. 8 s + 7 of the lane (s = 0, 1) as an operand fragment
__device__ __forceinline__ bf16x8 pack8(const f32x16& v, int s) {
  u32x4 p;
#pragma unroll
  for (int k = 0; k < 4; ++k) p[k] = pack_bf16x2(v[8 * s + 2 * k], v[8 * s + 2 * k + 1]);
  return __builtin_bit_cast(bf16x8, p);
}

// Ties a value to its place in the program. Used in blocks that few iterations need, which the compiler
// would otherwise run every time, with selects.
__device__ __forceinline__ void pin(f32x16& v) { asm volatile("" : "+v"(v)); }

// index of accumulator element i of this lane among the 32 result rows
__device__ __forceinline__ int acc_row(int i, int lane) { return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3); }

struct Range {
  int lo, hi;
};
// result rows r0 .. r0 + 31 outside [r.lo, r.hi) become `value`
__device__ __forceinline__ void hide(f32x16& v, Range r, int r0, int lane, float value) {
  pin(v);
  const int lo = r.lo - r0 - 4 * (lane >> 5);
  const uint32_t n = (uint32_t)max(r.hi - r.lo, 0);
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if ((uint32_t)(8 * (i >> 2) + (i & 3) - lo) >= n) v[i] = value;
}

// Stores a 32-row result tile (rows: columns 32 dt .. of a token's head, columns: tokens) as bf16:
// lane halves exchange groups of four so that every lane writes 16 contiguous bytes. dst: the lane's
// token and head, or null.
__device__ __forceinline__ void store_cols(uint16_t* dst, const f32x16& v, float scale, int dt, int d, int lane) {
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    u32x2 a, b;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      a[k] = pack_bf16x2(v[8 * g + 2 * k] * scale, v[8 * g + 2 * k + 1] * scale);
      b[k] = pack_bf16x2(v[8 * g + 4 + 2 * k] * scale, v[8 * g + 4 + 2 * k + 1] * scale);
    }
    const auto x = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
    const auto y = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
    const int c = 32 * dt + 16 * g + 8 * (lane >> 5);
    if (dst && c < d) *reinterpret_cast<u32x4*>(dst + c) = u32x4{x[0], y[0], x[1], y[1]};
  }
}

// ------------------------------------------------------------------------------------------
// Work lists. A launch takes up to kAttnSeqs sequences by value; workgroup indexes count tiles of
// the sequences in turn (first[s] .. first[s + 1] - 1 belong to sequence s).
// The sequence of a tile. Lane i reads sequence i's entries, all at once: read one after the other as the
// search goes, they cost a workgroup's start two more trips to the kernel arguments (a causal sequence of
// 2048, 32 heads over 8, forward and backward 249 us against 244).
struct Found {
  int index, first, next;   // the sequence, its first tile, the next sequence's
  AttnSeq seq;
};
__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ int64_t lane_value(int64_t v, int lane) {
  return (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)v, lane) | ((int64_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32);
}
__device__ __forceinline__ Found find_seq(const AttnSeqs& sq, int tile) {
  const int lane = threadIdx.x & 63;
  const int f = sq.first[lane], n = sq.first[lane + 1];
  const AttnSeq s = sq.seq[lane];
  Found r;
  r.index = __builtin_amdgcn_readfirstlane((int)__popcll(__ballot(lane < sq.count && f <= tile)) - 1);
  r.first = lane_value(f, r.index);
  r.next = lane_value(n, r.index);
  r.seq.q0 = lane_value(s.q0, r.index);
  r.seq.k0 = lane_value(s.k0, r.index);
  r.seq.nq = lane_value(s.nq, r.index);
  r.seq.nk = lane_value(s.nk, r.index);
  return r;
}

// Workgroup b of a launch over tiles x kv_heads x per (`per`: workgroups that share a tile and a key
// head). Consecutive workgroups go to the 8 XCDs in turn; with a multiple of 8 key heads each XCD
// takes its own heads, so their keys and values stay in its L2. Tiles vary slowest: the host orders
// them by falling work. `pairs`: the second workgroup of every compute unit (workgroups 256 to 511) comes
// from the other end, so that a unit that began with the most work goes on with the least.
struct Unit {
  int tile, kvh, sub;
};
__device__ __forceinline__ Unit unit_of(int b, int kv_heads, int per, bool pairs = false) {
  Unit u;
  if (pairs && b >= 256 && b < 512) {
    const int x = b & 7, m = (min((int)gridDim.x, 512) - 256 - x + 7) >> 3;   // of this XCD
    b = 256 + x + 8 * (m - 1 - ((b - 256) >> 3));
  }
  if (kv_heads % 8 == 0) {
    const int hx = kv_heads / 8, i = b >> 3;
    u.sub = i % per;
    u.kvh = (b & 7) * hx + (i / per) % hx;
    u.tile = i / (per * hx);
  } else {
    u.sub = b % per;
    u.kvh = (b / per) % kv_heads;
    u.tile = b / (per * kv_heads);
  }
  return u;
}

// visible keys [lo, hi) of the query at position p
__device__ __forceinline__ Range visible(int p, int nk, int causal, int window) {
  Range r;
  r.hi = causal ? min(nk, p + 1) : nk;
  r.lo = window ? max(0, p - window + 1) : 0;
  return r;
}

// A row's sum l is exactly 0 when the row saw no key, and NaN once a score was NaN (which no maximum shows:
// fmaxf drops it, and the reference maximum may still be -inf). So l alone tells a row without keys, which
// gives 0 and -inf, from one that is lost, which gives NaN, on every path alike.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float lse_of(float mc, float l) { return l == 0.f ? -INFINITY : mc * kLn2 + __logf(l); }

// Running softmax of a wave's 32 owned rows (one per lane column) over NT blocks of 32 streamed keys.
template <int DT>
struct Online {
  float m, mc, l;     // reference maximum (raw score), m * c (0 while no key was seen), the lane's part of the sum
  f32x16 o[DT];       // unnormalised output, rows d, columns owned rows
  __device__ __forceinline__ void init() {
    m = -INFINITY;
    mc = 0.f;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < DT; ++i) o[i] = zero16();
  }
  template <int NT>
  __device__ __forceinline__ void update(f32x16 (&s)[NT], float c, float slack) {
    float mx = -INFINITY;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[t][i]);
    mx = half_max(mx);
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
        for (int i = 0; i < 16; ++i) o[k][i] *= a;
    }
    float sum = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[t][i] = __builtin_amdgcn_exp2f(__fmaf_rn(s[t][i], c, -mc));
        sum += s[t][i];
      }
    l += sum;
  }
};

// ------------------------------------------------------------------------------------------
// Host side: sequences in order of falling length, in launches of up to kAttnSeqs.
constexpr int64_t kAttnGroups = kMaxThreads / 256;   // workgroups of a launch

inline int64_t ceil64(int64_t x, int64_t y) { return (x + y - 1) / y; }

// the heaviest sequences first, so that the last workgroups to start are short ones
inline std::vector<AttnSeq> by_work(const AttnSeq* seqs, int64_t count, bool keys) {
  std::vector<AttnSeq> v;
  v.reserve((size_t)count);
  for (int64_t i = 0; i < count; ++i)
    if (keys ? seqs[i].nk > 0 : seqs[i].nq > 0) v.push_back(seqs[i]);
  std::stable_sort(v.begin(), v.end(), [](const AttnSeq& x, const AttnSeq& y) { return x.nk > y.nk; });
  return v;
}

// The sequences of one launch from v[from] on, `tiles_of(seq)` workgroup tiles each and `per_tile` workgroups a
// tile: up to kAttnSeqs, and no more workgroups than a launch holds (`most`; by default those of 256 threads). One
// sequence alone always fits (the entry points refuse those that do not).
template <typename F>
inline AttnSeqs pack_seqs(const std::vector<AttnSeq>& v, size_t from, int64_t per_tile, F tiles_of,
                          int64_t most = kAttnGroups) {
  AttnSeqs q{};
  for (size_t i = from; i < v.size() && q.count < kAttnSeqs; ++i) {
    const int64_t end = q.first[q.count] + (int64_t)tiles_of(v[i]);
    if (q.count && end * per_tile > most) break;
    q.seq[q.count] = v[i];
    q.first[q.count + 1] = (int)end;
    ++q.count;
  }
  return q;
}

inline int padded_d(int d) { return d <= 64 ? 64 : 128; }

// first key that the first row of the sequence can see
inline int64_t first_key(const AttnSeq& s, int window) {
  return window ? std::max<int64_t>(0, (int64_t)s.nk - s.nq - window + 1) : 0;
}

}  // namespace nf4
